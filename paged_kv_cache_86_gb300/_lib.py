"""ctypes binding of libpkv (include/pkv.h): argument marshalling only.

Every function here takes torch tensors that already live on the GPU, checks
their dtype/shape/contiguity, passes raw device pointers and sizes to the C
entry point of the same name on the tensors' current CUDA stream, and turns a
non-zero status into :class:`PkvError`. No attention arithmetic happens here.
The library is built in-tree (``paged_kv_cache_86_gb300/libpkv.so``); if it is
missing, loading raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_BF16 = 0
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "unsupported dtype",
          -4: "workspace missing, misaligned or too small", -5: "CUDA runtime error",
          -6: "device-side range check fired"}
DEVERR_SLOT, DEVERR_BLOCK_ID, DEVERR_LENGTH, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEVERR_NO_BLOCKS, DEVERR_TREE = 0x10, 0x20

EXPORTED = ("pkv_store_kvcache", "pkv_decode_workspace_size", "pkv_paged_decode",
            "pkv_prefill_workspace_size", "pkv_paged_prefill", "pkv_get_device_errors",
            "pkv_status_string", "pkv_version", "pkv_qk_norm_rope", "pkv_qk_norm_rope_store",
            "pkv_plan_slots", "pkv_tree_masks", "pkv_tree_decode_workspace_size",
            "pkv_tree_decode", "pkv_store_kvcache_fp8_block", "pkv_load_kvcache_fp8_block",
            "pkv_decode_window_workspace_size", "pkv_paged_decode_window",
            "pkv_paged_decode_fp8_block", "pkv_paged_prefill_window")


class PkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load libpkv.so and declare the C signatures. Raises if it is not built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ImportError(f"libpkv.so is not built ({path}); run "
                              "`python -m paged_kv_cache_86_gb300.build`")
        lib = ctypes.CDLL(path)
        vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                 ctypes.c_size_t)
        lib.pkv_store_kvcache.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i64, i64,
                                          ctypes.c_int, vp]
        lib.pkv_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pkv_decode_workspace_size.restype = sz
        lib.pkv_paged_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                         i32, i32, f32, vp, sz, ctypes.c_int, vp]
        lib.pkv_decode_step.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, i32, vp, i32, i32,
                                        i32, i32, i32, i32, i32, f32, vp, sz, ctypes.c_int, vp]
        lib.pkv_store_kvcache_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                              i64, i64, vp]
        lib.pkv_paged_decode_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32,
                                             i32, i32, i32, i32, f32, vp, sz, vp]
        lib.pkv_decode_step_fp8.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, i32, vp,
                                            i32, i32, i32, i32, i32, i32, i32, f32, vp, sz, vp]
        lib.pkv_mixed_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pkv_mixed_workspace_size.restype = sz
        lib.pkv_mixed_step.argtypes = [vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, i32, i32, vp,
                                       i32, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, sz,
                                       ctypes.c_int, vp]
        lib.pkv_copy_blocks.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_int,
                                        vp]
        lib.pkv_prefill_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pkv_prefill_workspace_size.restype = sz
        lib.pkv_paged_prefill.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, vp, i32, i32, i32,
                                          i32, i32, i32, i32, i32, f32, i32, vp, sz, ctypes.c_int,
                                          vp]
        lib.pkv_qk_norm_rope.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, f32, vp, vp,
                                         i32, i32, i32, i32, i32, i32, i32, ctypes.c_int, vp]
        lib.pkv_qk_norm_rope_store.argtypes = [vp, i64, vp, vp, vp, i64, i64, i64, vp, vp, f32, vp,
                                               vp, i32, i32, i32, vp, vp, vp, i32, i32, i32, i32,
                                               i32, i32, ctypes.c_int, vp]
        lib.pkv_plan_slots.argtypes = [vp, vp, i32, vp, i32, vp, i32, vp, vp, vp, vp, i32, vp, vp,
                                       vp, i32, i32, vp]
        lib.pkv_tree_masks.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp]
        lib.pkv_tree_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pkv_tree_decode_workspace_size.restype = sz
        lib.pkv_tree_decode.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, vp, i32, vp, vp, vp, i32,
                                        i32, i32, i32, i32, i32, i32, i32, i32, i32, f32, vp, sz,
                                        ctypes.c_int, vp]
        lib.pkv_store_kvcache_fp8_block.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, vp, i32, vp,
                                                    vp, i32, i32, i32, i32, i32, i32, vp]
        lib.pkv_load_kvcache_fp8_block.argtypes = [vp, vp, i64, i64, vp, vp, vp, vp, vp, i32, vp,
                                                   vp, i32, i32, i32, i32, i32, i32, vp]
        lib.pkv_decode_window_workspace_size.argtypes = [i32, i32, i32, i32]
        lib.pkv_decode_window_workspace_size.restype = sz
        lib.pkv_paged_decode_window.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                                i32, i32, i32, i32, i32, f32, vp, sz,
                                                ctypes.c_int, vp]
        lib.pkv_paged_decode_fp8_block.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, i32, i32,
                                                   i32, i32, i32, i32, i32, i32, i32, f32, vp, sz,
                                                   vp]
        lib.pkv_paged_prefill_window.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, vp, i32, i32,
                                                 i32, i32, i32, i32, i32, i32, i32, i32, f32, vp,
                                                 sz, ctypes.c_int, vp]
        lib.pkv_get_device_errors.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.pkv_selftest_bounded_wait.argtypes = [i32, vp, vp]
        lib.pkv_status_string.argtypes = [ctypes.c_int]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_version.restype = i32
        for name in ("pkv_store_kvcache", "pkv_paged_decode", "pkv_decode_step",
                     "pkv_paged_prefill", "pkv_copy_blocks", "pkv_store_kvcache_fp8",
                     "pkv_paged_decode_fp8", "pkv_decode_step_fp8", "pkv_mixed_step",
                     "pkv_get_device_errors", "pkv_qk_norm_rope", "pkv_qk_norm_rope_store",
                     "pkv_plan_slots", "pkv_tree_masks", "pkv_tree_decode",
                     "pkv_store_kvcache_fp8_block", "pkv_load_kvcache_fp8_block",
                     "pkv_paged_decode_window", "pkv_paged_decode_fp8_block",
                     "pkv_paged_prefill_window", "pkv_selftest_bounded_wait"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int, what: str):
    if status != 0:
        raise PkvError(status, what)


def _stream(t: torch.Tensor, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, ndim=None, contiguous=False, on_gpu=True):
    """dtype, rank and (optionally) dense row-major layout, then the device (unless
    on_gpu is False: the caller checks every tensor's device after every layout).
    The kernels take a raw pointer and assume the layout, so a strided view would
    be misread."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if on_gpu:
        _need_gpu((t, name))


def _need_gpu(*named):
    for t, name in named:
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")


def _out_like(out, q: torch.Tensor) -> torch.Tensor:
    """The caller's output buffer (checked: bf16, contiguous, shaped like q, on q's
    device), or a new one."""
    if out is None:
        return torch.empty_like(q)
    _need(out, "out", torch.bfloat16, q.dim())
    if out.shape != q.shape or not out.is_contiguous() or out.device != q.device:
        raise ValueError("out must be a contiguous tensor shaped like q, on q's device")
    return out


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def version() -> int:
    return load().pkv_version()


def store_kvcache(key, value, k_cache, v_cache, slot_mapping, stream=None) -> None:
    """Write key/value [T, Hkv, D] (token rows may be strided) into the caches
    [NB, bs, Hkv, D] at slot_mapping [T] (int32; negative = skip)."""
    lib = load()
    for t, n in ((key, "key"), (value, "value")):
        _need(t, n, torch.bfloat16, 3)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} rows must be contiguous [Hkv, D] blocks")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    nb, bs, hkv, d = k_cache.shape
    t = slot_mapping.shape[0]
    if v_cache.shape != k_cache.shape or key.shape != (t, hkv, d) or value.shape != (t, hkv, d):
        raise ValueError("shape mismatch between key/value/caches/slot_mapping")
    _check(lib.pkv_store_kvcache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(slot_mapping.contiguous()), t, hkv, d, bs, nb,
                                 key.stride(0), value.stride(0), PKV_BF16,
                                 _stream(k_cache, stream)), "pkv_store_kvcache")


def _need_fp8_cache(k_cache, v_cache, k_scales, v_scales):
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, 4)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache shape mismatch")
    nb, bs, hkv, d = k_cache.shape
    for t, n in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        _need(t, n, torch.float32, 2)
        if t.shape != (nb * bs, hkv) or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous [num_blocks * block_size, Hkv] tensor")
    return nb, bs, hkv, d


def store_kvcache_fp8(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping,
                      stream=None) -> None:
    """Quantize key/value [T, Hkv, 128] bf16 into the fp8 E4M3 caches [NB, bs, Hkv, 128]
    (uint8 codes) and their row scales [NB * bs, Hkv] float32 at slot_mapping [T]."""
    lib = load()
    for t, n in ((key, "key"), (value, "value")):
        _need(t, n, torch.bfloat16, 3)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} rows must be contiguous [Hkv, D] blocks")
    nb, bs, hkv, d = _need_fp8_cache(k_cache, v_cache, k_scales, v_scales)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    t = slot_mapping.shape[0]
    if key.shape != (t, hkv, d) or value.shape != (t, hkv, d):
        raise ValueError("shape mismatch between key/value/caches/slot_mapping")
    _check(lib.pkv_store_kvcache_fp8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(k_scales), _ptr(v_scales),
                                     _ptr(slot_mapping.contiguous()), t, hkv, d, bs, nb,
                                     key.stride(0), value.stride(0), _stream(k_cache, stream)),
           "pkv_store_kvcache_fp8")


def paged_decode_fp8(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                     scale: float, max_context_len: int | None = None, out=None, workspace=None,
                     stream=None) -> torch.Tensor:
    """Decode attention over fp8 E4M3 caches with row scales; returns out [S, Hq, 128] bf16."""
    lib = load()
    _need(q, "q", torch.bfloat16, 3)
    nb, bs, hkv, d = _need_fp8_cache(k_cache, v_cache, k_scales, v_scales)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if not (q.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("decode tensors must be contiguous")
    s, hq, dq = q.shape
    if dq != d:
        raise ValueError("q / cache head_dim mismatch")
    if block_tables.shape[0] != s or context_lens.shape[0] != s:
        raise ValueError("metadata rows must equal the number of sequences")
    mb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = mb * bs
    out = _out_like(out, q)
    need = decode_workspace_size(s, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_paged_decode_fp8(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(k_scales), _ptr(v_scales), _ptr(block_tables), mb,
                                    _ptr(context_lens), s, int(max_context_len), hq, hkv, d, bs, nb,
                                    float(scale), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(q, stream)), "pkv_paged_decode_fp8")
    return out


def decode_step_fp8(q, key_new, value_new, k_cache, v_cache, k_scales, v_scales, block_tables,
                    context_lens, scale: float, max_context_len: int | None = None, out=None,
                    workspace=None, stream=None) -> torch.Tensor:
    """One decode step over fp8 E4M3 caches: quantizes each sequence's newest K/V row
    (key_new / value_new [S, Hkv, 128] bf16, token rows may be strided) into logical
    position context_lens[i] - 1 (codes and row scale), then decodes; returns out
    [S, Hq, 128] bf16."""
    lib = load()
    _need(q, "q", torch.bfloat16, 3)
    for t, n in ((key_new, "key_new"), (value_new, "value_new")):
        _need(t, n, torch.bfloat16, 3)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} rows must be contiguous [Hkv, D] blocks")
    nb, bs, hkv, d = _need_fp8_cache(k_cache, v_cache, k_scales, v_scales)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if not (q.is_contiguous() and block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("decode tensors must be contiguous")
    s, hq, dq = q.shape
    if dq != d:
        raise ValueError("q / cache head_dim mismatch")
    if key_new.shape != (s, hkv, d) or value_new.shape != (s, hkv, d):
        raise ValueError("key_new / value_new must be [S, Hkv, D]")
    if block_tables.shape[0] != s or context_lens.shape[0] != s:
        raise ValueError("metadata rows must equal the number of sequences")
    mb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = mb * bs
    out = _out_like(out, q)
    need = decode_workspace_size(s, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_decode_step_fp8(_ptr(out), _ptr(q), _ptr(key_new), _ptr(value_new),
                                   key_new.stride(0), value_new.stride(0), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                                   _ptr(block_tables), mb, _ptr(context_lens), s,
                                   int(max_context_len), hq, hkv, d, bs, nb, float(scale),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(q, stream)), "pkv_decode_step_fp8")
    return out


def mixed_workspace_size(num_decode_seqs: int, num_q_heads: int, num_kv_heads: int,
                         head_dim: int = 128) -> int:
    return int(load().pkv_mixed_workspace_size(num_decode_seqs, num_q_heads, num_kv_heads,
                                               head_dim))


def mixed_step(q, key, value, slot_mapping, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k,
               block_tables, num_decode_seqs: int, scale: float, max_seqlen_q: int,
               max_seqlen_k: int, out=None, workspace=None, stream=None) -> torch.Tensor:
    """One mixed round: sequences [0, num_decode_seqs) are decode requests with one
    query row each (rows 0..D-1), the rest prefill chunks; every query row's K/V
    (key / value [total_q, Hkv, D]) is stored at slot_mapping first. Returns out
    [total_q, Hq, D] bf16."""
    _need(q, "q", torch.bfloat16, 3, contiguous=True, on_gpu=False)
    for t, n in ((key, "key"), (value, "value")):
        _need(t, n, torch.bfloat16, 3, on_gpu=False)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} rows must be contiguous [Hkv, D] blocks")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4, contiguous=True, on_gpu=False)
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k"),
                 (slot_mapping, "slot_mapping")):
        _need(t, n, torch.int32, 1, contiguous=True, on_gpu=False)
    _need(block_tables, "block_tables", torch.int32, 2, contiguous=True, on_gpu=False)
    _need_gpu((q, "q"), (key, "key"), (value, "value"), (k_cache, "k_cache"),
              (v_cache, "v_cache"), (cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k"),
              (slot_mapping, "slot_mapping"), (block_tables, "block_tables"))
    lib = load()
    total_q, hq, d = q.shape
    nb, bs, hkv, _ = k_cache.shape
    s = cu_seqlens_q.shape[0] - 1
    if (cu_seqlens_k.shape[0] != s + 1 or block_tables.shape[0] != s
            or slot_mapping.shape[0] != total_q or key.shape != (total_q, hkv, d)
            or value.shape != (total_q, hkv, d)):
        raise ValueError("metadata shape mismatch")
    out = _out_like(out, q)
    need = mixed_workspace_size(num_decode_seqs, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_mixed_step(_ptr(out), _ptr(q), _ptr(key), _ptr(value), _ptr(slot_mapping),
                              key.stride(0), value.stride(0), _ptr(k_cache), _ptr(v_cache),
                              _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q),
                              int(max_seqlen_k), _ptr(block_tables), block_tables.shape[1], s,
                              int(num_decode_seqs), total_q, hq, hkv, d, bs, nb, float(scale),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              PKV_BF16, _stream(q, stream)), "pkv_mixed_step")
    return out


def copy_blocks(k_cache, v_cache, src_block_ids, dst_block_ids, num_rows=None,
                stream=None) -> None:
    """Copy rows [0, num_rows[p]) (whole blocks when num_rows is None) of block
    src_block_ids[p] to block dst_block_ids[p] in both caches [NB, bs, Hkv, D]."""
    lib = load()
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache shape mismatch")
    _need(src_block_ids, "src_block_ids", torch.int32, 1)
    _need(dst_block_ids, "dst_block_ids", torch.int32, 1)
    n = src_block_ids.shape[0]
    if dst_block_ids.shape[0] != n:
        raise ValueError("src / dst length mismatch")
    rows_ptr = ctypes.c_void_p(0)
    if num_rows is not None:
        _need(num_rows, "num_rows", torch.int32, 1)
        if num_rows.shape[0] != n:
            raise ValueError("num_rows length mismatch")
        num_rows = num_rows.contiguous()
        rows_ptr = _ptr(num_rows)
    nb, bs, hkv, d = k_cache.shape
    src_block_ids, dst_block_ids = src_block_ids.contiguous(), dst_block_ids.contiguous()
    _check(lib.pkv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(src_block_ids),
                               _ptr(dst_block_ids), rows_ptr, n, hkv, d, bs, nb, PKV_BF16,
                               _stream(k_cache, stream)), "pkv_copy_blocks")


def decode_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                          head_dim: int = 128) -> int:
    return int(load().pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim))


def paged_decode(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                 max_context_len: int | None = None, out=None, workspace=None,
                 stream=None) -> torch.Tensor:
    """Decode attention; returns out [S, Hq, D] bf16.

    ``max_context_len`` is the host-side upper bound of context_lens (defaults
    to the block-table capacity, max_blocks_per_seq * block_size)."""
    lib = load()
    _need(q, "q", torch.bfloat16, 3)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if not (q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("decode tensors must be contiguous")
    s, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("q / cache head_dim mismatch")
    if block_tables.shape[0] != s or context_lens.shape[0] != s:
        raise ValueError("metadata rows must equal the number of sequences")
    mb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = mb * bs
    out = _out_like(out, q)
    need = decode_workspace_size(s, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_paged_decode(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _ptr(block_tables), mb, _ptr(context_lens), s, int(max_context_len),
                                hq, hkv, d, bs, nb, float(scale), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), PKV_BF16,
                                _stream(q, stream)), "pkv_paged_decode")
    return out


def decode_step(q, key_new, value_new, k_cache, v_cache, block_tables, context_lens,
                scale: float, max_context_len: int | None = None, out=None, workspace=None,
                stream=None) -> torch.Tensor:
    """One decode step: writes each sequence's newest K/V row (key_new / value_new
    [S, Hkv, D], token rows may be strided) at its last logical position
    context_lens[i] - 1, then decodes; returns out [S, Hq, D] bf16."""
    lib = load()
    _need(q, "q", torch.bfloat16, 3)
    for t, n in ((key_new, "key_new"), (value_new, "value_new")):
        _need(t, n, torch.bfloat16, 3)
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{n} rows must be contiguous [Hkv, D] blocks")
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(context_lens, "context_lens", torch.int32, 1)
    if not (q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()):
        raise ValueError("decode tensors must be contiguous")
    s, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("q / cache head_dim mismatch")
    if key_new.shape != (s, hkv, d) or value_new.shape != (s, hkv, d):
        raise ValueError("key_new / value_new must be [S, Hkv, D]")
    if block_tables.shape[0] != s or context_lens.shape[0] != s:
        raise ValueError("metadata rows must equal the number of sequences")
    mb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = mb * bs
    out = _out_like(out, q)
    need = decode_workspace_size(s, hq, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(lib.pkv_decode_step(_ptr(out), _ptr(q), _ptr(key_new), _ptr(value_new),
                               key_new.stride(0), value_new.stride(0), _ptr(k_cache),
                               _ptr(v_cache), _ptr(block_tables), mb, _ptr(context_lens), s,
                               int(max_context_len), hq, hkv, d, bs, nb, float(scale),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               PKV_BF16, _stream(q, stream)), "pkv_decode_step")
    return out


def prefill_workspace_size(num_seqs: int, total_q: int, num_q_heads: int,
                           head_dim: int = 128) -> int:
    return int(load().pkv_prefill_workspace_size(num_seqs, total_q, num_q_heads, head_dim))


def paged_prefill(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables, scale: float,
                  max_seqlen_q: int, max_seqlen_k: int, causal: bool = True, out=None,
                  workspace=None, stream=None) -> torch.Tensor:
    """Varlen chunked-prefill attention; returns out [total_q, Hq, D] bf16. Every value of the
    blocks it reads has to be finite, rows behind a sequence's last key among them
    (paged_prefill_window takes any)."""
    named = ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (cu_seqlens_q, "cu_seqlens_q"),
             (cu_seqlens_k, "cu_seqlens_k"), (block_tables, "block_tables"))
    _need(q, "q", torch.bfloat16, 3, contiguous=True, on_gpu=False)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16, 4, contiguous=True, on_gpu=False)
    for t, n in ((cu_seqlens_q, "cu_seqlens_q"), (cu_seqlens_k, "cu_seqlens_k")):
        _need(t, n, torch.int32, 1, contiguous=True, on_gpu=False)
    _need(block_tables, "block_tables", torch.int32, 2, contiguous=True, on_gpu=False)
    _need_gpu(*named)
    lib = load()
    total_q, hq, d = q.shape
    nb, bs, hkv, _ = k_cache.shape
    s = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != s + 1 or block_tables.shape[0] != s:
        raise ValueError("metadata shape mismatch")
    out = _out_like(out, q)
    need = prefill_workspace_size(s, total_q, hq, d)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.pkv_paged_prefill(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), int(max_seqlen_q),
                                 int(max_seqlen_k), _ptr(block_tables), block_tables.shape[1], s,
                                 total_q, hq, hkv, d, bs, nb, float(scale), 1 if causal else 0,
                                 ws_ptr, ws_bytes, PKV_BF16, _stream(q, stream)),
           "pkv_paged_prefill")
    return out


# ------------------------------------------------ drafted rounds on the cache
#
# The smallest of these calls take a few microseconds on the GPU, so each one
# tests its arguments in one expression of plain attribute reads; only when that
# fails does it look for the tensor at fault and name it.

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_MAX_I32 = 0x7fffffff   # windows and sinks beyond it see the same: no context is longer
_MAX_TOKENS = _MAX_I32 - 512   # longest context of the windowed calls
# the current stream's handle without building a Stream object (2 us of a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dense(dtype, ndim, **tensors):
    """dtype, rank and dense row-major layout of each named tensor (see _need)."""
    for name, t in tensors.items():
        _need(t, name, dtype, ndim, contiguous=True, on_gpu=False)


def _rows(**tensors):
    """bf16 [T, H, D] tensors whose token rows are dense [H, D] blocks at any token stride."""
    for name, t in tensors.items():
        _need(t, name, _BF16, 3, on_gpu=False)
        _, h, d = t.shape
        if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
            raise ValueError(f"{name} rows must be contiguous [H, D] blocks")


def _row_stride(t) -> int:
    """Token stride of bf16 [T, H, D] rows, or -1 where _rows tells what is wrong."""
    if t.dtype is not _BF16:
        return -1
    try:
        n, h, d = t.shape
    except ValueError:
        return -1
    st, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        return -1
    return st if n > 1 else h * d   # the stride of a single row is arbitrary and never used


def _refuse_device(**tensors):
    """Raise for the first tensor that is not on the GPU of the ones before it."""
    dev = None
    for name, t in tensors.items():
        if not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not on {dev}")
    raise AssertionError("the tensors share a device")


def _enter(index: int, stream):
    """(context to leave, stream handle): makes GPU `index` current and, when a stream is
    named, that stream too, so that the launch and every buffer allocated until the
    context is left belong to it. None where both are current already."""
    if stream is None:
        if index == torch.cuda.current_device():
            return None, _raw_stream(index)
        ctx = torch.cuda.device(index)
        ctx.__enter__()
        return ctx, _raw_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    ctx = torch.cuda.stream(stream)
    ctx.__enter__()
    return ctx, stream.cuda_stream


def _leave(ctx):
    if ctx is not None:
        ctx.__exit__(None, None, None)


def _check_norm_rope(q, k, positions, cos_sin, q_weight, k_weight):
    """Checks the types, layouts and sizes that both head-norm-and-rotation calls share;
    the token strides of q and k."""
    try:
        qs, ks = _row_stride(q), _row_stride(k)
        fine = (qs >= 0 and ks >= 0 and positions.dtype is _I32 and positions.dim() == 1
                and positions.is_contiguous() and cos_sin.dtype is _F32 and cos_sin.dim() == 2
                and cos_sin.is_contiguous()
                and (q_weight is None or (q_weight.dtype is _BF16 and q_weight.dim() == 1
                                          and q_weight.is_contiguous()))
                and (k_weight is None or (k_weight.dtype is _BF16 and k_weight.dim() == 1
                                          and k_weight.is_contiguous())))
    except AttributeError:
        fine = False
    if not fine:
        _rows(q=q, k=k)
        _dense(_I32, 1, positions=positions)
        _dense(_F32, 2, cos_sin=cos_sin)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _dense(_BF16, 1, **{name: w})
    t, _, d = q.shape
    tk, _, dk = k.shape
    if tk != t or dk != d or positions.numel() != t:
        raise ValueError("shape mismatch between q/k/positions")
    if q_weight is not None and q_weight.numel() != d:
        raise ValueError("q_weight must have head_dim entries")
    if k_weight is not None and k_weight.numel() != d:
        raise ValueError("k_weight must have head_dim entries")
    return qs, ks


def _norm_rope_device(q, k, positions, cos_sin, q_weight, k_weight) -> int:
    """The GPU that all the tensors are on."""
    index = q.get_device()
    if not (index >= 0 and k.get_device() == index and positions.get_device() == index
            and cos_sin.get_device() == index
            and (q_weight is None or q_weight.get_device() == index)
            and (k_weight is None or k_weight.get_device() == index)):
        named = {"q": q, "k": k, "positions": positions, "cos_sin": cos_sin,
                 "q_weight": q_weight, "k_weight": k_weight}
        _refuse_device(**{n: t for n, t in named.items() if t is not None})
    return index


def _check_rows_out(out, like, name: str) -> int:
    """The caller's output rows; their token stride."""
    _rows(**{name: out})
    if out.shape != like.shape or out.device != like.device:
        raise ValueError(f"{name} must be shaped like its input, on the same device")
    return _row_stride(out)


def qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [T, Hq, D] and k [T, Hkv, D] (bf16, token rows may be
    strided; no norm where the weight [D] is None), then the position rotation by
    cos_sin[positions] (float32 [max_position, rotary_dim]: cosines, then sines).
    Returns (q_out, k_out); either may be given, and may be its own input."""
    if q_out is not None:
        qos = _check_rows_out(q_out, q, "q_out")
    if k_out is not None:
        kos = _check_rows_out(k_out, k, "k_out")
    qs, ks = _check_norm_rope(q, k, positions, cos_sin, q_weight, k_weight)
    index = _norm_rope_device(q, k, positions, cos_sin, q_weight, k_weight)
    lib = _lib or load()
    t, hq, d = q.shape
    hkv = k.shape[1]
    max_position, rotary_dim = cos_sin.shape
    ctx, st = _enter(index, stream)
    try:
        if q_out is None:
            q_out, qos = torch.empty((t, hq, d), dtype=_BF16, device=q.device), hq * d
        if k_out is None:
            k_out, kos = torch.empty((t, hkv, d), dtype=_BF16, device=q.device), hkv * d
        status = lib.pkv_qk_norm_rope(
            q_out.data_ptr(), qos, k_out.data_ptr(), kos, q.data_ptr(), k.data_ptr(), qs, ks,
            None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), eps, positions.data_ptr(),
            cos_sin.data_ptr(), max_position, rotary_dim, 1 if interleaved else 0, t, hq, hkv, d,
            PKV_BF16, st)
        if status != 0:
            raise PkvError(status, "pkv_qk_norm_rope")
    finally:
        _leave(ctx)
    return q_out, k_out


def qk_norm_rope_store(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_weight=None,
                       k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                       stream=None) -> torch.Tensor:
    """qk_norm_rope whose key rows go, with the value rows v [T, Hkv, D], into the caches
    [NB, bs, Hkv, D] at slot_mapping [T] (int32; negative = skip). Returns q_out."""
    if q_out is not None:
        qos = _check_rows_out(q_out, q, "q_out")
    qs, ks = _check_norm_rope(q, k, positions, cos_sin, q_weight, k_weight)
    try:
        vs = _row_stride(v)
        fine = (vs >= 0 and k_cache.dtype is _BF16 and k_cache.dim() == 4
                and k_cache.is_contiguous() and v_cache.dtype is _BF16 and v_cache.dim() == 4
                and v_cache.is_contiguous() and slot_mapping.dtype is _I32
                and slot_mapping.dim() == 1 and slot_mapping.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _rows(v=v)
        _dense(_BF16, 4, k_cache=k_cache, v_cache=v_cache)
        _dense(_I32, 1, slot_mapping=slot_mapping)
    t, hq, d = q.shape
    nb, bs, hkv, dc = k_cache.shape
    if (v.shape != k.shape or v_cache.shape != k_cache.shape or (hkv, dc) != k.shape[1:]
            or slot_mapping.shape[0] != t):
        raise ValueError("shape mismatch between k/v/caches/slot_mapping")
    index = _norm_rope_device(q, k, positions, cos_sin, q_weight, k_weight)
    if not (v.get_device() == index and k_cache.get_device() == index
            and v_cache.get_device() == index and slot_mapping.get_device() == index):
        _refuse_device(q=q, v=v, k_cache=k_cache, v_cache=v_cache, slot_mapping=slot_mapping)
    lib = _lib or load()
    ctx, st = _enter(index, stream)
    try:
        if q_out is None:
            q_out, qos = torch.empty((t, hq, d), dtype=_BF16, device=q.device), hq * d
        max_position, rotary_dim = cos_sin.shape
        status = lib.pkv_qk_norm_rope_store(
            q_out.data_ptr(), qos, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
            None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), eps, positions.data_ptr(),
            cos_sin.data_ptr(), max_position, rotary_dim, 1 if interleaved else 0,
            k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), t, hq, hkv, d, bs,
            nb, PKV_BF16, st)
        if status != 0:
            raise PkvError(status, "pkv_qk_norm_rope_store")
    finally:
        _leave(ctx)
    return q_out


class SlotPlan(NamedTuple):
    """What plan_slots computes, all int32 on the GPU."""
    slot_mapping: torch.Tensor   # [max_tokens]
    positions: torch.Tensor      # [max_tokens]
    cu_seqlens_q: torch.Tensor   # [S + 1]
    cu_seqlens_k: torch.Tensor   # [S + 1]
    context_lens: torch.Tensor   # [S], the new tokens included
    free_cursor: torch.Tensor    # [1], behind the blocks taken


def plan_slots(context_lens, new_lens, block_tables, free_blocks, free_cursor, block_size: int,
               num_blocks: int, max_tokens: int, out: SlotPlan | None = None,
               stream=None) -> SlotPlan:
    """Slots, positions and prefix sums of a round in which request i adds new_lens[i] tokens
    to its context_lens[i] cached ones; blocks it lacks are taken from free_blocks [F] at
    free_cursor [1] and entered in its row of block_tables [S, MB] (updated in place).
    Rows behind the last new token, up to max_tokens, get slot -1 and position 0.
    ``out`` may hold the buffers of an earlier plan of the same sizes. The new tensors
    are parts of one buffer."""
    try:
        fine = (context_lens.dtype is _I32 and context_lens.dim() == 1
                and context_lens.is_contiguous() and new_lens.dtype is _I32
                and new_lens.dim() == 1 and new_lens.is_contiguous()
                and free_blocks.dtype is _I32 and free_blocks.dim() == 1
                and free_blocks.is_contiguous() and free_cursor.dtype is _I32
                and free_cursor.dim() == 1 and free_cursor.is_contiguous()
                and block_tables.dtype is _I32 and block_tables.dim() == 2
                and block_tables.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _dense(_I32, 1, context_lens=context_lens, new_lens=new_lens, free_blocks=free_blocks,
               free_cursor=free_cursor)
        _dense(_I32, 2, block_tables=block_tables)
    s, mb = block_tables.shape
    if context_lens.shape[0] != s or new_lens.shape[0] != s or free_cursor.shape[0] != 1:
        raise ValueError("one length and one block table row per request, and one cursor")
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    index = context_lens.get_device()
    if not (index >= 0 and new_lens.get_device() == index and block_tables.get_device() == index
            and free_blocks.get_device() == index and free_cursor.get_device() == index):
        _dense_out_plan(out, max_tokens, s)
        _refuse_device(context_lens=context_lens, new_lens=new_lens, block_tables=block_tables,
                       free_blocks=free_blocks, free_cursor=free_cursor)
    if out is not None:
        _dense_out_plan(out, max_tokens, s)
        if any(t.get_device() != index for t in out):
            _refuse_device(context_lens=context_lens,
                           **{f"out.{n}": t for n, t in zip(SlotPlan._fields, out)})
    lib = _lib or load()
    ctx, st = _enter(index, stream)
    try:
        if out is None:
            buf = torch.empty(2 * max_tokens + 3 * s + 3, dtype=_I32, device=context_lens.device)
            out = SlotPlan(*buf.split_with_sizes((max_tokens, max_tokens, s + 1, s + 1, s, 1)))
        slots, pos, cu_q, cu_k, lens, cursor = out
        _check(lib.pkv_plan_slots(
            context_lens.data_ptr(), new_lens.data_ptr(), s, block_tables.data_ptr(), mb,
            free_blocks.data_ptr(), free_blocks.shape[0], free_cursor.data_ptr(),
            cursor.data_ptr(), slots.data_ptr(), pos.data_ptr(), max_tokens, cu_q.data_ptr(),
            cu_k.data_ptr(), lens.data_ptr(), block_size, num_blocks, st), "pkv_plan_slots")
    finally:
        _leave(ctx)
    return out


def _dense_out_plan(out, max_tokens: int, s: int):
    """The caller's plan buffers."""
    if out is None:
        return
    for name, t, n in zip(SlotPlan._fields, out, (max_tokens, max_tokens, s + 1, s + 1, s, 1)):
        _need(t, f"out.{name}", _I32, 1, contiguous=True, on_gpu=False)
        if t.shape[0] != n:
            raise ValueError(f"out.{name} must have {n} entries")


def tree_masks(parents, cu_seqlens_q, context_lens, max_seqlen_q: int, tree_mask=None,
               positions=None, stream=None):
    """Ancestor masks and positions of drafted trees: parents [total_q] holds each node's
    parent in its own tree (an earlier node, or -1). Returns (tree_mask [total_q, W] int32
    with W = ceil(max_seqlen_q / 32) or the given tensor's width, positions [total_q])."""
    try:
        fine = (parents.dtype is _I32 and parents.dim() == 1 and parents.is_contiguous()
                and cu_seqlens_q.dtype is _I32 and cu_seqlens_q.dim() == 1
                and cu_seqlens_q.is_contiguous() and context_lens.dtype is _I32
                and context_lens.dim() == 1 and context_lens.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _dense(_I32, 1, parents=parents, cu_seqlens_q=cu_seqlens_q, context_lens=context_lens)
    total, s = parents.shape[0], context_lens.shape[0]
    if cu_seqlens_q.shape[0] != s + 1:
        raise ValueError("cu_seqlens_q must have one entry more than context_lens")
    named = {"parents": parents, "cu_seqlens_q": cu_seqlens_q, "context_lens": context_lens}
    if tree_mask is not None:
        _dense(_I32, 2, tree_mask=tree_mask)
        if tree_mask.shape[0] != total:
            raise ValueError("tree_mask must have one row per node")
        named["tree_mask"] = tree_mask
    if positions is not None:
        _dense(_I32, 1, positions=positions)
        if positions.shape[0] != total:
            raise ValueError("positions must have one entry per node")
        named["positions"] = positions
    index = parents.get_device()
    if index < 0 or any(t.get_device() != index for t in named.values()):
        _refuse_device(**named)
    lib = _lib or load()
    ctx, st = _enter(index, stream)
    try:
        if tree_mask is None:
            words = max(0, int(max_seqlen_q) + 31) // 32
            tree_mask = torch.empty((total, words), dtype=_I32, device=parents.device)
        if positions is None:
            positions = torch.empty(total, dtype=_I32, device=parents.device)
        _check(lib.pkv_tree_masks(
            parents.data_ptr(), cu_seqlens_q.data_ptr(), context_lens.data_ptr(), s, total,
            int(max_seqlen_q), tree_mask.data_ptr(), tree_mask.shape[1], positions.data_ptr(),
            st), "pkv_tree_masks")
    finally:
        _leave(ctx)
    return tree_mask, positions


def tree_decode_workspace_size(max_seqlen_q: int, num_q_heads: int, num_kv_heads: int,
                               head_dim: int = 128) -> int:
    return int(load().pkv_tree_decode_workspace_size(max_seqlen_q, num_q_heads, num_kv_heads,
                                                     head_dim))


@functools.lru_cache(maxsize=256)
def _tree_workspace(index: int, max_seqlen_q: int, hq: int, hkv: int, d: int) -> int:
    """The size on device `index`, the current one; at least 256."""
    return max(load().pkv_tree_decode_workspace_size(max_seqlen_q, hq, hkv, d), 256)


def tree_decode(q, key, value, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q,
                tree_mask, scale: float, max_seqlen_q: int, max_context_len: int | None = None,
                out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of drafted rows q [total_q, Hq, 128] over their sequence's context_lens[i]
    cached tokens and the drafted rows key / value [total_q, Hkv, 128] (token rows may be
    strided; not written to the cache) whose bit is set in tree_mask [total_q, W].
    Returns out [total_q, Hq, 128] bf16; rows behind cu_seqlens_q[-1] are not written."""
    try:
        ks, vs = _row_stride(key), _row_stride(value)
        fine = (q.dtype is _BF16 and q.dim() == 3 and q.is_contiguous() and ks >= 0 and vs >= 0
                and k_cache.dtype is _BF16 and k_cache.dim() == 4
                and k_cache.is_contiguous() and v_cache.dtype is _BF16 and v_cache.dim() == 4
                and v_cache.is_contiguous() and block_tables.dtype is _I32
                and block_tables.dim() == 2 and block_tables.is_contiguous()
                and tree_mask.dtype is _I32 and tree_mask.dim() == 2
                and tree_mask.is_contiguous() and context_lens.dtype is _I32
                and context_lens.dim() == 1 and context_lens.is_contiguous()
                and cu_seqlens_q.dtype is _I32 and cu_seqlens_q.dim() == 1
                and cu_seqlens_q.is_contiguous())
    except AttributeError:
        fine = False
    if not fine:
        _dense(_BF16, 3, q=q)
        _rows(key=key, value=value)
        _dense(_BF16, 4, k_cache=k_cache, v_cache=v_cache)
        _dense(_I32, 2, block_tables=block_tables, tree_mask=tree_mask)
        _dense(_I32, 1, context_lens=context_lens, cu_seqlens_q=cu_seqlens_q)
    total, hq, d = q.shape
    nb, bs, hkv, dc = k_cache.shape
    s = context_lens.shape[0]
    if dc != d or v_cache.shape != k_cache.shape:
        raise ValueError("q / cache head_dim mismatch")
    rows = (total, hkv, d)
    if key.shape != rows or value.shape != rows:
        raise ValueError("key / value must be [total_q, Hkv, D]")
    tables, mb = block_tables.shape
    masks, words = tree_mask.shape
    if tables != s or cu_seqlens_q.shape[0] != s + 1 or masks != total:
        raise ValueError("metadata shape mismatch")
    index = q.get_device()
    if not (index >= 0 and key.get_device() == index and value.get_device() == index
            and k_cache.get_device() == index and v_cache.get_device() == index
            and block_tables.get_device() == index and context_lens.get_device() == index
            and cu_seqlens_q.get_device() == index and tree_mask.get_device() == index):
        _refuse_device(q=q, key=key, value=value, k_cache=k_cache, v_cache=v_cache,
                       block_tables=block_tables, context_lens=context_lens,
                       cu_seqlens_q=cu_seqlens_q, tree_mask=tree_mask)
    if max_context_len is None:
        max_context_len = mb * bs
    lib = _lib or load()
    ctx, st = _enter(index, stream)
    try:
        out = _out_like(out, q) if out is not None else torch.empty_like(q)
        if workspace is None:
            workspace = torch.empty(_tree_workspace(index, int(max_seqlen_q), hq, hkv, d),
                                    dtype=torch.uint8, device=q.device)
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on q's device")
        _check(lib.pkv_tree_decode(
            out.data_ptr(), q.data_ptr(), key.data_ptr(), value.data_ptr(), ks, vs,
            k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
            mb, context_lens.data_ptr(), cu_seqlens_q.data_ptr(), tree_mask.data_ptr(), words, s,
            total, int(max_seqlen_q), int(max_context_len), hq, hkv, d, bs, nb, scale,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), PKV_BF16, st),
            "pkv_tree_decode")
    finally:
        _leave(ctx)
    return out


def _clip(n: int) -> int:
    """n as a C int that means the same: ctypes keeps the low 32 bits of a larger one."""
    return n if 0 <= n <= _MAX_I32 else -1 if n < 0 else _MAX_I32


# The calls below check everything in one expression; where it does not hold, their
# _refuse says what is wrong. Where the tensors' GPU is current and no stream is named, they
# launch without _enter: a call on a few sequences is bound by the host.

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(queries, rows, fp8, k_cache, v_cache, k_scales, v_scales, block_tables, **lens):
    """Raise for the first argument with a wrong type, layout or pool shape; return if their
    other shapes or their devices are what was refused."""
    _dense(_BF16, 3, **queries)
    _rows(**rows)
    _dense(_U8 if fp8 else _BF16, 4, k_cache=k_cache, v_cache=v_cache)
    if fp8:
        _dense(_F32, 2, k_scales=k_scales, v_scales=v_scales)
    _dense(_I32, 2, block_tables=block_tables)
    _dense(_I32, 1, **lens)
    nb, _, hkv, _ = k_cache.shape
    if v_cache.shape != k_cache.shape or fp8 and not (k_scales.shape == v_scales.shape
                                                      == (nb, hkv)):
        raise ValueError("caches must be [NB, bs, Hkv, D], their scales [NB, Hkv]")


def store_kvcache_fp8_block(key, value, k_cache, v_cache, k_scales, v_scales, block_tables,
                            cu_seqlens_q, context_lens, stream=None) -> None:
    """Quantize the new rows key / value [total_q, Hkv, 128] bf16 (token rows may be strided)
    into the fp8 E4M3 caches [NB, bs, Hkv, 128] (uint8 codes), whose scales [NB, Hkv] float32
    are one power of two per (block, KV head). Sequence i's rows cu_seqlens_q[i] ..
    cu_seqlens_q[i + 1] - 1 are its last tokens; context_lens[i] counts them. Where a block
    holds older tokens and its scale has to grow, their codes are re-expressed."""
    try:
        nb, bs, hkv, d = k_cache.shape
        total, heads, dim = key.shape
        s, mb = block_tables.shape
        n, = context_lens.shape
        ends, = cu_seqlens_q.shape
        ks, vs, index = _row_stride(key), _row_stride(value), key.get_device()
        fine = (ks >= 0 and vs >= 0 and k_cache.dtype is _U8 and v_cache.dtype is _U8
                and k_scales.dtype is _F32 and v_scales.dtype is _F32
                and block_tables.dtype is _I32 and cu_seqlens_q.dtype is _I32
                and context_lens.dtype is _I32 and k_cache.is_contiguous()
                and v_cache.is_contiguous() and k_scales.is_contiguous()
                and v_scales.is_contiguous() and block_tables.is_contiguous()
                and cu_seqlens_q.is_contiguous() and context_lens.is_contiguous()
                and v_cache.shape == k_cache.shape and k_scales.shape == v_scales.shape
                == (nb, hkv) and heads == hkv and dim == d and value.shape == key.shape
                and n == s and ends == s + 1 and index >= 0 and value.get_device() == index
                and k_cache.get_device() == index and v_cache.get_device() == index
                and k_scales.get_device() == index and v_scales.get_device() == index
                and block_tables.get_device() == index and cu_seqlens_q.get_device() == index
                and context_lens.get_device() == index)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse({}, dict(key=key, value=value), True, k_cache, v_cache, k_scales, v_scales,
                block_tables, cu_seqlens_q=cu_seqlens_q, context_lens=context_lens)
        if key.shape != (key.shape[0],) + k_cache.shape[2:] or value.shape != key.shape:
            raise ValueError("key / value must be [total_q, Hkv, D]")
        if context_lens.shape[0] != s or cu_seqlens_q.shape[0] != s + 1:
            raise ValueError("metadata shape mismatch")
        _refuse_device(key=key, value=value, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
                       v_scales=v_scales, block_tables=block_tables, cu_seqlens_q=cu_seqlens_q,
                       context_lens=context_lens)
    lib = _lib or load()
    here = stream is None and index == _current_device()
    ctx, st = (None, _raw_stream(index)) if here else _enter(index, stream)
    status = lib.pkv_store_kvcache_fp8_block(
        key.data_ptr(), value.data_ptr(), ks, vs, k_cache.data_ptr(), v_cache.data_ptr(),
        k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), mb,
        cu_seqlens_q.data_ptr(), context_lens.data_ptr(), s, total, hkv, d, bs, nb, st)
    if ctx is not None:
        _leave(ctx)
    if status != 0:
        raise PkvError(status, "pkv_store_kvcache_fp8_block")


def load_kvcache_fp8_block(k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                           row_starts, num_rows: int | None = None, key_out=None, value_out=None,
                           stream=None):
    """The tokens of an fp8 cache with block scales back in bf16: position p < context_lens[i]
    of sequence i goes to row row_starts[i] + p (int32 [S], non-decreasing, rows of one
    sequence ending before the next one's start). Returns (key, value) [num_rows, Hkv, 128];
    rows that no sequence has are left as they were. key_out / value_out may be given (token
    rows may be strided); a bf16 block pool [NB, bs, Hkv, 128] viewed as rows is one.
    paged_prefill_window reads such a pool as it is; for paged_prefill and mixed_step the rows
    of value_out behind each sequence's last one have to be finite, so clear a new one first."""
    if (key_out is None) != (value_out is None):
        raise ValueError("key_out and value_out go together")
    if key_out is None and (num_rows is None or num_rows < 0):
        raise ValueError("num_rows must be given, and not negative, without key_out / value_out")
    try:
        nb, bs, hkv, d = k_cache.shape
        s, mb = block_tables.shape
        n, = context_lens.shape
        starts, = row_starts.shape
        index = k_cache.get_device()
        fine = (k_cache.dtype is _U8 and v_cache.dtype is _U8 and k_scales.dtype is _F32
                and v_scales.dtype is _F32 and block_tables.dtype is _I32
                and context_lens.dtype is _I32 and row_starts.dtype is _I32
                and k_cache.is_contiguous() and v_cache.is_contiguous()
                and k_scales.is_contiguous() and v_scales.is_contiguous()
                and block_tables.is_contiguous() and context_lens.is_contiguous()
                and row_starts.is_contiguous() and v_cache.shape == k_cache.shape
                and k_scales.shape == v_scales.shape == (nb, hkv) and n == s and starts == s
                and index >= 0 and v_cache.get_device() == index
                and k_scales.get_device() == index and v_scales.get_device() == index
                and block_tables.get_device() == index and context_lens.get_device() == index
                and row_starts.get_device() == index)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse({}, {}, True, k_cache, v_cache, k_scales, v_scales, block_tables,
                context_lens=context_lens, row_starts=row_starts)
        if context_lens.shape[0] != s or row_starts.shape[0] != s:
            raise ValueError("metadata shape mismatch")
    if key_out is not None:
        if not (isinstance(key_out, torch.Tensor) and isinstance(value_out, torch.Tensor)):
            raise TypeError("key_out and value_out must be torch tensors")
        ks, vs = _row_stride(key_out), _row_stride(value_out)
        if ks < 0 or vs < 0:
            _rows(key_out=key_out, value_out=value_out)
        if num_rows is None:
            num_rows = key_out.shape[0]
        if key_out.shape != (num_rows, hkv, d) or value_out.shape != key_out.shape:
            raise ValueError("key_out / value_out must be [num_rows, Hkv, D]")
    if not fine:
        _refuse_device(k_cache=k_cache, v_cache=v_cache, k_scales=k_scales, v_scales=v_scales,
                       block_tables=block_tables, context_lens=context_lens,
                       row_starts=row_starts)
    if key_out is not None and not key_out.get_device() == value_out.get_device() == index:
        _refuse_device(k_cache=k_cache, key_out=key_out, value_out=value_out)
    lib = _lib or load()
    here = stream is None and index == _current_device()
    ctx, st = (None, _raw_stream(index)) if here else _enter(index, stream)
    try:
        if key_out is None:
            ks = vs = hkv * d
            key_out = torch.empty((num_rows, hkv, d), dtype=_BF16, device=k_cache.device)
            value_out = torch.empty((num_rows, hkv, d), dtype=_BF16, device=k_cache.device)
        _check(lib.pkv_load_kvcache_fp8_block(
            key_out.data_ptr(), value_out.data_ptr(), ks, vs, k_cache.data_ptr(),
            v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
            mb, context_lens.data_ptr(), row_starts.data_ptr(), s, num_rows, hkv, d, bs, nb, st),
            "pkv_load_kvcache_fp8_block")
    finally:
        if ctx is not None:
            _leave(ctx)
    return key_out, value_out


def decode_window_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                 head_dim: int = 128) -> int:
    return int(load().pkv_decode_window_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                       head_dim))


@functools.lru_cache(maxsize=256)
def _decode_window_workspace(index: int, hq: int, hkv: int, d: int) -> int:
    """The size on device `index`, the current one, for any number of sequences; at least 256."""
    return max(load().pkv_decode_window_workspace_size(0, hq, hkv, d), 256)


def _need_workspace(workspace, q):
    """The caller's workspace is dense and on q's device."""
    if workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on q's device")


def paged_decode_fp8_block(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                           scale: float, window: int = 0, sinks: int = 0,
                           max_context_len: int | None = None, out=None, workspace=None,
                           stream=None) -> torch.Tensor:
    """Decode attention over fp8 E4M3 caches [NB, bs, Hkv, 128] with scales [NB, Hkv], one
    query row q [S, Hq, 128] per sequence. window 0: over the whole context; otherwise over
    the last `window` tokens and the first `sinks`. Returns out [S, Hq, 128] bf16."""
    try:
        nb, bs, hkv, d = k_cache.shape
        s, hq, dim = q.shape
        tables, mb = block_tables.shape
        n, = context_lens.shape
        index = q.get_device()
        fine = (q.dtype is _BF16 and k_cache.dtype is _U8 and v_cache.dtype is _U8
                and k_scales.dtype is _F32 and v_scales.dtype is _F32
                and block_tables.dtype is _I32 and context_lens.dtype is _I32
                and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
                and k_scales.is_contiguous() and v_scales.is_contiguous()
                and block_tables.is_contiguous() and context_lens.is_contiguous()
                and v_cache.shape == k_cache.shape and k_scales.shape == v_scales.shape
                == (nb, hkv) and dim == d and tables == s and n == s and index >= 0
                and k_cache.get_device() == index and v_cache.get_device() == index
                and k_scales.get_device() == index and v_scales.get_device() == index
                and block_tables.get_device() == index and context_lens.get_device() == index)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(dict(q=q), {}, True, k_cache, v_cache, k_scales, v_scales, block_tables,
                context_lens=context_lens)
        if dim != d or tables != s or n != s:
            raise ValueError("q / cache / metadata shape mismatch")
        _refuse_device(q=q, k_cache=k_cache, v_cache=v_cache, k_scales=k_scales,
                       v_scales=v_scales, block_tables=block_tables, context_lens=context_lens)
    lib = _lib or load()
    here = stream is None and index == _current_device()
    ctx, st = (None, _raw_stream(index)) if here else _enter(index, stream)
    try:
        out = torch.empty_like(q) if out is None else _out_like(out, q)
        if workspace is None:
            workspace = torch.empty(_decode_window_workspace(index, hq, hkv, d), dtype=_U8,
                                    device=q.device)
        else:
            _need_workspace(workspace, q)
        status = lib.pkv_paged_decode_fp8_block(
            out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), mb,
            context_lens.data_ptr(), s,
            min(mb * bs, _MAX_TOKENS) if max_context_len is None else _clip(max_context_len),
            _clip(window), _clip(sinks),
            hq, hkv, d, bs, nb, scale, workspace.data_ptr(), workspace.nbytes, st)
        if status != 0:
            raise PkvError(status, "pkv_paged_decode_fp8_block")
    finally:
        if ctx is not None:
            _leave(ctx)
    return out


def paged_decode_window(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                        window: int, sinks: int = 0, max_context_len: int | None = None, out=None,
                        workspace=None, stream=None) -> torch.Tensor:
    """Decode attention over the last `window` tokens and the first `sinks` of each sequence
    in bf16 caches [NB, bs, Hkv, 128], one query row q [S, Hq, 128] per sequence. Returns out
    [S, Hq, 128] bf16."""
    try:
        nb, bs, hkv, d = k_cache.shape
        s, hq, dim = q.shape
        tables, mb = block_tables.shape
        n, = context_lens.shape
        index = q.get_device()
        fine = (q.dtype is _BF16 and k_cache.dtype is _BF16 and v_cache.dtype is _BF16
                and block_tables.dtype is _I32 and context_lens.dtype is _I32
                and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
                and block_tables.is_contiguous() and context_lens.is_contiguous()
                and v_cache.shape == k_cache.shape and dim == d and tables == s and n == s
                and index >= 0 and k_cache.get_device() == index and v_cache.get_device() == index
                and block_tables.get_device() == index and context_lens.get_device() == index)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(dict(q=q), {}, False, k_cache, v_cache, None, None, block_tables,
                context_lens=context_lens)
        if dim != d or tables != s or n != s:
            raise ValueError("q / cache / metadata shape mismatch")
        _refuse_device(q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                       context_lens=context_lens)
    lib = _lib or load()
    here = stream is None and index == _current_device()
    ctx, st = (None, _raw_stream(index)) if here else _enter(index, stream)
    try:
        out = torch.empty_like(q) if out is None else _out_like(out, q)
        if workspace is None:
            workspace = torch.empty(_decode_window_workspace(index, hq, hkv, d), dtype=_U8,
                                    device=q.device)
        else:
            _need_workspace(workspace, q)
        status = lib.pkv_paged_decode_window(
            out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            block_tables.data_ptr(), mb, context_lens.data_ptr(), s,
            min(mb * bs, _MAX_TOKENS) if max_context_len is None else _clip(max_context_len),
            _clip(window), _clip(sinks),
            hq, hkv, d, bs, nb, scale, workspace.data_ptr(), workspace.nbytes, PKV_BF16, st)
        if status != 0:
            raise PkvError(status, "pkv_paged_decode_window")
    finally:
        if ctx is not None:
            _leave(ctx)
    return out


def paged_prefill_window(q, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, block_tables,
                         scale: float, window: int, sinks: int, max_seqlen_q: int,
                         max_seqlen_k: int, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Causal chunked-prefill attention in which the row at position t sees the keys p <= t
    with p < sinks or p > t - window; otherwise as paged_prefill. Returns out
    [total_q, Hq, 128] bf16; rows behind cu_seqlens_q[-1] are not written."""
    try:
        nb, bs, hkv, d = k_cache.shape
        total, hq, dim = q.shape
        s, mb = block_tables.shape
        ends, = cu_seqlens_q.shape
        k_ends, = cu_seqlens_k.shape
        index = q.get_device()
        fine = (q.dtype is _BF16 and k_cache.dtype is _BF16 and v_cache.dtype is _BF16
                and block_tables.dtype is _I32 and cu_seqlens_q.dtype is _I32
                and cu_seqlens_k.dtype is _I32 and q.is_contiguous() and k_cache.is_contiguous()
                and v_cache.is_contiguous() and block_tables.is_contiguous()
                and cu_seqlens_q.is_contiguous() and cu_seqlens_k.is_contiguous()
                and v_cache.shape == k_cache.shape and dim == d and ends == s + 1
                and k_ends == s + 1 and index >= 0 and k_cache.get_device() == index
                and v_cache.get_device() == index and block_tables.get_device() == index
                and cu_seqlens_q.get_device() == index and cu_seqlens_k.get_device() == index)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(dict(q=q), {}, False, k_cache, v_cache, None, None, block_tables,
                cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k)
        if dim != d or ends != s + 1 or k_ends != s + 1:
            raise ValueError("q / cache / metadata shape mismatch")
        _refuse_device(q=q, k_cache=k_cache, v_cache=v_cache, block_tables=block_tables,
                       cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k)
    lib = _lib or load()
    here = stream is None and index == _current_device()
    ctx, st = (None, _raw_stream(index)) if here else _enter(index, stream)
    try:
        out = torch.empty_like(q) if out is None else _out_like(out, q)
        if workspace is None:
            workspace = torch.empty(256, dtype=_U8, device=q.device)
        else:
            _need_workspace(workspace, q)
        status = lib.pkv_paged_prefill_window(
            out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), _clip(max_seqlen_q),
            _clip(max_seqlen_k), block_tables.data_ptr(), mb, s, total, _clip(window),
            _clip(sinks), hq, hkv, d, bs, nb, scale,
            workspace.data_ptr(), workspace.nbytes, PKV_BF16, st)
        if status != 0:
            raise PkvError(status, "pkv_paged_prefill_window")
    finally:
        if ctx is not None:
            _leave(ctx)
    return out


def selftest_bounded_wait(fail_step: int, stream=None) -> list:
    """Run the library's on-GPU failure-path check (see pkv.h); returns
    [step warp 0 left, step warp 1 left, timeout reported, steps completed]."""
    lib = load()
    res = torch.zeros(4, dtype=torch.int32, device="cuda")
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(lib.pkv_selftest_bounded_wait(int(fail_step), _ptr(res), ctypes.c_void_p(s.cuda_stream)),
           "pkv_selftest_bounded_wait")
    return res.cpu().tolist()


def get_device_errors(stream=None) -> int:
    """Synchronise the stream, then return and clear the device error bits."""
    lib = load()
    bits = ctypes.c_uint32(0)
    s = stream if stream is not None else torch.cuda.current_stream()
    st = lib.pkv_get_device_errors(ctypes.c_void_p(s.cuda_stream), ctypes.byref(bits))
    if st not in (0, -6):
        raise PkvError(st, "pkv_get_device_errors")
    return int(bits.value)
