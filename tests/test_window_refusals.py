"""Refusals of the calls over an fp8 cache with block scales and behind a sliding window: the
library's own checks of arguments and the binding's checks of layouts, types and shapes. All of
them answer without a GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from paged_kv_cache_86_gb300 import _lib
from paged_kv_cache_86_gb300.build import build

BF16, I32, U8, F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
P, NULL = ctypes.c_void_p(4096), ctypes.c_void_p(0)
ARG, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


STORE = ["key", "value", "ks", "vs", "k_cache", "v_cache", "k_scales", "v_scales", "tables", "mb", "cu", "lens",
         "s", "total", "hkv", "d", "bs", "nb", "stream"]
LOAD = ["key", "value", "ks", "vs", "k_cache", "v_cache", "k_scales", "v_scales", "tables", "mb", "lens", "starts",
        "s", "rows", "hkv", "d", "bs", "nb", "stream"]
DEC8 = ["out", "q", "k_cache", "v_cache", "k_scales", "v_scales", "tables", "mb", "lens", "s", "most", "window",
        "sinks", "hq", "hkv", "d", "bs", "nb", "scale", "ws", "bytes", "stream"]
DEC = [n for n in DEC8 if "scales" not in n][:-1] + ["dtype", "stream"]
PRE = ["out", "q", "k_cache", "v_cache", "cu", "cuk", "mq", "mk", "tables", "mb", "s", "total", "window", "sinks",
       "hq", "hkv", "d", "bs", "nb", "scale", "ws", "bytes", "dtype", "stream"]
GOOD = dict(out=ctypes.c_void_p(1 << 20), q=P, key=P, value=ctypes.c_void_p(8192), ks=1024, vs=1024, k_cache=P,
            v_cache=ctypes.c_void_p(1 << 21), k_scales=P, v_scales=ctypes.c_void_p(1 << 22), tables=P, mb=4, cu=P,
            cuk=P, lens=P, starts=P, s=2, total=4, rows=8, hkv=8, hq=32, d=128, bs=16, nb=9, most=64, mq=3, mk=64,
            window=8, sinks=2, scale=0.1, ws=P, bytes=1 << 40, dtype=0, stream=NULL)
CALLS = {"store_kvcache_fp8_block": STORE, "load_kvcache_fp8_block": LOAD, "paged_decode_fp8_block": DEC8,
         "paged_decode_window": DEC, "paged_prefill_window": PRE}


def call(lib, name, **over):
    a = {**GOOD, **over}
    return getattr(lib, "pkv_" + name)(*[a[n] for n in CALLS[name]])


def cases():
    pool = [dict(hkv=0), dict(bs=0), dict(nb=0), dict(mb=-1), dict(s=-1)]
    for name in ("store_kvcache_fp8_block", "load_kvcache_fp8_block"):
        rows = "total" if name.startswith("store") else "rows"
        for over in pool + [{rows: -1}, dict(key=NULL), dict(value=NULL), dict(k_cache=NULL), dict(v_cache=NULL),
                            dict(k_scales=NULL), dict(v_scales=NULL), dict(tables=NULL), dict(lens=NULL),
                            dict(key=ctypes.c_void_p(4104)), dict(v_cache=ctypes.c_void_p(4104)), dict(ks=1016),
                            dict(vs=1028)]:
            yield name, over, ARG
        yield name, dict(d=64), SHAPE
        yield name, dict(hkv=32768, ks=1 << 23, vs=1 << 23), SHAPE
        yield name, {rows: 0, "key": NULL}, 0
        yield name, dict(s=0, key=NULL), 0
    yield "store_kvcache_fp8_block", dict(cu=NULL), ARG
    yield "store_kvcache_fp8_block", dict(v_cache=P), ARG
    yield "store_kvcache_fp8_block", dict(v_scales=P), ARG
    yield "load_kvcache_fp8_block", dict(starts=NULL), ARG
    yield "load_kvcache_fp8_block", dict(value=P), ARG
    for name in ("paged_decode_fp8_block", "paged_decode_window", "paged_prefill_window"):
        far = dict(mk=65) if name == "paged_prefill_window" else dict(most=65)
        for over in pool + [dict(hq=0), dict(sinks=-1), dict(window=-1), dict(scale=0.0), dict(scale=-0.1),
                            dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), far, dict(out=NULL),
                            dict(q=NULL), dict(k_cache=NULL), dict(v_cache=NULL), dict(tables=NULL),
                            dict(q=ctypes.c_void_p(4104)), dict(out=ctypes.c_void_p((1 << 20) + 8)), dict(out=P),
                            dict(out=ctypes.c_void_p(4096 + 256)), dict(nb=1 << 28)]:
            yield name, over, ARG
        for over in (dict(d=64), dict(hq=31)):
            yield name, over, SHAPE
        yield name, dict(s=0, q=NULL), 0
        yield name, dict(ws=NULL), WORKSPACE
        yield name, dict(ws=ctypes.c_void_p(4096 + 64)), WORKSPACE
        yield name, dict(bytes=255), WORKSPACE
    for name in ("paged_decode_window", "paged_prefill_window"):
        yield name, dict(dtype=1), DTYPE
        yield name, dict(window=0), ARG
    yield "paged_decode_fp8_block", dict(k_scales=NULL), ARG
    yield "paged_decode_fp8_block", dict(v_scales=NULL), ARG
    yield "paged_decode_fp8_block", dict(s=1 << 30, most=64), ARG          # tiles past 32 bits
    yield "paged_decode_window", dict(s=1 << 29), ARG
    yield "paged_prefill_window", dict(cu=NULL), ARG
    yield "paged_prefill_window", dict(cuk=NULL), ARG
    yield "paged_prefill_window", dict(total=-1), ARG
    yield "paged_prefill_window", dict(mq=-1), ARG
    yield "paged_prefill_window", dict(s=65536), ARG
    yield "paged_prefill_window", dict(mq=65535 * 128 + 1), ARG
    yield "paged_prefill_window", dict(mk=0x7fffffff, mb=1 << 27), ARG     # positions past 32 bits
    yield "paged_prefill_window", dict(total=0, q=NULL), 0
    yield "paged_prefill_window", dict(mq=0, q=NULL), 0


@pytest.mark.parametrize("name,over,want", list(cases()))
def test_library_refuses_without_a_gpu(lib, name, over, want):
    assert call(lib, name, **over) == want


def test_workspace_size_of_bad_shapes_is_zero(lib):
    for bad in ((-1, 8, 2, 128), (1, 0, 1, 128), (1, 8, 0, 128), (1, 8, 3, 128), (1, 8, 2, 64)):
        assert lib.pkv_decode_window_workspace_size(*bad) == 0


def args(name):
    """CPU tensors of one call: two sequences of 20 tokens, 8 query / 2 KV heads, block 16."""
    pool = dict(k_cache=torch.zeros(6, 16, 2, 128, dtype=U8), v_cache=torch.zeros(6, 16, 2, 128, dtype=U8),
                k_scales=torch.ones(6, 2), v_scales=torch.ones(6, 2))
    wide = dict(k_cache=torch.zeros(6, 16, 2, 128, dtype=BF16), v_cache=torch.zeros(6, 16, 2, 128, dtype=BF16))
    meta = dict(block_tables=torch.tensor([[0, 1], [2, 3]], dtype=I32), context_lens=torch.tensor([20, 20], dtype=I32))
    q = dict(q=torch.zeros(2, 8, 128, dtype=BF16))
    if name == "store_kvcache_fp8_block":
        return dict(key=torch.zeros(4, 2, 128, dtype=BF16), value=torch.zeros(4, 2, 128, dtype=BF16), **pool, **meta,
                    cu_seqlens_q=torch.tensor([0, 2, 4], dtype=I32))
    if name == "load_kvcache_fp8_block":
        return dict(**pool, **meta, row_starts=torch.tensor([0, 20], dtype=I32), num_rows=40)
    if name == "paged_decode_fp8_block":
        return dict(**q, **pool, **meta, scale=0.1)
    if name == "paged_decode_window":
        return dict(**q, **wide, **meta, scale=0.1, window=8)
    return dict(**q, **wide, block_tables=meta["block_tables"], cu_seqlens_q=torch.tensor([0, 1, 2], dtype=I32),
                cu_seqlens_k=torch.tensor([0, 20, 40], dtype=I32), scale=0.1, window=8, sinks=0, max_seqlen_q=1,
                max_seqlen_k=20)


def tensors():
    return [(c, n) for c in CALLS for n, t in args(c).items() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name,what", tensors())
def test_binding_refuses_wrong_types_layouts_and_shapes(name, what):
    a = args(name)
    t = a[what]
    f = getattr(pkv, name)
    with pytest.raises(TypeError):
        f(**{**a, what: None})
    with pytest.raises(TypeError):
        f(**{**a, what: t.to(torch.float64)})
    with pytest.raises(ValueError):                        # another rank
        f(**{**a, what: t.unsqueeze(0)})
    strided = torch.stack([t, t], -1)[..., 0]              # the same values, every second element
    with pytest.raises(ValueError, match="contiguous"):
        f(**{**a, what: strided})
    if (name, what) != ("paged_prefill_window", "q"):      # (rows behind the last sequence are allowed there)
        with pytest.raises(ValueError):
            f(**{**a, what: torch.cat([t, t])})            # twice as many rows


@pytest.mark.parametrize("name", list(CALLS))
def test_dense_cpu_tensors_are_refused_for_their_device(name):
    with pytest.raises(TypeError, match="CUDA tensor"):
        getattr(pkv, name)(**args(name))


def test_strided_token_rows_pass_the_layout_check():
    a = args("store_kvcache_fp8_block")
    fused = torch.zeros(4, 6, 128, dtype=BF16)
    a.update(key=fused[:, :2], value=fused[:, 4:])
    with pytest.raises(TypeError, match="CUDA tensor"):
        pkv.store_kvcache_fp8_block(**a)


def test_load_needs_rows_or_both_outputs():
    a = args("load_kvcache_fp8_block")
    out = torch.zeros(40, 2, 128, dtype=BF16)
    for bad in (dict(num_rows=None), dict(num_rows=-1), dict(key_out=out), dict(value_out=out),
                dict(key_out=out, value_out=out[:39]), dict(key_out=out, value_out=out, num_rows=41)):
        with pytest.raises(ValueError):
            pkv.load_kvcache_fp8_block(**{**a, **bad})
