"""pkv_qk_norm_rope and pkv_qk_norm_rope_store against the formula in 64 bits."""
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import HALF_BF16, i32, normal
from paged_kv_cache_86_gb300 import _lib

pytestmark = pytest.mark.gpu


def angles(max_position, rotary):
    p = torch.arange(max_position, dtype=torch.float64)[:, None]
    a = p * 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    return torch.cat([a.cos(), a.sin()], 1).float()


def reference(x, weight, eps, positions, table, interleaved):
    """(result, size) in 64 bits; size: the larger of each pair, which bounds what an
    fp32 turn can lose to cancellation."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    r = table.shape[1]
    cos, sin = table[positions].double()[:, None].chunk(2, -1)
    head = x[..., :r]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
    else:
        a, b = head.chunk(2, -1)
    u, w = a * cos - b * sin, b * cos + a * sin
    big = torch.maximum(a.abs(), b.abs())
    if interleaved:
        head, size = torch.stack([u, w], -1).flatten(-2), torch.stack([big, big], -1).flatten(-2)
    else:
        head, size = torch.cat([u, w], -1), torch.cat([big, big], -1)
    return torch.cat([head, x[..., r:]], -1), torch.cat([size, x[..., r:].abs()], -1)


def assert_rows(got, want):
    """One rounding to bf16 (half a step of the result) of an fp32 value that is off by at
    most 32 * 2^-24 of the pair's larger value: 20 roundings in the sum of squares (16
    terms in a lane, 4 exchanges) count half, rsqrtf has 2 ulp, and four products and a
    sum follow."""
    ref, size = want
    err = (got.double().cpu() - ref).abs()
    bound = HALF_BF16 * ref.abs() + 32 * 2.0 ** -24 * (1 + HALF_BF16) * size * 1.42 + 1e-38
    assert bool((err <= bound).all()), float((err - bound).max())


CASES = [
    # tokens, hq, hkv, head_dim, rotary, interleaved, q norm, k norm
    (1, 8, 2, 128, 128, False, True, True),
    (7, 32, 8, 128, 128, False, True, True),
    (33, 16, 8, 128, 64, True, False, False),
    (5, 3, 1, 128, 16, False, True, False),
    (5, 3, 1, 128, 112, True, False, True),
    (9, 5, 5, 64, 64, False, True, True),
    (9, 7, 1, 64, 32, True, True, True),
    (4, 6, 2, 256, 256, False, True, True),
    (4, 6, 3, 256, 80, True, True, True),
    (1200, 12, 4, 128, 128, False, True, True),
]


def inputs(tokens, hq, hkv, d, rotary, qn, kn, seed=1, fused=True):
    qkv = normal((tokens, (hq + 2 * hkv) * d), seed)
    x = {"q": qkv[:, :hq * d].unflatten(1, (hq, d)),
         "k": qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
         "v": qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))}
    dev = qkv.cuda()
    g = {"q": dev[:, :hq * d].unflatten(1, (hq, d)),
         "k": dev[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
         "v": dev[:, (hq + hkv) * d:].unflatten(1, (hkv, d))}
    x["qw"] = 1 + normal((d,), seed + 1, 0.2) if qn else None
    x["kw"] = 1 + normal((d,), seed + 2, 0.2) if kn else None
    x["pos"] = torch.randint(0, 5000, (tokens,), generator=torch.Generator().manual_seed(seed))
    x["table"] = angles(5000, rotary)
    g.update({n: None if x[n] is None else x[n].cuda() for n in ("qw", "kw", "table")})
    g["pos"] = i32(x["pos"])
    return x, g


@pytest.mark.parametrize("tokens,hq,hkv,d,rotary,inter,qn,kn", CASES)
def test_matches_the_formula(tokens, hq, hkv, d, rotary, inter, qn, kn):
    x, g = inputs(tokens, hq, hkv, d, rotary, qn, kn)
    q, k = pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"], 1e-5, inter)
    assert pkv.get_device_errors() == 0
    assert_rows(q, reference(x["q"], x["qw"], 1e-5, x["pos"], x["table"], inter))
    assert_rows(k, reference(x["k"], x["kw"], 1e-5, x["pos"], x["table"], inter))


@pytest.mark.parametrize("tokens,hq,hkv,d,rotary,inter,qn,kn", CASES)
def test_store_writes_the_slots_and_nothing_else(tokens, hq, hkv, d, rotary, inter, qn, kn):
    x, g = inputs(tokens, hq, hkv, d, rotary, qn, kn, seed=5)
    bs = 6
    nb = tokens // bs + 3
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(3))[:tokens]
    slots[::4] = -1
    kc = torch.full((nb, bs, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 4.0)
    q = pkv.qk_norm_rope_store(g["q"], g["k"], g["v"], kc, vc, i32(slots), g["pos"], g["table"],
                               g["qw"], g["kw"], 1e-6, inter)
    assert pkv.get_device_errors() == 0
    assert_rows(q, reference(x["q"], x["qw"], 1e-6, x["pos"], x["table"], inter))
    k, v = kc.flatten(0, 1).cpu(), vc.flatten(0, 1).cpu()
    kept = slots >= 0
    want, size = reference(x["k"], x["kw"], 1e-6, x["pos"], x["table"], inter)
    assert_rows(k[slots[kept]], (want[kept], size[kept]))
    assert torch.equal(v[slots[kept]], x["v"][kept])
    rest = torch.ones(nb * bs, dtype=torch.bool)
    rest[slots[kept]] = False
    assert bool((k[rest] == 3.0).all()) and bool((v[rest] == 4.0).all())


@pytest.mark.parametrize("tokens,hq,hkv,d,rotary,inter,qn,kn", [
    # more tokens than warps fit the GPU: one warp a token in fewer, fuller waves, or two
    (5003, 3, 1, 64, 64, False, True, True),
    (5003, 2, 1, 256, 128, True, False, True),
    (10001, 4, 2, 128, 64, True, True, False),
    (10001, 4, 2, 128, 128, False, False, False),
    (6007, 14, 2, 256, 256, False, True, True),
    (6007, 28, 4, 128, 128, True, True, True),
])
def test_more_tokens_than_resident_warps(tokens, hq, hkv, d, rotary, inter, qn, kn):
    x, g = inputs(tokens, hq, hkv, d, rotary, qn, kn, seed=12)
    kc = torch.full((tokens // 16 + 2, 16, hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 4.0)
    slots = torch.randperm(tokens + 1, generator=torch.Generator().manual_seed(4))[:tokens]
    q = pkv.qk_norm_rope_store(g["q"], g["k"], g["v"], kc, vc, i32(slots), g["pos"], g["table"],
                               g["qw"], g["kw"], 1e-6, inter)
    q2, k2 = pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"], 1e-6, inter)
    assert pkv.get_device_errors() == 0
    assert_rows(q, reference(x["q"], x["qw"], 1e-6, x["pos"], x["table"], inter))
    assert_rows(k2, reference(x["k"], x["kw"], 1e-6, x["pos"], x["table"], inter))
    at = slots.cuda()
    assert torch.equal(q, q2) and torch.equal(kc.flatten(0, 1)[at], k2)
    assert torch.equal(vc.flatten(0, 1)[at], g["v"])
    rest = torch.ones(kc.shape[0] * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((kc.flatten(0, 1)[rest] == 3.0).all()) and bool((vc.flatten(0, 1)[rest] == 4.0).all())


def test_in_place_and_strided_outputs():
    x, g = inputs(40, 8, 2, 128, 128, True, True, seed=7)
    q, k = pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"])
    v = g["v"].clone()
    q2, k2 = pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"],
                              q_out=g["q"], k_out=g["k"])
    assert q2.data_ptr() == g["q"].data_ptr()
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, g["v"])


def test_value_and_unturned_bits_pass_as_they_are():
    x, g = inputs(6, 4, 2, 128, 32, False, False, seed=8)
    g["q"][:, :, 40] = float("nan")
    g["v"][:, 0, 3] = float("inf")
    kc = torch.zeros((1, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q = pkv.qk_norm_rope_store(g["q"], g["k"], g["v"], kc, vc, i32(range(6)), g["pos"], g["table"])
    assert torch.equal(q[:, :, 32:].contiguous().view(torch.int16),
                       g["q"][:, :, 32:].contiguous().view(torch.int16))
    assert torch.equal(vc[0, :6], g["v"]) and torch.isfinite(q[:, :, :32]).all()


def test_bad_positions_and_slots_are_skipped_and_reported():
    x, g = inputs(8, 4, 2, 128, 128, True, True, seed=9)
    kc = torch.full((2, 16, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 3.0)
    g["pos"][2], g["pos"][5] = -1, 5000
    slots = i32([0, 1, 2, 32, 4, 5, 6, -9])
    out = torch.full((8, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_store(g["q"], g["k"], g["v"], kc, vc, slots, g["pos"], g["table"], g["qw"],
                           g["kw"], q_out=out)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH | _lib.DEVERR_SLOT
    assert bool((out[[2, 5]] == 9.0).all())
    x["pos"][2], x["pos"][5] = 0, 0
    want, size = reference(x["q"], x["qw"], 1e-6, x["pos"], x["table"], False)
    keep = [0, 1, 3, 4, 6, 7]
    assert_rows(out[keep], (want[keep], size[keep]))
    v = vc.flatten(0, 1)
    assert torch.equal(v[[0, 1, 4, 6]], g["v"][[0, 1, 4, 6]])
    assert bool((v[[2, 3, 5, 7]] == 3.0).all()) and bool((v[8:] == 3.0).all())


def test_no_tokens_and_a_captured_call():
    x, g = inputs(5, 8, 2, 128, 128, True, True, seed=10)
    q, k = pkv.qk_norm_rope(g["q"][:0], g["k"][:0], g["pos"][:0], g["table"])
    assert q.shape == (0, 8, 128) and k.shape == (0, 2, 128)
    q, k = (torch.empty_like(g[n].contiguous()) for n in ("q", "k"))
    pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"], q_out=q, k_out=k)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.qk_norm_rope(g["q"], g["k"], g["pos"], g["table"], g["qw"], g["kw"], q_out=q, k_out=k)
    y, h = inputs(5, 8, 2, 128, 128, True, True, seed=11)
    for n in ("q", "k", "qw", "kw", "pos"):
        g[n].copy_(h[n])
    graph.replay()
    assert_rows(q, reference(y["q"], y["qw"], 1e-6, y["pos"], y["table"], False))
    assert_rows(k, reference(y["k"], y["kw"], 1e-6, y["pos"], y["table"], False))


def test_cache_rows_beyond_32_bit_element_offsets():
    x, g = inputs(3, 8, 8, 128, 128, True, True, seed=12)
    nb = (1 << 31) // (256 * 8 * 128) + 1
    kc = torch.empty((nb, 256, 8, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    last = nb * 256 - 1
    pkv.qk_norm_rope_store(g["q"], g["k"], g["v"], kc, vc, i32([last, 0, last - 1]), g["pos"],
                           g["table"], g["qw"], g["kw"])
    want, size = reference(x["k"], x["kw"], 1e-6, x["pos"], x["table"], False)
    assert_rows(torch.stack([kc[-1, -1], kc[0, 0], kc[-1, -2]]), (want, size))
    assert torch.equal(vc[-1, -1], g["v"][0]) and torch.equal(vc[0, 0], g["v"][1])
