"""Decode behind a sliding window with sinks, over the bf16 cache and over the fp8 cache with block
scales (there also over the whole context), against 64-bit attention."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32
from window_testutil import Window, assert_window_close

pytestmark = pytest.mark.gpu

SHAPES = [
    # hq, hkv, bs, ctx, window, sinks
    (8, 2, 16, [300, 1, 70, 16, 17], 64, 4),
    (32, 8, 16, [1, 0, 15, 33, 500, 130], 100, 0),
    (16, 8, 256, [700, 256, 257, 5], 300, 64),
    (8, 8, 1, [40, 3], 17, 2),                       # one token a block, one query head a KV head
    (6, 2, 6, [100, 7], 33, 5),                      # odd block and group
    (21, 3, 24, [200, 50], 1, 0),                    # the token itself
    (12, 1, 16, [90, 400], 128, 300),                # a group over one tile of heads
    (32, 2, 48, [77, 10], 40, 1),                    # a group of 16
    (40, 1, 16, [64, 350], 90, 3),                   # a group of 40: three chunks of heads
    (40, 8, 16, [120, 65], 1 << 30, 7),              # a window past everything
    (8, 2, 16, [120, 65], 20, 1 << 30),              # sinks past everything
    (2, 1, 16, [3000], 2900, 16),                    # one request over many ranges
    (4, 2, 16, [5] * 300, 3, 1),                     # many short requests
]


@pytest.mark.parametrize("hq,hkv,bs,ctx,window,sinks", SHAPES, ids=str)
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_window_decode(hq, hkv, bs, ctx, window, sinks, fp8):
    w = Window(hq, hkv, bs, ctx, window, sinks, fp8=fp8).poison_unseen()
    assert_window_close(w.call(pkv, w.device()), w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("hq,hkv,bs,ctx", [s[:4] for s in SHAPES], ids=str)
def test_whole_context_decode_over_fp8(hq, hkv, bs, ctx):
    w = Window(hq, hkv, bs, ctx, 0, 0, fp8=True, seed=5).poison_unseen()
    assert_window_close(w.call(pkv, w.device()), w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_every_window_edge(fp8):
    """Windows and sinks around the edges of a tile of 16 and of a block."""
    ctx = [33, 64, 47]
    for window, sinks in [(1, 1), (15, 1), (16, 0), (17, 3), (31, 16), (32, 17), (33, 15), (46, 1), (30, 2), (62, 2)]:
        w = Window(8, 2, 16, ctx, window, sinks, fp8=fp8, seed=window).poison_unseen()
        assert_window_close(w.call(pkv, w.device()), w)


def test_window_over_everything_is_plain_decode():
    w = Window(32, 8, 16, [100, 900, 0, 3], 1 << 20, 0)
    d = w.device()
    a = w.call(pkv, d)
    b = pkv.paged_decode(d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], w.scale)
    assert_window_close(a, w)
    assert_window_close(b, w)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_one_token_is_its_value(fp8):
    w = Window(8, 2, 16, [1, 1], 5, 0, fp8=fp8)
    out = w.call(pkv, w.device()).cpu()
    for i in range(2):
        v = w.rows_of(w.v_cache, getattr(w, "v_scales", None), w.slots(i, [0]))[0].repeat_interleave(4, 0)
        assert torch.equal(out[i], v.to(torch.bfloat16))


def test_scales_of_every_size_and_zero():
    """Block scales from 2^-120 to 2^100, and values of scale 0; keys' scales stay near 1 so that
    the softmax is no step."""
    w = Window(8, 2, 16, [200, 64], 0, 0, fp8=True, seed=9)
    rng = np.random.default_rng(1)
    e = rng.integers(-120, 101, tuple(w.v_scales.shape))
    w.v_scales = torch.from_numpy(2.0 ** e.astype(np.float64)).float()
    assert_window_close(w.call(pkv, w.device()), w)
    w.v_scales[:] = 0.0
    assert torch.equal(w.call(pkv, w.device()).cpu(), torch.zeros(2, 8, 128, dtype=torch.bfloat16))
    w.v_scales[:] = torch.from_numpy(rng.uniform(0.01, 0.3, tuple(w.v_scales.shape))).float()   # no power of two
    assert_window_close(w.call(pkv, w.device()), w)


def test_queries_of_every_size():
    for up in (2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 6):
        w = Window(8, 2, 16, [50, 17], 0, 0, fp8=True, seed=4)
        w.q = (w.q.float() * up).to(torch.bfloat16)
        # scores grow with q, and their errors with them: |score| error below 2^-11 * up moves a weight by as much
        ref, spread, _ = w.reference()
        got = w.call(pkv, w.device()).double().cpu()
        bound = 2.0 ** -8 * (spread + ref.abs()) + 2.0 ** -10 * max(up, 1.0) * spread
        assert ((got - ref).abs() <= bound).all(), up
    w.q[:] = 0.0
    assert_window_close(w.call(pkv, w.device()), w)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_growing_maxima(fp8):
    """Scores that rise along the sequence, so that the kept maximum is replaced again and again."""
    w = Window(4, 1, 16, [700], 600, 3, fp8=fp8, seed=6)
    w.q[:] = 0.25
    if fp8:
        w.k_cache.view(-1, 1, 128)[w.slots(0, range(700))] = 0x38                    # 1.0
        blocks = torch.from_numpy(w.tables[0, :44])
        w.k_scales[blocks, 0] = torch.linspace(0.0, 40.0, 44)
    else:
        w.k_cache.view(-1, 1, 128)[w.slots(0, range(700))] = torch.linspace(0, 40, 700)[:, None, None].to(torch.bfloat16)
    # scores up to 113: an fp32 sum's error of 128 * 2^-23 of it is 2^-9.2, doubled for the sum of weights
    ref, spread, most = w.reference()
    got = w.call(pkv, w.device()).double().cpu()
    assert ((got - ref).abs() <= 2.0 ** -8 * (spread + ref.abs()) + 2.0 ** -8 * spread + 2.0 ** -24 * most).all()


def test_seen_values_that_are_not_finite():
    w = Window(4, 2, 16, [90, 40, 30], 40, 2)
    k, v = w.k_cache.view(-1, 2, 128), w.v_cache.view(-1, 2, 128)
    v[w.slots(0, [60]), 0, 5] = float("inf")
    v[w.slots(0, [61]), 1, 6] = float("nan")
    v[w.slots(0, [45]), :, :] = float("nan")                 # left out: positions 2 .. 49
    k[w.slots(0, [46]), :, :] = float("inf")
    k[w.slots(1, range(40)), 0, :] = float("-inf")           # every score of a head is -inf or NaN
    w.q[1] = w.q[1].abs()
    k[w.slots(2, [3]), 1, :] = float("-inf")                 # weight 0
    w.q[2] = w.q[2].abs()
    out = w.call(pkv, w.device()).float().cpu()
    assert out[0, :2, 5].isposinf().all() and out[0, 2:, 6].isnan().all()
    out[0, :2, 5] = out[0, 2:, 6] = 0.0
    assert out[0].isfinite().all()
    assert out[1, :2].isnan().all() and out[1, 2:].isfinite().all()
    assert out[2].isfinite().all()
    assert_window_close(w.call(pkv, w.device())[2:], _only(w, 2))


def _only(w, i):
    """The same requests, request i alone."""
    one = Window(w.hq, w.hkv, w.bs, [w.ctx[i]], w.window, w.sinks, fp8=w.fp8)
    one.tables, one.k_cache, one.v_cache, one.q = w.tables[i:i + 1], w.k_cache, w.v_cache, w.q[i:i + 1]
    return one


def test_fp8_nan_codes_and_nan_queries():
    w = Window(4, 2, 16, [90, 40], 0, 0, fp8=True)
    w.v_cache.view(-1, 2, 128)[w.slots(0, [50]), 0, 9] = 0x7F
    w.k_cache.view(-1, 2, 128)[w.slots(0, [50]), 1, 9] = 0xFF
    w.q[1, 1, 3] = float("nan")
    w.q[1, 2, 3] = float("inf")
    out = w.call(pkv, w.device()).float().cpu()
    assert out[0, :2, 9].isnan().all() and out[0, 2:].isnan().all()
    assert out[0, :2, :9].isfinite().all() and out[0, :2, 10:].isfinite().all()
    assert out[1, 1].isnan().all() and out[1, 2].isnan().all()
    assert out[1, 0].isfinite().all() and out[1, 3].isfinite().all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bad_blocks_and_lengths_are_reported(fp8):
    w = Window(8, 2, 16, [100, 40], 60, 2, fp8=fp8)
    d = w.device()
    bad = w.tables.copy()
    bad[0, 5] = w.num_blocks
    out = w.call(pkv, {**d, "block_tables": i32(bad)})
    assert pkv.get_device_errors() == 2
    assert_window_close(out[1:], _only_any(w, 1))
    out = w.call(pkv, {**d, "context_lens": i32([-1, 40])})
    assert pkv.get_device_errors() == 4
    assert_window_close(out[1:], _only_any(w, 1))
    w.call(pkv, {**d, "context_lens": i32([101, 40])}, max_context_len=100)
    assert pkv.get_device_errors() == 4


def _only_any(w, i):
    one = _only(w, i)
    if w.fp8:
        one.k_scales, one.v_scales = w.k_scales, w.v_scales
    return one


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_calls_replay_with_other_lengths(fp8):
    """Two graphs that share a workspace, replayed in turn on new lengths in the same buffers, and a
    call on another stream with a workspace of its own."""
    w = Window(32, 8, 16, [600, 30, 5, 200], 90, 4, fp8=fp8)
    d = w.device()
    out = torch.empty_like(d["q"])
    ws = torch.empty(pkv.decode_window_workspace_size(4, 32, 8), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w.call(pkv, d, out=out, workspace=ws, max_context_len=600)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            w.call(pkv, d, out=o, workspace=ws, max_context_len=600)
    for ctx in ([600, 30, 5, 200], [1, 0, 600, 17], [100, 100, 100, 100]):
        short = [min(c, len(w.tables[i][w.tables[i] >= 0]) * 16) for i, c in enumerate(ctx)]
        d["context_lens"].copy_(i32(short))
        for g in graphs:
            g.replay()
        own = w.call(pkv, d, max_context_len=600, stream=side)
        torch.cuda.synchronize()
        w.ctx = short
        assert_window_close(outs[0], w)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], own)
    assert pkv.get_device_errors() == 0


def test_results_do_not_depend_on_the_workspace():
    w = Window(16, 4, 16, [2000, 100], 1500, 4, fp8=True)
    d = w.device()
    n = pkv.decode_window_workspace_size(2, 16, 4)
    outs = [w.call(pkv, d, workspace=torch.full((n,), b, dtype=torch.uint8, device="cuda")) for b in (0, 255)]
    assert torch.equal(*outs)


@pytest.mark.parametrize("hq,hkv,bs,ctx,window,sinks", [
    (12, 12, 16, [70, 33], 40, 2),                   # heads in two groups of six
    (18, 9, 8, [70, 33], 40, 2),                     # nine heads: groups of five with one to spare, boxes of 8 tokens
    (64, 16, 8, [90, 5, 0], 33, 9),
    (48, 3, 8, [200, 21], 100, 12),
    (33, 1, 8, [300, 9], 77, 8),                     # three chunks of eleven heads
    (130, 1, 16, [40, 100], 64, 3),                  # nine chunks
    (400, 1, 16, [20], 9, 3),                        # more chunks than a CTA has warps
], ids=str)
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_head_layouts(hq, hkv, bs, ctx, window, sinks, fp8):
    for win in (window, 0) if fp8 else (window,):
        w = Window(hq, hkv, bs, ctx, win, sinks, fp8=fp8, seed=hq).poison_unseen()
        assert_window_close(w.call(pkv, w.device()), w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_more_sequences_than_ranges(fp8):
    """Cut sequences are found by range where there are fewer ranges than sequences; empty ones among
    them, and at both ends."""
    rng = np.random.default_rng(3)
    ctx = [0, 0] + [int(c) for c in rng.integers(0, 90, 900)] + [700, 0]
    w = Window(16, 8, 16, ctx, 60, 5, fp8=fp8).poison_unseen()
    out = torch.full((len(ctx), 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    w.call(pkv, w.device(), out=out)
    assert_window_close(out, w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("hkv,bs", [(8, 16), (1, 8), (2, 6)])
def test_one_long_sequence(hkv, bs):
    """One request over every range: many records merged by several warps."""
    w = Window(2 * hkv, hkv, bs, [40000], 0, 0, fp8=True, seed=2)
    assert_window_close(w.call(pkv, w.device()), w)


def test_no_sequences_and_no_context():
    w = Window(8, 2, 16, [0, 0], 5, 1)
    out = torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    w.call(pkv, w.device(), out=out)
    assert torch.equal(out, torch.zeros_like(out))
    d = w.device()
    pkv.paged_decode_window(d["q"][:0], d["k_cache"], d["v_cache"], d["block_tables"][:0], d["context_lens"][:0],
                            w.scale, 5)
    assert pkv.get_device_errors() == 0


def test_windows_past_32_bits_see_everything():
    w = Window(8, 2, 16, [50, 3], 1 << 20, 0)
    d = w.device()
    a = w.call(pkv, d)
    w.window, w.sinks = (1 << 32) + 5, 1 << 33
    assert torch.equal(a, w.call(pkv, d))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bs", [16, 6])
def test_pools_past_32_bit_offsets(fp8, bs):
    """The request's blocks lie behind the first 4 GB of the caches."""
    w = Window(16, 8, bs, [300, 40], 200, 4, fp8=fp8)
    d = w.device()
    far = (1 << 32) // (bs * 8 * 128 * (1 if fp8 else 2)) + 7
    for n in ("k_cache", "v_cache"):
        pool = torch.empty((far + w.num_blocks,) + tuple(d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
        pool[far:] = d[n]
        d[n] = pool
    for n in ("k_scales", "v_scales") if fp8 else ():
        pool = torch.ones((far + w.num_blocks, 8), device="cuda")
        pool[far:] = d[n]
        d[n] = pool
    d["block_tables"] = torch.where(d["block_tables"] >= 0, d["block_tables"] + far, -1).to(torch.int32)
    assert_window_close(w.call(pkv, d), w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_two_calls_at_once(fp8):
    """Calls on two streams, each with its own workspace, over and over."""
    ws = [Window(32, 8, 16, ctx, 300, 4, fp8=fp8, seed=i) for i, ctx in enumerate(([900, 50, 3], [20, 1500]))]
    ds = [w.device() for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    outs = [[w.call(pkv, d, stream=s) for w, d, s in zip(ws, ds, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in outs:
        for o, first in zip(pair, outs[0]):
            assert torch.equal(o, first)
    for o, w in zip(outs[0], ws):
        assert_window_close(o, w)
