"""Chunked prefill behind a sliding window with sinks, against 64-bit attention of every row."""
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32
from window_testutil import Window, assert_window_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,bs,ctx,q_lens,window,sinks", [
    (8, 2, 16, [300, 70], [130, 70], 64, 4),
    (4, 2, 16, [1, 16, 17, 500], [1, 16, 1, 3], 33, 0),
    (8, 2, 256, [700, 300], [200, 129], 300, 64),
    (4, 4, 16, [400], [300], 100, 17),               # one query head a KV head: pairs of query tiles
    (6, 2, 24, [333, 100], [257, 5], 50, 5),         # an odd group and boxes of 8 rows
    (4, 2, 1, [150], [140], 40, 3),                  # gathered rows
    (4, 2, 6, [280, 20], [150, 20], 129, 1),
    (4, 2, 48, [500], [256], 1, 0),                  # the token itself
    (4, 2, 16, [500], [256], 1, 1),
    (4, 2, 16, [300, 140], [128, 140], 1 << 30, 3),  # a window past everything: plain causal
    (4, 2, 16, [300], [150], 20, 1 << 30),           # sinks past everything
    (4, 2, 16, [1000], [140], 128, 300),             # sinks over several tiles
    (4, 2, 16, [600], [129], 400, 130),              # sinks that meet the window for some rows
    (4, 2, 16, [0, 40, 0], [0, 40, 0], 8, 2),        # empty requests
    (24, 8, 8, [200], [130], 70, 9),
], ids=str)
def test_window_prefill(hq, hkv, bs, ctx, q_lens, window, sinks):
    w = Window(hq, hkv, bs, ctx, window, sinks, q_lens=q_lens, extra_rows=3).poison_unseen()
    out = torch.full((w.rows, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    w.call(pkv, w.device(), out=out)
    assert_window_close(out, w)
    assert (out[int(w.cu[-1]):] == 7.0).all()                # rows behind the last sequence
    assert pkv.get_device_errors() == 0


def test_every_window_edge():
    """Windows and sinks around tile, box and block edges."""
    for window, sinks in [(31, 1), (32, 31), (33, 32), (127, 33), (128, 0), (129, 16), (160, 129), (255, 127),
                          (256, 1), (257, 64)]:
        w = Window(2, 1, 16, [390, 128], window, sinks, q_lens=[150, 127], seed=window).poison_unseen()
        assert_window_close(w.call(pkv, w.device()), w)


def test_window_over_everything_is_plain_prefill():
    w = Window(8, 2, 16, [400, 33], 1 << 20, 0, q_lens=[200, 33])
    d = w.device()
    out = pkv.paged_prefill(d["q"], d["k_cache"], d["v_cache"], d["cu_seqlens_q"], d["cu_seqlens_k"],
                            d["block_tables"], w.scale, 200, 400)
    assert torch.equal(out, w.call(pkv, d))


@pytest.mark.parametrize("bs", [16, 6, 256])
@pytest.mark.parametrize("group", [2, 1])
def test_what_is_not_finite_reaches_only_the_rows_that_see_it(bs, group):
    """Keys and values that some rows of a tile see and others do not, behind the window, in front of
    it and among the later rows of the chunk."""
    w = Window(2 * group, 2, bs, [420], 60, 3, q_lens=[200])
    k, v = w.k_cache.view(-1, 2, 128), w.v_cache.view(-1, 2, 128)
    v[w.slots(0, [1]), 0, 7] = float("inf")                  # a sink: every row
    v[w.slots(0, [230]), 1, 5] = float("nan")                # rows 220 .. 289: seen by 230 .. 289
    v[w.slots(0, [300]), :, 6] = float("-inf")
    k[w.slots(0, [260]), 1, :] = float("nan")                # whole rows 260 .. 319 of head 1
    v[w.slots(0, [419]), :, :] = float("nan")                # the last row alone
    out = w.call(pkv, w.device()).float().cpu()
    ref, spread, _ = w.reference()
    g, r = out.double(), ref
    assert torch.equal(g.isnan(), r.isnan())
    assert torch.equal(g.isinf(), r.isinf()) and (g[r.isinf()] == r[r.isinf()]).all()
    fine = r.isfinite() & spread.isfinite()
    bound = 2.0 ** -8 * (spread + r.abs()) + 2.0 ** -10 * spread
    assert ((g - r).abs()[fine] <= bound[fine]).all()
    assert pkv.get_device_errors() == 0


def test_scores_of_minus_infinity_alone_give_nan():
    w = Window(2, 1, 16, [100], 10, 0, q_lens=[60])
    w.q[:] = w.q.abs()
    k = w.k_cache.view(-1, 1, 128)
    k[w.slots(0, range(60, 80)), 0] = float("-inf")
    out = w.call(pkv, w.device()).float().cpu()
    seen_only_bad = torch.tensor([t - 9 >= 60 and t < 80 for t in range(40, 100)])
    assert out[seen_only_bad].isnan().all() and out[~seen_only_bad].isfinite().all()


def test_bad_blocks_and_lengths_are_reported():
    w = Window(4, 2, 16, [100, 40], 30, 2, q_lens=[50, 40])
    d = w.device()
    bad = w.tables.copy()
    bad[0, 5] = w.num_blocks
    w.call(pkv, {**d, "block_tables": i32(bad)})
    assert pkv.get_device_errors() == 2
    w.call(pkv, {**d, "cu_seqlens_k": i32([0, 30, 70])})     # fewer keys than query rows
    assert pkv.get_device_errors() == 4


def test_captured_call_replays_with_other_lengths():
    w = Window(8, 2, 16, [300, 100], 64, 4, q_lens=[100, 100])
    d = w.device()
    out = torch.empty_like(d["q"])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w.call(pkv, d, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.call(pkv, d, out=out, workspace=ws)
    for q_lens, ctx in (([100, 100], [300, 100]), ([3, 70], [250, 90])):
        w.q_lens, w.ctx = q_lens, ctx
        w.cu = torch.tensor([0, q_lens[0], sum(q_lens)]).numpy()
        d["cu_seqlens_q"].copy_(i32(w.cu))
        d["cu_seqlens_k"].copy_(i32([0, ctx[0], sum(ctx)]))
        g.replay()
        torch.cuda.synchronize()
        assert_window_close(out, w)
    assert pkv.get_device_errors() == 0


def test_pools_past_32_bit_offsets():
    w = Window(4, 2, 16, [200, 40], 50, 4, q_lens=[140, 40])
    d = w.device()
    far = (1 << 32) // (16 * 2 * 128 * 2) + 7
    for n in ("k_cache", "v_cache"):
        pool = torch.empty((far + w.num_blocks,) + tuple(d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
        pool[far:] = d[n]
        d[n] = pool
    d["block_tables"] = torch.where(d["block_tables"] >= 0, d["block_tables"] + far, -1).to(torch.int32)
    assert_window_close(w.call(pkv, d), w)


def test_output_at_any_16_byte_boundary():
    w = Window(4, 2, 16, [150], 40, 2, q_lens=[150])
    room = torch.zeros(w.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    d = w.device()
    for at in (0, 8):
        out = room[at:at + w.q.numel()].view(w.q.shape)
        w.call(pkv, d, out=out)
        assert_window_close(out, w)


def test_more_items_than_sms_and_calls_at_once():
    """Items claimed from the ticket, on two streams with workspaces of their own."""
    ws = [Window(16, 2, 16, [260] * 12, 70, 3, q_lens=[256] * 12, seed=i) for i in range(2)]
    ds = [w.device() for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    outs = [[w.call(pkv, d, stream=s) for w, d, s in zip(ws, ds, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    for pair in outs:
        for o, first in zip(pair, outs[0]):
            assert torch.equal(o, first)
    for o, w, d in zip(outs[0], ws, ds):
        one = Window(16, 2, 16, [260], 70, 3, q_lens=[256])
        one.tables, one.k_cache, one.v_cache, one.q = w.tables[5:6], w.k_cache, w.v_cache, w.q[5 * 256:6 * 256]
        assert_window_close(o[5 * 256:6 * 256], one)
