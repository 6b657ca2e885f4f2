"""pkv_tree_decode against the plain 64-bit attention of draft_testutil."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import Trees, assert_tree_close, i32
from paged_kv_cache_86_gb300 import _lib

pytestmark = pytest.mark.gpu

CASES = [
    # hq, hkv, block, cached tokens, drafts
    (8, 2, 16, [300], [8]),
    (8, 2, 16, [0], [1]),
    (8, 2, 16, [1], [1]),
    (1, 1, 16, [5], [3]),
    (32, 8, 16, [300, 0, 129, 17, 128, 1], [8, 3, 1, 32, 5, 2]),
    (32, 8, 256, [1000, 255, 256, 257], [33, 64, 1, 20]),
    (16, 8, 8, [127, 128, 129, 640], [16, 16, 16, 16]),
    (4, 4, 1, [130, 7, 0], [5, 9, 40]),
    (6, 2, 6, [200, 11], [12, 50]),              # 3 query heads a KV head
    (10, 2, 12, [77, 400], [30, 7]),             # 5
    (14, 2, 48, [77, 400], [30, 7]),             # 7
    (9, 1, 16, [77], [30]),                      # 9
    (12, 1, 16, [77], [30]),                     # 12
    (16, 1, 5, [77, 500], [30, 17]),             # 16
    (15, 1, 16, [300], [9]),                     # 15
    (8, 8, 16, [64, 300], [64, 65]),             # 1
    (32, 8, 16, [100, 60], [64, 33]),            # 256 rows a KV head: two full row tiles
    (8, 2, 16, [90, 4], [100, 65]),              # drafts that fill more than one row tile
    (4, 2, 16, [250, 0], [200, 130]),            # drafts that fill more than one key tile
    (2, 1, 16, [40], [300]),
    (32, 8, 16, [2000, 3], [1, 1]),              # single tokens: plain decode
]


@pytest.mark.parametrize("hq,hkv,bs,ctx,sizes", CASES)
def test_matches_the_plain_attention(hq, hkv, bs, ctx, sizes):
    t = Trees(hq, hkv, bs, ctx, sizes, seed=hq * 100 + bs)
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert_tree_close(out, t)


def test_many_sequences_with_and_without_drafts():
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 90, 700).tolist()
    sizes = rng.integers(0, 6, 700).tolist()
    t = Trees(4, 2, 16, ctx, sizes, seed=9)
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert_tree_close(out, t)


def test_a_context_cut_over_the_whole_gpu():
    t = Trees(8, 2, 16, [9000, 40, 5000], [12, 3, 40], seed=11)
    out = t.call(pkv, t.device())
    assert_tree_close(out, t)


def test_any_mask_and_rows_that_see_nothing():
    rng = np.random.default_rng(5)
    masks = [rng.random((9, 9)) < 0.3, np.zeros((4, 4), bool), rng.random((70, 70)) < 0.1,
             np.zeros((3, 3), bool)]
    masks[2][10] = False
    t = Trees(8, 2, 16, [0, 0, 0, 33], [9, 4, 70, 3], seed=6, masks=masks)
    d = t.device()
    # bits beyond the tree are nobody's: they must not matter
    d["tree_mask"][:9] |= -1 << 9
    out = t.call(pkv, d)
    assert pkv.get_device_errors() == 0
    assert_tree_close(out, t)
    assert torch.count_nonzero(out[9:13]) == 0
    assert torch.count_nonzero(out[13 + 10]) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bs", [16, 5])
def test_what_is_not_seen_has_no_part(bad, bs):
    # cache rows of nobody, rows behind the last drafts, drafts that some or all rows do not see
    masks = [np.eye(6, dtype=bool), np.eye(20, dtype=bool)]
    masks[0][3, 3] = False                       # nobody sees draft 3 of sequence 0
    t = Trees(8, 2, bs, [37, 131], [6, 20], seed=7, masks=masks, extra_rows=5).poison_unseen(bad)
    for x in (t.key, t.value, t.q):
        x[26:] = bad
    t.key[3], t.value[3] = bad, bad
    out = t.call(pkv, t.device())
    assert_tree_close(out, t)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_seen_value_that_is_not_finite_reaches_only_the_rows_that_see_it(bad):
    masks = [np.tril(np.ones((6, 6), bool))]
    t = Trees(8, 2, 16, [40], [6], seed=8, masks=masks)
    t.value[4, 1, 17] = bad
    out = t.call(pkv, t.device()).float().cpu()
    want = torch.zeros_like(out, dtype=torch.bool)
    want[4:6, 4:8, 17] = True                    # rows 4, 5; the heads of KV head 1; dim 17
    assert torch.equal(~torch.isfinite(out), want)


@pytest.mark.parametrize("ctx,drafts,at", [
    (9000, 6, 4),        # a context cut over the whole GPU: the draft is in the last piece
    (300, 140, 130),     # drafts over two key tiles and two row tiles
    (5, 100, 3),
])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_a_seen_value_that_is_not_finite_in_a_cut_sequence(ctx, drafts, at, bad):
    masks = [np.tril(np.ones((drafts, drafts), bool)), np.eye(9, dtype=bool)]
    t = Trees(8, 2, 16, [ctx, 700], [drafts, 9], seed=13, masks=masks)
    t.value[at, 0, 99] = bad
    out = t.call(pkv, t.device()).cpu()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:drafts, 0:4, 99] = True               # the rows that see it, the heads of KV head 0
    got = out[hit]
    assert torch.isnan(got).all() if bad != bad else (got == bad).all()
    # everything else is what it is without that value
    t.value[at, 0, 99] = 0
    clean = t.call(pkv, t.device()).cpu()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.5])
def test_any_scale(scale):
    t = Trees(8, 2, 16, [70, 200], [5, 30], seed=12)
    t.q *= 0.25                                  # keeps scale * sum |q k| at the documented size
    out = t.call(pkv, t.device(), scale=scale)
    # scores of up to 1.5 * 0.25 / 0.0884 = 4.3 times the size the bound is written for:
    # their fp32 error moves a weight by up to 4.3 * 2^-10 of itself
    ref, spread = t.reference(scale)
    err = (out.double().cpu() - ref).abs()
    assert bool((err <= 2.0 ** -8 * (spread + ref.abs()) + 4.3 * 2.0 ** -10 * spread).all())


def test_rows_behind_the_last_sequence_stay():
    t = Trees(8, 2, 16, [33, 64], [5, 9], seed=13, extra_rows=7)
    d = t.device()
    out = torch.full_like(d["q"], 7.0)
    assert t.call(pkv, d, out=out) is out
    assert bool((out[14:] == 7.0).all())
    assert_tree_close(out, t)


def test_strided_drafts_and_larger_bounds():
    t = Trees(8, 2, 16, [33, 64], [5, 9], seed=14)
    d = t.device()
    fused = torch.full((t.rows, 12 * 128 + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 8 * 128:10 * 128] = d["key"].flatten(1)
    fused[:, 10 * 128:12 * 128] = d["value"].flatten(1)
    d["key"] = fused[:, 8 * 128:10 * 128].unflatten(1, (2, 128))
    d["value"] = fused[:, 10 * 128:12 * 128].unflatten(1, (2, 128))
    wide = torch.full((t.rows, 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :1] = d["tree_mask"]
    d["tree_mask"] = wide
    out = t.call(pkv, d, max_seqlen_q=70, max_context_len=None)
    assert_tree_close(out, t)


def test_cache_rows_beyond_32_bit_element_offsets():
    hkv, bs = 8, 256
    nb = (1 << 31) // (bs * hkv * 128) + 40      # over 2^31 elements a cache
    t = Trees(32, hkv, bs, [700, 300], [6, 20], seed=15)
    d = t.device()
    used = {int(b): nb - 1 - j for j, b in enumerate(np.unique(t.tables[t.tables >= 0]))}
    for name in ("k_cache", "v_cache"):
        big = torch.empty((nb, bs, hkv, 128), dtype=torch.bfloat16, device="cuda")
        for src, dst in used.items():
            big[dst] = d[name][src]
        d[name] = big
    d["block_tables"] = i32([[used.get(int(b), -1) for b in row] for row in t.tables])
    out = t.call(pkv, d)
    assert pkv.get_device_errors() == 0
    assert_tree_close(out, t)


def test_chain_of_drafts_equals_a_prefill_chunk():
    # a chain's mask is the causal one: the same rows through the cache and paged_prefill
    t = Trees(32, 8, 16, [100, 37], [20, 7], seed=16,
              masks=[np.tril(np.ones((n, n), bool)) for n in (20, 7)])
    d = t.device()
    out = t.call(pkv, d)
    slots, tables, nb = [], [], t.num_blocks
    kc = torch.zeros((nb + 8, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[:nb], vc[:nb] = d["k_cache"], d["v_cache"]
    fresh = nb
    for i, (c, n) in enumerate(zip(t.ctx, t.sizes)):
        row = [int(b) for b in t.tables[i] if b >= 0]
        while len(row) * 16 < c + n:
            row.append(fresh)
            fresh += 1
        tables.append(row + [-1] * (16 - len(row)))
        slots += [row[p // 16] * 16 + p % 16 for p in range(c, c + n)]
    pkv.store_kvcache(d["key"], d["value"], kc, vc, i32(slots))
    ref = pkv.paged_prefill(d["q"], kc, vc, d["cu_seqlens_q"], i32([0, 120, 164]), i32(tables),
                            t.scale, 20, 120)
    assert_tree_close(ref, t)
    assert_tree_close(out, t)


def test_bad_blocks_and_lengths_are_reported_and_others_kept():
    t = Trees(8, 2, 16, [100, 50, 80, 33], [4, 6, 5, 3], seed=17)
    d = t.device()
    d["block_tables"][1, 1] = t.num_blocks + 5
    d["block_tables"][2, 0] = -7
    out = t.call(pkv, d)
    assert pkv.get_device_errors() == _lib.DEVERR_BLOCK_ID
    keep = list(range(0, 4)) + list(range(15, 18))
    ref, spread = t.reference()
    err = (out.double().cpu() - ref).abs()[keep]
    assert bool((err <= 2.0 ** -8 * (spread + ref.abs())[keep] + 2.0 ** -10 * spread[keep]).all())
    d = t.device()
    d["context_lens"][1] = 101                   # over max_context_len
    d["context_lens"][2] = -1
    out = t.call(pkv, d)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH
    err = (out.double().cpu() - ref).abs()[keep]
    assert bool((err <= 2.0 ** -8 * (spread + ref.abs())[keep] + 2.0 ** -10 * spread[keep]).all())
    d = t.device()
    t.call(pkv, d, max_seqlen_q=5)               # a tree over the bound
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH


def test_same_bits_again_and_on_another_stream():
    t = Trees(32, 8, 16, [900, 40, 5000], [12, 3, 40], seed=18)
    d = t.device()
    a = t.call(pkv, d)
    b = t.call(pkv, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = t.call(pkv, d, stream=side)              # buffers come from the side stream's pool
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)
    # two calls at once, each with a workspace of its own
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append(t.call(pkv, d))
    torch.cuda.synchronize()
    assert torch.equal(a, outs[0]) and torch.equal(a, outs[1])


def test_calls_and_replays_at_the_same_time_on_two_streams():
    batches = [Trees(8, 2, 16, [3000, 40], [12, 3], seed=21), Trees(8, 2, 12, [70, 2500], [5, 40], seed=22)]
    inputs = [t.device() for t in batches]
    alone = [t.call(pkv, d) for t, d in zip(batches, inputs)]
    streams = [torch.cuda.Stream() for _ in batches]
    outs = [torch.empty_like(a) for a in alone]
    torch.cuda.synchronize()
    for _ in range(20):
        for t, d, st, o in zip(batches, inputs, streams, outs):
            t.call(pkv, d, out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))
    graphs = []
    for t, d, o in zip(batches, inputs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.call(pkv, d, out=o)
        graphs.append(g)
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert pkv.get_device_errors() == 0
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))


def test_captured_once_and_replayed_with_other_lengths():
    big = Trees(16, 4, 16, [600, 0, 333, 90], [10, 4, 16, 2], seed=19)
    d = big.device()
    rows, width = 40, big.width
    buf = {"q": torch.zeros((rows, 16, 128), dtype=torch.bfloat16, device="cuda"),
           "key": torch.zeros((rows, 4, 128), dtype=torch.bfloat16, device="cuda"),
           "value": torch.zeros((rows, 4, 128), dtype=torch.bfloat16, device="cuda"),
           "tree_mask": torch.zeros((rows, 1), dtype=torch.int32, device="cuda"),
           "block_tables": torch.full((4, width), -1, dtype=torch.int32, device="cuda"),
           "context_lens": i32([0] * 4), "cu_seqlens_q": i32([0] * 5),
           "k_cache": torch.zeros((200, 16, 4, 128), dtype=torch.bfloat16, device="cuda"),
           "v_cache": torch.zeros((200, 16, 4, 128), dtype=torch.bfloat16, device="cuda")}
    ws = torch.empty(pkv.tree_decode_workspace_size(32, 16, 4), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(buf["q"])

    def call():
        big.call(pkv, buf, max_seqlen_q=32, max_context_len=600, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (big, Trees(16, 4, 16, [3, 512, 600], [32, 1, 7], seed=20),
              Trees(16, 4, 16, [17], [30], seed=21)):
        d, s = t.device(), len(t.ctx)
        for n in ("q", "key", "value", "tree_mask"):
            buf[n][:t.rows] = d[n]
        for n in ("k_cache", "v_cache"):
            buf[n][:t.num_blocks] = d[n]
        w = min(width, t.width)
        buf["block_tables"].fill_(-1)
        buf["block_tables"][:s, :w] = d["block_tables"][:, :w]
        buf["context_lens"].zero_()
        buf["context_lens"][:s] = d["context_lens"]
        buf["cu_seqlens_q"].fill_(int(t.cu[-1]))  # padded with sequences of no rows
        buf["cu_seqlens_q"][:s + 1] = d["cu_seqlens_q"]
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.get_device_errors() == 0
        assert_tree_close(out, t)


def test_no_rows_is_a_noop():
    t = Trees(8, 2, 16, [33, 64], [0, 0], seed=22)
    out = t.call(pkv, t.device(), max_seqlen_q=4)
    assert tuple(out.shape) == (0, 8, 128)
