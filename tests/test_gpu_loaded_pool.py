"""A bf16 pool that load_kvcache_fp8_block filled, attended to: rows of each sequence's last block
behind its last token are not written, so whatever was there stays. The windowed prefill takes them
whatever they hold; the calls without a window want their values (V) finite, and nothing of their keys."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32, normal
from window_testutil import Window, assert_window_close

pytestmark = pytest.mark.gpu


def loaded(w, *junk):
    """w's cache (fp8) read back into a pool of consecutive blocks whose keys and values held `junk`; w
    becomes that bf16 pool, where 0 stands for what is not finite."""
    blocks = [-(-c // w.bs) for c in w.ctx]
    first = np.concatenate([[0], np.cumsum(blocks)])
    shape = (max(int(first[-1]), 1), w.bs, w.hkv, 128)
    pool = [torch.full(shape, j, dtype=torch.bfloat16, device="cuda") for j in junk]
    d = w.device()
    pkv.load_kvcache_fp8_block(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["block_tables"],
                               d["context_lens"], i32(first[:-1] * w.bs), key_out=pool[0].view(-1, w.hkv, 128),
                               value_out=pool[1].view(-1, w.hkv, 128))
    own = np.full((len(w.ctx), max(max(blocks), 1)), -1)
    for i, n in enumerate(blocks):
        own[i, :n] = first[i] + np.arange(n)
    w.fp8, w.tables, w.num_blocks = False, own, shape[0]
    w.k_cache, w.v_cache = [p.cpu().nan_to_num(0.0, 0.0, 0.0) for p in pool]
    return pool, own


NAN, INF, LARGE = float("nan"), float("inf"), 3.3e38
CTX, NEW = [70, 1, 200, 33, 300], [70, 1, 130, 5, 300]


@pytest.mark.parametrize("bs", [16, 8, 24, 256, 6])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3)], ids=["pairs of heads", "pairs of tiles"])
@pytest.mark.parametrize("junk", [(NAN, NAN), (INF, INF), (LARGE, -INF)], ids=str)
@pytest.mark.parametrize("window", [1 << 20, 40])
def test_prefill_behind_a_window(bs, hq, hkv, junk, window):
    w = Window(hq, hkv, bs, CTX, window, 0, q_lens=NEW, fp8=True, seed=bs)
    d = w.device()
    pool, own = loaded(w, *junk)
    out = pkv.paged_prefill_window(d["q"], *pool, d["cu_seqlens_q"], d["cu_seqlens_k"], i32(own), w.scale, window, 0,
                                   max(NEW), max(CTX))
    assert_window_close(out, w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("bs", [16, 8, 24, 256, 6])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3)], ids=["pairs of heads", "pairs of tiles"])
@pytest.mark.parametrize("junk", [(0.0, 0.0), (NAN, LARGE), (INF, -LARGE)], ids=str)
def test_prefill(bs, hq, hkv, junk):
    w = Window(hq, hkv, bs, CTX, 0, 0, q_lens=NEW, fp8=True, seed=bs)
    d = w.device()
    pool, own = loaded(w, *junk)
    out = pkv.paged_prefill(d["q"], *pool, d["cu_seqlens_q"], d["cu_seqlens_k"], i32(own), w.scale, max(NEW), max(CTX))
    assert_window_close(out, w)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("bs", [16, 48])
def test_prefill_that_is_not_causal(bs):
    """The same keys for every row: those that the last row of a causal call sees."""
    w = Window(4, 2, bs, [70, 150], 0, 0, q_lens=[1, 1], fp8=True, seed=3)
    pool, own = loaded(w, NAN, LARGE)
    rows = [9, 140]
    q = torch.cat([w.q[i:i + 1].expand(n, 4, 128) for i, n in enumerate(rows)]).contiguous()
    out = pkv.paged_prefill(q.cuda(), *pool, i32([0, 9, 149]), i32([0, 70, 220]), i32(own), w.scale, 140, 150,
                            causal=False)
    for at in ([0, 9], [8, 148]):
        assert_window_close(out[at], w)


def test_mixed_round():
    """The chunks of a mixed round, whose new rows end inside a block."""
    hq, hkv, bs = 8, 2, 16
    w = Window(hq, hkv, bs, [40, 90, 21], 0, 0, q_lens=[1, 30, 21], fp8=True, seed=8)
    d = w.device()
    pool, own = loaded(w, NAN, LARGE)
    slots = torch.cat([w.slots(i, range(c - n, c)) for i, (c, n) in enumerate(zip(w.ctx, w.q_lens))])
    new = [c.view(-1, hkv, 128)[slots].contiguous().cuda() for c in (w.k_cache, w.v_cache)]
    out = pkv.mixed_step(d["q"], *new, i32(slots), *pool, d["cu_seqlens_q"], d["cu_seqlens_k"], i32(own), 1, w.scale,
                         30, 90)
    assert_window_close(out, w)
    assert pkv.get_device_errors() == 0
