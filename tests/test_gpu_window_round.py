"""Rounds over an fp8 cache with block scales as a server runs them: slots planned, prompts stored and
attended to through the read-back, then tokens one by one, behind a sliding window and without one."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32, normal
from window_testutil import Window, assert_window_close, store_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 7])
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_rounds(bs, window, sinks):
    hq, hkv, s = 8, 2, 4
    prompts = [70, 1, 33, 0]
    num_blocks, mb = 64, 24
    shape = (num_blocks, bs, hkv, 128)
    caches = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(num_blocks, hkv, device="cuda") for _ in range(2)]
    tables = torch.full((s, mb), -1, dtype=torch.int32, device="cuda")
    free = i32(np.random.default_rng(0).permutation(num_blocks))
    cursor, lens = i32([0]), i32([0] * s)
    held = [(np.zeros(shape, np.uint8), np.ones((num_blocks, hkv))) for _ in range(2)]
    for step in range(20):
        new = prompts if step == 0 else [1, 1, 0 if step == 3 else 1, 2 if step == 1 else 1]
        plan = pkv.plan_slots(lens, i32(new), tables, free, cursor, bs, num_blocks, sum(new))
        lens, cursor = plan.context_lens, plan.free_cursor
        key, value = normal((sum(new), hkv, 128), 100 + step), normal((sum(new), hkv, 128), 200 + step)
        key = (key.float() * (1 + step % 5)).to(torch.bfloat16)
        pkv.store_kvcache_fp8_block(key.cuda(), value.cuda(), *caches, *scales, tables, plan.cu_seqlens_q, lens)
        t, ctx, cu = tables.cpu().numpy(), lens.tolist(), plan.cu_seqlens_q.tolist()
        held = [store_reference(x, *h, t, cu, ctx) for x, h in zip((key, value), held)]
        for c, sc, h in zip(caches, scales, held):
            assert np.array_equal(c.cpu().numpy(), h[0]) and np.array_equal(sc.double().cpu().numpy(), h[1])
        w = Window(hq, hkv, bs, ctx, window, sinks, q_lens=new if step == 0 else None, fp8=True, seed=step)
        w.tables, w.num_blocks = t, num_blocks
        w.k_cache, w.v_cache = torch.from_numpy(held[0][0]), torch.from_numpy(held[1][0])
        w.k_scales, w.v_scales = torch.from_numpy(held[0][1]).float(), torch.from_numpy(held[1][1]).float()
        if step == 0:
            # prompts: the cache read back into a bf16 pool of consecutive blocks
            blocks = [-(-c // bs) for c in ctx]
            first = np.concatenate([[0], np.cumsum(blocks)])
            pool = [torch.full((int(first[-1]), bs, hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
                    for _ in range(2)]
            pkv.load_kvcache_fp8_block(*caches, *scales, tables, lens, i32(first[:-1] * bs),
                                       key_out=pool[0].view(-1, hkv, 128), value_out=pool[1].view(-1, hkv, 128))
            own = np.full((s, max(blocks)), -1)
            for i, n in enumerate(blocks):
                own[i, :n] = first[i] + np.arange(n)
            out = pkv.paged_prefill_window(w.q.cuda(), *pool, plan.cu_seqlens_q, plan.cu_seqlens_k, i32(own),
                                           w.scale, window or 1 << 20, sinks, max(new), max(ctx))
            w.fp8, (w.k_cache, w.v_cache), w.tables = False, [p.cpu() for p in pool], own
            w.num_blocks = int(first[-1])
        else:
            out = pkv.paged_decode_fp8_block(w.q.cuda(), *caches, *scales, tables, lens, w.scale, window, sinks)
        assert_window_close(out, w)
    assert pkv.get_device_errors() == 0


def test_plan_after_plan_slots_counts_new_tokens():
    """context_lens of a plan already counts the new tokens: the arrays go to the store unchanged."""
    tables = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    plan = pkv.plan_slots(i32([0, 0]), i32([3, 5]), tables, i32(range(8)), i32([0]), 4, 8, 8)
    assert plan.context_lens.tolist() == [3, 5] and plan.cu_seqlens_q.tolist() == [0, 3, 8]
