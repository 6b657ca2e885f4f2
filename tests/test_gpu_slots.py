"""pkv_plan_slots and pkv_tree_masks against the host's bookkeeping, number for number."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import ancestors, bits_of, i32, random_parents
from paged_kv_cache_86_gb300 import _lib

pytestmark = pytest.mark.gpu


class Host:
    """The same plan in plain Python: FIFO free list, one entry at a time."""

    def __init__(self, ctx, new, bs, tables, free, cursor, max_tokens):
        self.tables = [list(map(int, r)) for r in tables]
        self.slots, self.pos, self.lens = [], [], []
        self.cu_q, self.cu_k = [0], [0]
        for i, (c, n) in enumerate(zip(ctx, new)):
            for p in range(c, c + n):
                if p % bs == 0:
                    self.tables[i][p // bs] = int(free[cursor])
                    cursor += 1
                self.slots.append(self.tables[i][p // bs] * bs + p % bs)
                self.pos.append(p)
            self.lens.append(c + n)
            self.cu_q.append(self.cu_q[-1] + n)
            self.cu_k.append(self.cu_k[-1] + c + n)
        pad = max_tokens - len(self.slots)
        self.slots += [-1] * pad
        self.pos += [0] * pad
        self.cursor = cursor


def setup(ctx, new, bs, seed=0, spare=4, width=None):
    rng = np.random.default_rng(seed)
    have = [-(-c // bs) for c in ctx]
    need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    nb = sum(need) + spare + 3
    perm = rng.permutation(nb)
    width = width or max(need + [1]) + 2
    tables = np.full((len(ctx), width), -1, np.int64)
    at = 0
    for i, n in enumerate(have):
        tables[i, :n] = perm[at:at + n]
        at += n
    return tables, perm[at:], nb


def run(ctx, new, bs, tables, free, cursor, nb, max_tokens, **kw):
    bt = i32(tables)
    p = pkv.plan_slots(i32(ctx), i32(new), bt, i32(free), i32([cursor]), bs, nb, max_tokens, **kw)
    return p, bt


def same(plan, bt, h):
    assert plan.slot_mapping.tolist() == h.slots
    assert plan.positions.tolist() == h.pos
    assert plan.cu_seqlens_q.tolist() == h.cu_q and plan.cu_seqlens_k.tolist() == h.cu_k
    assert plan.context_lens.tolist() == h.lens
    assert plan.free_cursor.tolist() == [h.cursor]
    assert bt.tolist() == h.tables


RNG = np.random.default_rng(1)
CASES = [
    ([5], [1], 16, 0),
    ([0], [1], 1, 0),
    ([16], [1], 16, 3),
    ([15, 16, 17, 0], [1, 1, 1, 0], 16, 0),
    ([0, 0, 3], [0, 40, 0], 7, 5),
    ([100, 0, 33], [512, 600, 1], 16, 11),
    (RNG.integers(0, 4096, 512).tolist(), [1] * 512, 16, 0),
    (RNG.integers(0, 90, 1025).tolist(), RNG.integers(0, 5, 1025).tolist(), 3, 0),
    (RNG.integers(0, 50, 3000).tolist(), RNG.integers(0, 3, 3000).tolist(), 256, 100),
    ([0] * 1024 + [9], [0] * 1024 + [2000], 8, 0),
    ([7], [5000], 16, 0),
    ([], [], 16, 5),
]


@pytest.mark.parametrize("ctx,new,bs,pad", CASES)
def test_plan_equals_the_host(ctx, new, bs, pad):
    tables, free, nb = setup(ctx, new, bs, seed=len(ctx))
    n = sum(new) + pad
    plan, bt = run(ctx, new, bs, tables, free, 2, nb, n)
    assert pkv.get_device_errors() == 0
    same(plan, bt, Host(ctx, new, bs, tables, free, 2, n))


def test_plan_follows_the_block_manager():
    from paged_kv_cache_86_gb300.block_manager import BlockManager, Sequence
    bm = BlockManager(64, 4)
    for i, n in enumerate((5, 8, 1)):
        bm.allocate(Sequence(i, [i * 100 + t for t in range(n)], 4))
    tables, free = bm.block_table_rows(range(3), width=8), list(bm.free_block_ids)
    ctx = [len(bm.seqs[i]) for i in range(3)]
    plan, bt = run(ctx, [1, 1, 1], 4, tables, free, 0, 64, 3)
    for i in range(3):
        bm.append_token(i, 7)
    assert bt.tolist() == bm.block_table_rows(range(3), width=8)
    assert plan.slot_mapping.tolist() == [bm.seqs[i].slot(ctx[i]) for i in range(3)]


def test_rounds_chain_on_the_device_and_in_a_graph():
    ctx, new, bs = [3, 0, 15, 40], [1, 1, 1, 1], 8
    tables, free, nb = setup(ctx, [60] * 4, bs)
    bt, lens, cursor = i32(tables), i32(ctx), i32([0])
    nl, fr = i32(new), i32(free)
    out = pkv.plan_slots(lens, nl, bt.clone(), fr, cursor, bs, nb, 6)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.plan_slots(lens, nl, bt, fr, cursor, bs, nb, 6, out=out)
        lens.copy_(out.context_lens)
        cursor.copy_(out.free_cursor)
    cur, h_tables = 0, tables
    for _ in range(30):
        h = Host(ctx, new, bs, h_tables, free, cur, 6)
        graph.replay()
        torch.cuda.synchronize()
        same(out, bt, h)
        ctx, cur, h_tables = h.lens, h.cursor, h.tables
    assert pkv.get_device_errors() == 0


def test_lengths_and_rows_that_do_not_fit_are_cut():
    # rows: 30 wanted, 20 given; the second request keeps 8 of its 18, the third none
    ctx, new, bs = [4, 10, 7], [12, 18, 5], 8
    tables, free, nb = setup(ctx, new, bs)
    plan, bt = run(ctx, new, bs, tables, free, 0, nb, 20)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH
    same(plan, bt, Host(ctx, [12, 8, 0], bs, tables, free, 0, 20))
    # a table of 2 blocks of 8: the request stops at 16 tokens; negative lengths count as none
    tables, free, nb = setup([10, 3, 0], [6, 1, 0], 8, width=2)
    plan, bt = run([10, 3, -4], [20, 1, -1], 8, tables, free, 0, nb, 9)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH
    same(plan, bt, Host([10, 3, 0], [6, 1, 0], 8, tables, free, 0, 9))


def test_a_free_list_that_runs_out():
    ctx, new, bs = [8, 8, 8], [9, 1, 8], 8       # 2 + 1 + 1 blocks wanted, 3 left
    tables, free, nb = setup(ctx, new, bs)
    free = free[:5]
    plan, bt = run(ctx, new, bs, tables, free, 2, nb, 18)
    assert pkv.get_device_errors() == _lib.DEVERR_NO_BLOCKS
    h = Host(ctx, [9, 1, 0], bs, tables, free, 2, 18)
    assert plan.slot_mapping.tolist() == h.slots[:10] + [-1] * 8
    assert plan.positions.tolist() == h.pos[:10] + list(range(8, 16))
    assert plan.context_lens.tolist() == [17, 9, 16] and plan.free_cursor.tolist() == [5]
    assert bt.tolist() == h.tables
    for cursor in (-1, 6):                       # a cursor outside the list
        plan, _ = run(ctx, [0, 0, 0], bs, tables, free, cursor, nb, 1)
        assert pkv.get_device_errors() == _lib.DEVERR_NO_BLOCKS


def test_bad_ids_give_skipped_slots():
    ctx, new, bs = [3, 8, 5], [2, 2, 1], 8
    tables, free, nb = setup(ctx, new, bs)
    tables[0, 0], tables[2, 0] = nb, -1
    free[0] = nb + 9
    plan, bt = run(ctx, new, bs, tables, free, 0, nb, 5)
    assert pkv.get_device_errors() == _lib.DEVERR_BLOCK_ID
    assert plan.slot_mapping.tolist() == [-1] * 5
    assert plan.positions.tolist() == [3, 4, 8, 9, 5]
    assert bt[1, 1].item() == -1


def test_plan_on_another_stream_and_on_used_buffers():
    ctx, new, bs = [100, 5, 33], [70, 1, 9], 16
    tables, free, nb = setup(ctx, new, bs)
    h = Host(ctx, new, bs, tables, free, 0, 90)
    args = [i32(a) for a in (ctx, new, tables, free, [0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = pkv.plan_slots(*args, bs, nb, 90, stream=side)
    side.synchronize()
    same(plan, args[2], h)
    for t in plan:
        t.fill_(77)
    again = pkv.plan_slots(*args, bs, nb, 90, out=plan)
    assert again is plan
    same(plan, args[2], h)


# ------------------------------------------------------------------- masks --

SIZES = [[1], [8], [0, 5, 0, 1, 0], [64, 33, 32, 31], [129, 2, 128], [1500, 700],
         RNG.integers(0, 65, 300).tolist()]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_masks_equal_the_ancestors(sizes, kind):
    rng = np.random.default_rng(len(sizes))
    make = {"random": lambda n: random_parents(rng, n), "chain": lambda n: np.arange(n) - 1,
            "star": lambda n: np.full(n, -1)}[kind]
    parents = [make(n) for n in sizes]
    ctx = rng.integers(0, 30000, len(sizes))
    cu = np.concatenate([[0], np.cumsum(sizes)])
    words = (max(sizes) + 31) // 32
    mask, pos = pkv.tree_masks(i32(np.concatenate(parents)), i32(cu), i32(ctx), max(sizes))
    assert pkv.get_device_errors() == 0
    anc = [ancestors(p) for p in parents]
    want = torch.cat([bits_of(m, words) for m in anc])
    assert torch.equal(mask.cpu(), want)
    assert pos.tolist() == [int(c + r.sum()) - 1 for c, m in zip(ctx, anc) for r in m]


def test_masks_keep_rows_behind_the_last_tree_and_fill_wide_rows():
    parents = i32([-1, 0, 0, -1, 0, 5, 5])
    mask = torch.full((7, 3), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((7,), 77, dtype=torch.int32, device="cuda")
    pkv.tree_masks(parents, i32([0, 3, 5]), i32([10, 20]), 3, tree_mask=mask, positions=pos)
    assert pkv.get_device_errors() == 0
    assert mask.tolist() == [[1, 0, 0], [3, 0, 0], [5, 0, 0], [1, 0, 0], [3, 0, 0],
                             [77] * 3, [77] * 3]
    assert pos.tolist() == [10, 11, 11, 20, 21, 77, 77]


def test_bad_links_and_lengths_are_reported():
    # a link to itself, forwards and below -1 counts as the root
    mask, pos = pkv.tree_masks(i32([0, 0, 3, 1, -2]), i32([0, 5]), i32([9]), 5)
    assert pkv.get_device_errors() == _lib.DEVERR_TREE
    assert mask.flatten().tolist() == [1, 3, 4, 11, 16] and pos.tolist() == [9, 10, 9, 11, 9]
    mask = torch.full((5, 1), 77, dtype=torch.int32, device="cuda")
    pkv.tree_masks(i32([-1] * 5), i32([0, 4, 5]), i32([9, 9]), 3, tree_mask=mask)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH
    assert mask.flatten().tolist() == [77] * 4 + [1]
    pkv.tree_masks(i32([-1] * 5), i32([0, 2, 6]), i32([9, 9]), 5, tree_mask=mask)
    assert pkv.get_device_errors() == _lib.DEVERR_LENGTH
