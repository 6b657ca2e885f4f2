"""A drafted round as an engine runs it, on one layer: plan the prompts' slots, rotate
and store them, prefill; then draft trees, mask them, rotate their rows, attend over
the cache; accept a path of each tree, plan its slots and store the accepted rows.
Held against the same requests decoded token by token through plain decode calls."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import HALF_BF16, i32, normal

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, VOCAB = 8, 2, 128, 16, 96, 50
SCALE = D ** -0.5


class Layer:
    """Projections of a token id (a fixed table), norms, angles, and one layer's cache."""

    def __init__(self, seed):
        self.table = normal((VOCAB, (HQ + 2 * HKV) * D), seed).cuda()
        self.qw, self.kw = (1 + normal((D,), seed + i, 0.1) for i in (1, 2))
        self.qw, self.kw = self.qw.cuda(), self.kw.cuda()
        angle = torch.arange(512, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def qkv(self, ids):
        x = self.table[torch.as_tensor(ids, device="cuda", dtype=torch.long)]
        return (x[:, :HQ * D].unflatten(1, (HQ, D)), x[:, HQ * D:-HKV * D].unflatten(1, (HKV, D)),
                x[:, -HKV * D:].unflatten(1, (HKV, D)))


class World:
    """One cache with its block tables, lengths and free list, all on the GPU."""

    def __init__(self, layer, n, seed):
        self.layer = layer
        # rows that nobody has written hold a large number, so that a read of one shows
        # (finite: paged_prefill multiplies the rows behind a chunk's last key by 0)
        self.k = torch.full((NB, BS, HKV, D), 3.0e4, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.tables = torch.full((n, 24), -1, dtype=torch.int32, device="cuda")
        self.free = i32(np.random.default_rng(seed).permutation(NB))
        self.cursor, self.lens = i32([0]), i32([0] * n)

    def plan(self, new):
        p = pkv.plan_slots(self.lens, i32(new), self.tables, self.free, self.cursor, BS, NB, sum(new))
        self.lens, self.cursor = p.context_lens, p.free_cursor
        return p

    def append(self, ids, new):
        """Rotate and store the next tokens of each request; their plan and queries."""
        p = self.plan(new)
        q, k, v = self.layer.qkv(ids)
        return p, pkv.qk_norm_rope_store(q, k, v, self.k, self.v, p.slot_mapping, p.positions,
                                         self.layer.cos_sin, self.layer.qw, self.layer.kw)

    def rows(self, i):
        n = int(self.lens[i])
        p = torch.arange(n, device="cuda")
        slots = self.tables[i].long()[p // BS] * BS + p % BS
        return self.k.flatten(0, 1)[slots], self.v.flatten(0, 1)[slots]


def test_drafted_rounds_equal_token_by_token_decoding():
    layer = Layer(3)
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in (37, 1, 16, 130)]
    n = len(prompts)
    drafted, plain = World(layer, n, 5), World(layer, n, 6)
    flat = sum(prompts, [])
    outs = []
    for w in (drafted, plain):
        p, q = w.append(flat, [len(x) for x in prompts])
        outs.append(pkv.paged_prefill(q, w.k, w.v, p.cu_seqlens_q, p.cu_seqlens_k, w.tables, SCALE,
                                      130, 130))
    assert torch.equal(outs[0], outs[1])         # blocks at other places, the same bits
    for trees in ((9, 5, 1, 33), (4, 64, 20, 2)):
        ids = [rng.integers(0, VOCAB, t).tolist() for t in trees]
        parents = [np.maximum(-1, np.arange(t) - 1 - rng.integers(0, 3, t)) for t in trees]
        cu = np.concatenate([[0], np.cumsum(trees)])
        mask, pos = pkv.tree_masks(i32(np.concatenate(parents)), i32(cu), drafted.lens, max(trees))
        q, k, v = layer.qkv(sum(ids, []))
        q, k = pkv.qk_norm_rope(q, k, pos, layer.cos_sin, layer.qw, layer.kw)
        before = [t.clone() for t in (drafted.k, drafted.v, drafted.tables)]
        out = pkv.tree_decode(q, k, v, drafted.k, drafted.v, drafted.tables, drafted.lens, i32(cu),
                              mask, SCALE, max(trees))
        for a, b in zip(before, (drafted.k, drafted.v, drafted.tables)):
            assert torch.equal(a, b)                               # drafts leave no trace
        # accept a path of each tree (none of the third's): from a node up to the root
        paths = []
        for i, t in enumerate(trees):
            path, node = [], -1 if i == 2 else int(rng.integers(0, t))
            while node >= 0:
                path.insert(0, node)
                node = int(parents[i][node])
            paths.append(path)
        rows = torch.tensor([int(cu[i]) + u for i, p in enumerate(paths) for u in p], device="cuda")
        base = drafted.lens.tolist()
        p = drafted.plan([len(x) for x in paths])
        pkv.store_kvcache(k[rows], v[rows], drafted.k, drafted.v, p.slot_mapping)
        assert p.positions.tolist() == [base[i] + d for i, x in enumerate(paths) for d in range(len(x))]
        # the same tokens, one a step
        for d in range(max(len(x) for x in paths)):
            who = [i for i, x in enumerate(paths) if d < len(x)]
            new = [1 if i in who else 0 for i in range(n)]
            _, q1 = plain.append([ids[i][paths[i][d]] for i in who], new)
            sel = torch.tensor(who, device="cuda")
            one = pkv.paged_decode(q1, plain.k, plain.v, plain.tables[sel], plain.lens[sel], SCALE)
            for j, i in enumerate(who):
                got = out[int(cu[i]) + paths[i][d]].double()
                kr, vr = (x.double().repeat_interleave(HQ // HKV, 1) for x in plain.rows(i))
                w = torch.softmax(torch.einsum("hd,xhd->hx", q1[j].double(), kr) * SCALE, -1)
                ref = torch.einsum("hx,xhd->hd", w, vr)
                spread = torch.einsum("hx,xhd->hd", w, vr.abs())
                # weights and result rounded to bf16 once each, scores in fp32 (|q|, |k| are
                # those of normed rows: sqrt(128) * 1.4 at most, so scores are off by less
                # than 2^-11 and weights by less than 2^-10 of themselves)
                bound = HALF_BF16 * (spread + ref.abs()) + 2.0 ** -10 * spread
                assert bool(((got - ref).abs() <= bound).all())
                assert bool(((one[j].double() - ref).abs() <= bound).all())
        assert pkv.get_device_errors() == 0
        assert torch.equal(drafted.lens, plain.lens)
        for i in range(n):
            for a, b in zip(drafted.rows(i), plain.rows(i)):
                assert torch.equal(a, b)
