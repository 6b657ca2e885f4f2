"""Plain 64-bit references of the drafted-round operators, on the CPU, from their
formulas, and the inputs their tests share."""
from __future__ import annotations

import numpy as np
import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2   # largest relative error of one rounding


def i32(a, device="cuda"):
    return torch.as_tensor(np.asarray(a, np.int64).astype(np.int32)).to(device)


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16)


def bits_of(mask: np.ndarray, words: int) -> torch.Tensor:
    """[rows, n] truth values -> [rows, words] int32, bit u % 32 of word u / 32."""
    full = np.zeros((mask.shape[0], words * 32), np.uint8)
    full[:, :mask.shape[1]] = mask
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view("<i4").copy())


def ancestors(parents) -> np.ndarray:
    """[n, n] truth values: row t has t and all its ancestors."""
    n = len(parents)
    m = np.zeros((n, n), bool)
    for t, p in enumerate(parents):
        if p >= 0:
            m[t] = m[p]
        m[t, t] = True
    return m


def random_parents(rng, n):
    t = np.arange(n)
    return np.maximum(-1, t - 1 - rng.exponential(2.0, n).astype(np.int64))


class Trees:
    """A batch of drafted trees over a paged cache, on the CPU: `ctx` cached tokens and
    `sizes` drafts of each sequence, blocks at random places, -1 behind a row's blocks."""

    def __init__(self, hq, hkv, bs, ctx, sizes, seed=0, extra_rows=0, masks=None):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.bs, self.ctx, self.sizes = hq, hkv, bs, list(ctx), list(sizes)
        nblk = [-(-c // bs) for c in ctx]
        self.num_blocks = sum(nblk) + 3
        perm = rng.permutation(self.num_blocks)
        self.width = max(max(nblk, default=0), 1) + 1
        self.tables = np.full((len(ctx), self.width), -1, np.int64)
        at = 0
        for i, n in enumerate(nblk):
            self.tables[i, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
        self.rows = int(self.cu[-1]) + extra_rows
        self.max_q = max(sizes, default=0)
        self.words = max(1, (self.max_q + 31) // 32)
        self.masks = masks or [ancestors(random_parents(rng, n)) for n in sizes]
        self.q = normal((self.rows, hq, 128), seed + 1)
        self.key = normal((self.rows, hkv, 128), seed + 2)
        self.value = normal((self.rows, hkv, 128), seed + 3)
        self.k_cache = normal((self.num_blocks, bs, hkv, 128), seed + 4)
        self.v_cache = normal((self.num_blocks, bs, hkv, 128), seed + 5)
        self.scale = 128 ** -0.5

    def mask_words(self):
        w = torch.zeros((self.rows, self.words), dtype=torch.int32)
        for i, m in enumerate(self.masks):
            w[self.cu[i]:self.cu[i + 1]] = bits_of(m, self.words)
        return w

    def poison_unseen(self, bad=float("nan")):
        """Fill every cache row that no sequence owns with `bad`."""
        seen = torch.zeros(self.num_blocks * self.bs, dtype=torch.bool)
        for i, c in enumerate(self.ctx):
            p = np.arange(c)
            seen[torch.from_numpy(self.tables[i, p // self.bs] * self.bs + p % self.bs)] = True
        for c in (self.k_cache, self.v_cache):
            c.view(-1, self.hkv, 128)[~seen] = bad
        return self

    def device(self):
        d = {n: getattr(self, n).cuda() for n in ("q", "key", "value", "k_cache", "v_cache")}
        d["block_tables"], d["context_lens"] = i32(self.tables), i32(self.ctx)
        d["cu_seqlens_q"], d["tree_mask"] = i32(self.cu), self.mask_words().cuda()
        return d

    def call(self, pkv, d, **kw):
        args = dict(scale=self.scale, max_seqlen_q=self.max_q,
                    max_context_len=max(self.ctx, default=0))
        args.update(kw)
        return pkv.tree_decode(d["q"], d["key"], d["value"], d["k_cache"], d["v_cache"],
                               d["block_tables"], d["context_lens"], d["cu_seqlens_q"],
                               d["tree_mask"], **args)

    def reference(self, scale=None):
        """(out, spread) [cu[-1], Hq, 128] float64: the attention, and the same sum with
        |V|, which bounds how far rounded weights can move it."""
        scale = self.scale if scale is None else scale
        n_rows = int(self.cu[-1])
        out = torch.zeros((n_rows, self.hq, 128), dtype=torch.float64)
        spread = torch.zeros_like(out)
        group = self.hq // self.hkv
        for i, c in enumerate(self.ctx):
            a, b = int(self.cu[i]), int(self.cu[i + 1])
            p = np.arange(c)
            slots = torch.from_numpy(self.tables[i, p // self.bs] * self.bs + p % self.bs)
            kc = self.k_cache.view(-1, self.hkv, 128)[slots].double()
            vc = self.v_cache.view(-1, self.hkv, 128)[slots].double()
            for t in range(b - a):
                seen = torch.from_numpy(np.nonzero(self.masks[i][t])[0]) + a
                k = torch.cat([kc, self.key[seen].double()]).repeat_interleave(group, 1)
                v = torch.cat([vc, self.value[seen].double()]).repeat_interleave(group, 1)
                if k.shape[0] == 0:
                    continue
                s = torch.einsum("hd,xhd->hx", self.q[a + t].double(), k) * scale
                w = torch.softmax(s, -1)
                out[a + t] = torch.einsum("hx,xhd->hd", w, v)
                spread[a + t] = torch.einsum("hx,xhd->hd", w, v.abs())
        return out, spread


def assert_tree_close(got, trees, scale=None):
    """Per element: the weights are rounded to bf16 once (half a step of each term of the
    weighted sum, so of `spread`) and the result once (half a step of it). The scores are
    fp32 sums of 128 exact products: each is off by at most 128 * 2^-23 of sum |q k|,
    below 2^-16 * 0.0884 * 128 * 1.3 < 2^-11 for N(0, 1) values at scale 128^-0.5, which
    moves a weight by less than 2^-10 of itself, and so does everything else in fp32."""
    ref, spread = trees.reference(scale)
    g = got[:ref.shape[0]].double().cpu()
    bound = HALF_BF16 * (spread + ref.abs()) + 2.0 ** -10 * spread + 1e-30
    bad = ~((g - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(),
                           float((g - ref).abs().nan_to_num(1e9).max()))
