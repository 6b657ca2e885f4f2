"""Plain 64-bit references of the fp8 cache with block scales and of attention behind a
sliding window, on the CPU, from their formulas, and the inputs their tests share."""
from __future__ import annotations

import numpy as np
import torch

from draft_testutil import HALF_BF16, i32, normal

HALF_F16 = torch.finfo(torch.float16).eps / 2


def e4m3_table() -> np.ndarray:
    """[256] float64: the value of every code (0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


TABLE = e4m3_table()


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """float64 -> codes: nearest, ties to the even code, saturated at 448, NaN to 0x7F."""
    x = np.asarray(x, np.float64)
    mag = np.where(np.isnan(x), 0.0, np.minimum(np.abs(x), 448.0))
    grid = TABLE[:127]
    hi = np.searchsorted(grid, mag).clip(0, 126)      # first code with a value >= mag
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - mag, mag - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def place(rng, counts, extra=3, width=None):
    """Block tables (-1 behind a row's blocks) over a shuffled pool, and its size."""
    num_blocks = sum(counts) + extra
    perm = rng.permutation(num_blocks)
    table = np.full((len(counts), width or max(max(counts, default=0), 1) + 1), -1, np.int64)
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, num_blocks


def store_reference(x, cache, scales, table, cu, ctx):
    """cache [NB, bs, H, 128] uint8 and scales [NB, H] float64 after the rows x [T, H, 128]."""
    cache, scales = cache.copy(), scales.copy()
    bs = cache.shape[1]
    x = x.double().numpy()
    for i, c in enumerate(ctx):
        n = cu[i + 1] - cu[i]
        start = c - n
        p = start
        while p < c:
            b, off = table[i][p // bs], p % bs
            end = min(c, p - off + bs)
            rows = x[cu[i] + p - start:cu[i] + end - start]                # [m, H, 128]
            top = np.where(np.isfinite(rows), np.abs(rows), 0.0).max((0, 2))
            s = np.full(top.shape, 2.0 ** -120)
            for e in range(-120, 119):
                s = np.where(top > 448 * 2.0 ** e, 2.0 ** (e + 1), s)
            if off:
                s = np.maximum(s, scales[b])
                old = TABLE[cache[b, :off]] * (scales[b] / s)[None, :, None]
                cache[b, :off] = np.where((s == scales[b])[None, :, None], cache[b, :off], to_e4m3(old))
            cache[b, off:off + end - p] = to_e4m3(rows / s[None, :, None])
            scales[b] = s
            p = end
    return cache, scales


def codes_pool(shape, seed):
    """Random finite codes and power-of-two scales [NB, H] of a pool [NB, bs, H, 128]."""
    rng = np.random.default_rng(seed)
    mag = to_e4m3(rng.standard_normal(shape) * 100)
    return mag, 2.0 ** rng.integers(-9, -4, (shape[0], shape[2])).astype(np.float64)


class Window:
    """Requests over a paged cache, bf16 or fp8 with block scales, on the CPU: sequence i has
    ctx[i] tokens, and queries at its last q_lens[i] positions."""

    def __init__(self, hq, hkv, bs, ctx, window, sinks, q_lens=None, fp8=False, seed=0, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.bs, self.ctx = hq, hkv, bs, list(ctx)
        self.window, self.sinks, self.fp8 = window, sinks, fp8
        self.q_lens = list(q_lens) if q_lens is not None else [1] * len(self.ctx)
        self.prefill = q_lens is not None
        self.tables, self.num_blocks = place(rng, [-(-c // bs) for c in ctx])
        self.cu = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int64)
        self.rows = int(self.cu[-1]) + extra_rows
        self.q = normal((self.rows, hq, 128), seed + 1)
        shape = (self.num_blocks, bs, hkv, 128)
        if fp8:
            (k, ks), (v, vs) = codes_pool(shape, seed + 2), codes_pool(shape, seed + 3)
            self.k_cache, self.v_cache = torch.from_numpy(k), torch.from_numpy(v)
            self.k_scales, self.v_scales = torch.from_numpy(ks).float(), torch.from_numpy(vs).float()
        else:
            self.k_cache, self.v_cache = normal(shape, seed + 4), normal(shape, seed + 5)
        self.scale = 128 ** -0.5

    def slots(self, i, p):
        p = np.asarray(p)
        return torch.from_numpy(self.tables[i, p // self.bs] * self.bs + p % self.bs)

    def seen(self, i, t):
        """Positions that the query at position t sees."""
        p = np.arange(t + 1)
        return p[(p < self.sinks) | (p > t - self.window)] if self.window else p

    def rows_of(self, cache, scales, slots):
        if not self.fp8:
            return cache.view(-1, self.hkv, 128)[slots].double()
        x = torch.from_numpy(TABLE[cache.view(-1, self.hkv, 128)[slots].numpy()])
        return x * scales[slots // self.bs].double()[..., None]

    def poison_unseen(self):
        """NaN into every cache row that no query sees."""
        seen = torch.zeros(self.num_blocks * self.bs, dtype=torch.bool)
        for i, c in enumerate(self.ctx):
            for t in range(c - self.q_lens[i], c) if c else ():
                seen[self.slots(i, self.seen(i, t))] = True
        for c in (self.k_cache, self.v_cache):
            c.view(-1, self.hkv, 128)[~seen] = 0x7F if self.fp8 else float("nan")
        return self

    def device(self):
        names = ["q", "k_cache", "v_cache"] + (["k_scales", "v_scales"] if self.fp8 else [])
        d = {n: getattr(self, n).cuda() for n in names}
        d["block_tables"], d["context_lens"] = i32(self.tables), i32(self.ctx)
        d["cu_seqlens_q"] = i32(self.cu)
        d["cu_seqlens_k"] = i32(np.concatenate([[0], np.cumsum(self.ctx)]))
        return d

    def call(self, pkv, d, **kw):
        longest = max(self.ctx, default=0)
        if self.prefill:
            return pkv.paged_prefill_window(d["q"], d["k_cache"], d["v_cache"], d["cu_seqlens_q"],
                                            d["cu_seqlens_k"], d["block_tables"], self.scale, self.window,
                                            self.sinks, max(self.q_lens, default=0), longest, **kw)
        kw.setdefault("max_context_len", longest)
        if self.fp8:
            return pkv.paged_decode_fp8_block(d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"],
                                              d["block_tables"], d["context_lens"], self.scale,
                                              window=self.window, sinks=self.sinks, **kw)
        return pkv.paged_decode_window(d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"],
                                       self.scale, self.window, self.sinks, **kw)

    def reference(self):
        """(out, spread, most) [cu[-1], Hq, 128]: the attention, the same sum with |V|, and the
        number of seen keys times the largest |V| among them."""
        out = torch.zeros((int(self.cu[-1]), self.hq, 128), dtype=torch.float64)
        spread, most = torch.zeros_like(out), torch.zeros_like(out)
        g = self.hq // self.hkv
        for i, c in enumerate(self.ctx):
            for u in range(self.q_lens[i] if c else 0):
                p = self.seen(i, c - self.q_lens[i] + u)
                sl = self.slots(i, p)
                k = self.rows_of(self.k_cache, getattr(self, "k_scales", None), sl).repeat_interleave(g, 1)
                v = self.rows_of(self.v_cache, getattr(self, "v_scales", None), sl).repeat_interleave(g, 1)
                r = int(self.cu[i]) + u
                w = torch.softmax(torch.einsum("hd,xhd->hx", self.q[r].double(), k) * self.scale, -1)
                out[r] = torch.einsum("hx,xhd->hd", w, v)
                spread[r] = torch.einsum("hx,xhd->hd", w, v.abs())
                most[r] = len(p) * v.abs().amax(0)
        return out, spread, most


def assert_window_close(got, w):
    """Per element. bf16 cache: the weights are rounded to bf16 (half a step of each term of the
    weighted sum, so of `spread`); fp8 cache: to f16, whose step below 2^-14 is fixed, so that a
    weight is also off by up to 2^-25 where the largest is at least 2^-1: together below
    2^-24 * `most`. The result is rounded once (half a bf16 step of it). The scores are fp32 sums
    of 128 exact products: each is off by at most 128 * 2^-23 of scale * sum |q k|, which is about
    0.0884 * 128 * 0.8 * 0.8 for N(0, 1) values and at most 3.2 times that for the fp8 pools (their
    largest deviation is 100 * 2^-5), so below 2^-16 * 23 < 2^-11; that moves a weight and the sum of
    weights by less than 2^-11 of themselves each, and everything else in fp32 is far below it."""
    ref, spread, most = w.reference()
    g = got[:ref.shape[0]].double().cpu()
    half = HALF_F16 if w.fp8 else HALF_BF16
    bound = half * spread + HALF_BF16 * ref.abs() + 2.0 ** -10 * spread + (2.0 ** -24 * most if w.fp8 else 0) + 1e-30
    same = (g - ref).abs() <= bound
    same |= (ref.isnan() & g.isnan()) | (ref == g)
    bad = ~same
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(),
                           float((g - ref).abs().nan_to_num(1e9).max()))
