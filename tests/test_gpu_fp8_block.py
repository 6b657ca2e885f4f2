"""The fp8 cache with block scales, written and read back, against the plain definition: codes and
scales are whole numbers and powers of two, so everything is compared exactly."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32, normal
from window_testutil import TABLE, codes_pool, place, store_reference

pytestmark = pytest.mark.gpu


class Store:
    def __init__(self, hkv, bs, before, new, seed=0, extra_rows=0, size=0.7):
        rng = np.random.default_rng(seed)
        self.hkv, self.bs = hkv, bs
        self.after = [c + n for c, n in zip(before, new)]
        self.tables, self.num_blocks = place(rng, [-(-a // bs) for a in self.after])
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        rows = int(self.cu[-1]) + extra_rows
        shape = (self.num_blocks, bs, hkv, 128)
        g = torch.Generator().manual_seed(seed)
        grow = torch.exp(size * torch.randn(rows, 1, 1, generator=g))
        self.x = [(normal((rows, hkv, 128), seed + i).float() * grow).to(torch.bfloat16) for i in (1, 2)]
        self.pools = [codes_pool(shape, seed + i) for i in (3, 4)]

    def run(self, x=None, tables=None, after=None, cu=None, total=None):
        x = [t.cuda() for t in (x or self.x)]
        caches = [torch.from_numpy(c).cuda() for c, _ in self.pools]
        scales = [torch.from_numpy(s).float().cuda() for _, s in self.pools]
        pkv.store_kvcache_fp8_block(x[0], x[1], *caches, *scales,
                                    i32(self.tables if tables is None else tables),
                                    i32(self.cu if cu is None else cu),
                                    i32(self.after if after is None else after))
        return [c.cpu().numpy() for c in caches], [s.double().cpu().numpy() for s in scales]

    def check(self, x=None, ref=None):
        caches, scales = self.run(x)
        for i in range(2):
            want = ref[i] if ref else store_reference((x or self.x)[i], *self.pools[i], self.tables, self.cu,
                                                      self.after)
            assert np.array_equal(scales[i], want[1])
            assert np.array_equal(caches[i], want[0])
        assert pkv.get_device_errors() == 0
        return caches, scales


@pytest.mark.parametrize("hkv,bs,before,new", [
    (2, 16, [0], [1]),
    (8, 16, [0, 5, 15, 16, 31, 40], [1, 1, 1, 1, 1, 1]),          # a decode round, blocks begun and filled
    (8, 16, [0, 3, 16, 100], [40, 13, 16, 1]),                    # a prefill round
    (1, 1, [0, 4], [7, 1]),                                       # one token a block
    (3, 7, [0, 6, 20], [1, 30, 0]),                               # an odd block size, an empty row
    (6, 24, [11, 0, 0, 5], [0, 0, 50, 1]),
    (5, 8, [9, 4], [100, 3]),                                     # ten (head, K or V) pairs in CTAs of sixteen
    (17, 16, [5, 0], [20, 2]),                                    # more pairs than a CTA has half-warps
    (2, 256, [0, 200, 255, 256], [256, 300, 1, 700]),             # full blocks of many rows
    (2, 256, [3] + [10] * 40, [500] + [1] * 40),                  # one long request among single tokens
    (4, 300, [290, 0], [400, 5]),                                 # more rows a block than half-warps hold at once
], ids=str)
def test_store_is_exact(hkv, bs, before, new):
    Store(hkv, bs, before, new).check()


def test_scales_grow_and_older_codes_move():
    """New rows far above, near and far below what the blocks hold."""
    for size in (1e-3, 0.5, 4.0, 300.0, 1e6):
        s = Store(4, 16, [5, 8, 1, 15], [1, 2, 15, 30], seed=7)
        x = [(t.float() * size).to(torch.bfloat16) for t in s.x]
        caches, scales = s.check(x)
        grown = sum((a != p[1]).sum() for a, p in zip(scales, s.pools))
        assert grown > 0 or size < 1


def test_codes_that_turn_subnormal_round_to_nearest_even():
    s = Store(1, 16, [15], [1])
    b = s.tables[0, 0]
    for cache, scale in s.pools:
        cache[b, :15] = (np.arange(15 * 128) % 127).reshape(15, 1, 128)      # every magnitude
        scale[b] = 2.0 ** -6
    for e in (1, 3, 6, 9, 12, 20):
        x = [torch.full_like(t, 2.0 ** e) for t in s.x]
        s.check(x)


def test_values_at_the_borders_of_a_scale():
    """448 * 2^e is the last value of its scale; the next bf16 value takes the next one."""
    for v, e in ((448.0, 0), (450.0, 1), (1.75, -8), (1.7578125, -7), (2.0 ** -130, -120), (0.0, -120),
                 (3.3e38, 119), (2.0 ** 127, 119)):
        s = Store(1, 4, [0], [1])
        x = [torch.zeros_like(t) for t in s.x]
        for t in x:
            t[0, 0, 5] = -v
        _, scales = s.check(x)
        assert scales[0][s.tables[0, 0], 0] == 2.0 ** e


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("new", [[3], [200]], ids=str)
def test_what_is_not_finite_stays_out_of_the_scale(bad, new):
    s = Store(2, 64, [2], new, seed=3)
    x = [t.clone() for t in s.x]
    for t in x:
        t[1, 1, 7] = bad
        t[new[0] - 1, 0, 100] = bad
    caches, _ = s.check(x)
    want = {float("inf"): 0x7E, float("-inf"): 0xFE}.get(bad, 0x7F)
    p = 2 + 1
    assert caches[0][s.tables[0, p // 64], p % 64, 1, 7] == want
    x = [torch.full_like(t, bad) for t in s.x]              # nothing finite at all
    s.check(x)


def test_token_by_token_is_one_store_of_rows_of_falling_size():
    """A block filled in steps ends as it does in one call when the first row is the largest, and in
    any order its scale does."""
    full = Store(2, 16, [0, 0], [40, 17], seed=11, size=0.0)
    for falling in (True, False):
        x = [t.float() * torch.linspace(4, 1, t.shape[0])[:, None, None] if falling else t.float() for t in full.x]
        x = [t.to(torch.bfloat16) for t in x]
        whole_c, whole_s = full.check(x)
        caches = [torch.from_numpy(c).cuda() for c, _ in full.pools]
        scales = [torch.from_numpy(s).float().cuda() for _, s in full.pools]
        tables, xg = i32(full.tables), [t.cuda() for t in x]
        for t in range(40):
            rows = [0, 1] if t < 17 else [0]
            at = torch.tensor([full.cu[r] + t for r in rows]).cuda()
            pkv.store_kvcache_fp8_block(xg[0][at], xg[1][at], *caches, *scales, tables[:len(rows)].contiguous(),
                                        i32(range(len(rows) + 1)), i32([t + 1] * len(rows)))
        for i in range(2):
            assert np.array_equal(scales[i].double().cpu().numpy(), whole_s[i])
            if falling and i == 0:
                live = full.tables[0, :2]
                assert np.array_equal(caches[i].cpu().numpy()[live], whole_c[i][live])


def test_strided_rows_padding_and_other_rows():
    s = Store(4, 16, [3, 9], [20, 1], extra_rows=6)
    fused = torch.cat([s.x[0], normal((s.x[0].shape[0], 3, 128), 5), s.x[1]], 1).cuda()
    ref = [store_reference(x, *p, s.tables, s.cu, s.after) for x, p in zip(s.x, s.pools)]
    caches = [torch.from_numpy(c).cuda() for c, _ in s.pools]
    scales = [torch.from_numpy(c).float().cuda() for _, c in s.pools]
    pkv.store_kvcache_fp8_block(fused[:, :4], fused[:, 7:], *caches, *scales, i32(s.tables), i32(s.cu), i32(s.after))
    for i in range(2):
        assert np.array_equal(caches[i].cpu().numpy(), ref[i][0])
        assert np.array_equal(scales[i].double().cpu().numpy(), ref[i][1])


def test_bad_blocks_and_lengths_are_skipped():
    s = Store(2, 16, [5, 0, 20], [30, 4, 2], seed=2)
    ref = [store_reference(x, *p, s.tables, s.cu, s.after) for x, p in zip(s.x, s.pools)]
    tables = s.tables.copy()
    lost = tables[0, 1]
    tables[0, 1] = s.num_blocks
    caches, scales = s.run(tables=tables)
    assert pkv.get_device_errors() == 2
    for i in range(2):
        keep = np.arange(s.num_blocks) != lost
        assert np.array_equal(caches[i][keep], ref[i][0][keep]) and np.array_equal(scales[i][keep], ref[i][1][keep])
        assert np.array_equal(caches[i][lost], s.pools[i][0][lost])
    for bad in (-1, 29, s.tables.shape[1] * 16 + 1):
        caches, scales = s.run(after=[bad] + s.after[1:])
        assert pkv.get_device_errors() == 4
        first = s.tables[0][s.tables[0] >= 0]
        for i in range(2):
            keep = ~np.isin(np.arange(s.num_blocks), first)
            assert np.array_equal(caches[i][keep], ref[i][0][keep])
            assert np.array_equal(caches[i][first], s.pools[i][0][first])


# ------------------------------------------------------------------ load --

class Load:
    def __init__(self, hkv, bs, ctx, seed=0):
        rng = np.random.default_rng(seed)
        self.ctx, self.bs, self.hkv = list(ctx), bs, hkv
        self.tables, self.num_blocks = place(rng, [-(-c // bs) for c in ctx])
        self.pools = [codes_pool((self.num_blocks, bs, hkv, 128), seed + i) for i in (1, 2)]

    def args(self):
        return ([torch.from_numpy(c).cuda() for c, _ in self.pools]
                + [torch.from_numpy(s).float().cuda() for _, s in self.pools]
                + [i32(self.tables), i32(self.ctx)])

    def rows(self, which, i):
        c, s = self.pools[which]
        p = np.arange(self.ctx[i])
        b = self.tables[i, p // self.bs]
        return torch.from_numpy(TABLE[c[b, p % self.bs]] * s[b][..., None]).to(torch.bfloat16)


@pytest.mark.parametrize("hkv,bs,ctx", [(2, 16, [300, 70]), (8, 16, [1, 0, 17, 64]), (1, 1, [5, 1]), (3, 7, [20, 6, 7]),
                                        (6, 256, [257, 255, 3]), (16, 48, [100]), (8, 16, [1] * 60 + [0] * 5 + [40])],
                         ids=str)
@pytest.mark.parametrize("gap", [0, 3])
def test_load_is_exact_and_leaves_other_rows(hkv, bs, ctx, gap):
    w = Load(hkv, bs, ctx)
    starts = np.concatenate([[0], np.cumsum([c + gap for c in ctx])])[:-1] + gap
    num = int(starts[-1]) + ctx[-1] + gap
    out = [torch.full((num, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = pkv.load_kvcache_fp8_block(*w.args(), i32(starts), key_out=out[0], value_out=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    for which in range(2):
        want = torch.full((num, hkv, 128), 7.0, dtype=torch.bfloat16)
        for i, c in enumerate(ctx):
            want[starts[i]:starts[i] + c] = w.rows(which, i)
        assert torch.equal(got[which].cpu(), want)
    assert pkv.get_device_errors() == 0


def test_load_strided_nan_and_cut_rows():
    w = Load(2, 16, [40, 9])
    b = w.tables[0, 1]
    w.pools[0][0][b, 3, 1, 9] = 0x7F
    w.pools[1][1][b, 0] = 0.3                                # a scale that is no power of two: one rounding
    fused = torch.zeros(45, 4, 128, dtype=torch.bfloat16, device="cuda")
    pkv.load_kvcache_fp8_block(*w.args(), i32([0, 40]), key_out=fused[:, :2], value_out=fused[:, 2:])
    for which in range(2):
        want = torch.cat([w.rows(which, 0), w.rows(which, 1)])[:45]
        c, s = w.pools[which]
        if which == 1:                                       # fp32 scale, rounded to bf16 from the exact product
            x = torch.from_numpy(TABLE[c[b, :, 0]] * float(np.float32(0.3)))
            want[16:32, 0] = x.to(torch.bfloat16)
        got = fused[:, 2 * which:2 * which + 2].cpu()
        assert torch.equal(got.nan_to_num(99.0), want.nan_to_num(99.0))
    assert pkv.get_device_errors() == 0


def test_load_bad_blocks_and_lengths():
    w = Load(2, 16, [40, 9])
    a = w.args()
    bad = w.tables.copy()
    bad[0, 1] = -5
    a[4] = i32(bad)
    out = [torch.full((49, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkv.load_kvcache_fp8_block(*a, i32([0, 40]), key_out=out[0], value_out=out[1])
    assert pkv.get_device_errors() == 2
    want = torch.cat([w.rows(0, 0), w.rows(0, 1)])
    want[16:32] = 7.0
    assert torch.equal(out[0].cpu(), want)
    a = w.args()
    a[5] = i32([40, w.tables.shape[1] * 16 + 1])
    pkv.load_kvcache_fp8_block(*a, i32([0, 40]), num_rows=40 + w.tables.shape[1] * 16 + 1)
    assert pkv.get_device_errors() & 4
    a[5] = i32([-3, 9])
    pkv.load_kvcache_fp8_block(*a, i32([0, 40]), num_rows=49)
    assert pkv.get_device_errors() == 4


def test_pools_past_32_bit_offsets():
    """Blocks behind the first 4 GB of the caches, written and read back."""
    s = Store(8, 16, [5, 0], [30, 20])
    far = (1 << 32) // (16 * 8 * 128) + 3
    caches, scales = [], []
    for c, sc in s.pools:
        cache = torch.empty((far + s.num_blocks, 16, 8, 128), dtype=torch.uint8, device="cuda")
        cache[far:] = torch.from_numpy(c).cuda()
        scale = torch.ones((far + s.num_blocks, 8), device="cuda")
        scale[far:] = torch.from_numpy(sc).float().cuda()
        caches.append(cache)
        scales.append(scale)
    tables = i32(np.where(s.tables >= 0, s.tables + far, -1))
    pkv.store_kvcache_fp8_block(s.x[0].cuda(), s.x[1].cuda(), *caches, *scales, tables, i32(s.cu), i32(s.after))
    got = pkv.load_kvcache_fp8_block(*caches, *scales, tables, i32(s.after), i32([0, s.after[0]]), sum(s.after))
    for i in range(2):
        want = store_reference(s.x[i], *s.pools[i], s.tables, s.cu, s.after)
        assert np.array_equal(caches[i][far:].cpu().numpy(), want[0])
        rows = []
        for r, a in enumerate(s.after):
            p = np.arange(a)
            b = s.tables[r, p // 16]
            rows.append(torch.from_numpy(TABLE[want[0][b, p % 16]] * want[1][b][..., None]).to(torch.bfloat16))
        assert torch.equal(got[i].cpu(), torch.cat(rows))
    assert pkv.get_device_errors() == 0


def test_captured_store_replays_with_new_rows():
    s = Store(4, 16, [3, 20], [1, 1])
    caches = [torch.from_numpy(c).cuda() for c, _ in s.pools]
    scales = [torch.from_numpy(c).float().cuda() for _, c in s.pools]
    x, tables, cu = [t.cuda() for t in s.x], i32(s.tables), i32(s.cu)
    lens = i32(s.after)
    held = [tuple(p) for p in s.pools]
    args = (*x, *caches, *scales, tables, cu, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.store_kvcache_fp8_block(*args)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.store_kvcache_fp8_block(*args)
    after = list(s.after)
    held = [store_reference(t, *h, s.tables, s.cu, after) for t, h in zip(s.x, held)]
    for step in range(8):
        new = [(normal((2, 4, 128), 50 + 2 * step + i).float() * (1 + step)).to(torch.bfloat16) for i in range(2)]
        after = [after[0] + 1, after[1] + (1 if after[1] < 32 else 0)]
        for dst, src in zip(x, new):
            dst.copy_(src)
        lens.copy_(i32(after))
        g.replay()
        held = [store_reference(t, *h, s.tables, s.cu, after) for t, h in zip(new, held)]
        for i in range(2):
            assert np.array_equal(caches[i].cpu().numpy(), held[i][0])
            assert np.array_equal(scales[i].double().cpu().numpy(), held[i][1])
    assert pkv.get_device_errors() == 0


def test_store_of_many_short_sequences_and_empty_ones():
    rng = np.random.default_rng(4)
    new = [int(n) for n in rng.integers(0, 4, 700)]
    before = [int(n) for n in rng.integers(0, 20, 700)]
    Store(2, 8, before, new).check()
    Store(1, 16, [0] * 40 + [7], [0] * 40 + [33]).check()
