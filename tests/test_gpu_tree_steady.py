"""pkv_tree_decode where every CTA stays in one sequence for many key tiles: the MMA issuer's
two-steps-at-a-time loop, the rings going round several times inside a stream, and the way in
and out of both. Against 64-bit attention computed on the GPU from the same inputs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import HALF_BF16, Trees

pytestmark = pytest.mark.gpu


def reference(t, d, scale):
    """(out, spread) [rows, Hq, 128] float64 as Trees.reference, a sequence and head at a time."""
    n_rows, group = int(t.cu[-1]), t.hq // t.hkv
    out = torch.zeros((n_rows, t.hq, 128), dtype=torch.float64, device="cuda")
    spread = torch.zeros_like(out)
    for i, c in enumerate(t.ctx):
        a, b = int(t.cu[i]), int(t.cu[i + 1])
        p = np.arange(c)
        slots = torch.from_numpy(t.tables[i, p // t.bs] * t.bs + p % t.bs).cuda()
        k = torch.cat([d["k_cache"].flatten(0, 1)[slots], d["key"][a:b]])
        v = torch.cat([d["v_cache"].flatten(0, 1)[slots], d["value"][a:b]])
        hidden = torch.zeros((b - a, c + b - a), dtype=torch.bool, device="cuda")
        hidden[:, c:] = torch.from_numpy(~t.masks[i]).cuda()
        for g in range(t.hq):
            s = d["q"][a:b, g].double() @ k[:, g // group].double().T * scale
            w = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
            vg = v[:, g // group].double()
            out[a:b, g] = w @ vg
            spread[a:b, g] = w @ vg.abs()
    return out, spread


def longest_pieces(t):
    """Key tiles of each CTA's longest piece of one stream, by the documented division: the
    tiles of all streams, head by head, in one equal range a SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    group = t.hq // t.hkv
    streams = []
    for _ in range(t.hkv):
        for c, n in zip(t.ctx, t.sizes):
            tiles = -(-c // 128) + (0 if (c % 128 + 7) // 8 * 8 + n <= 128 else -(-n // 128))
            streams += [tiles] * -(-n * group // 256)
    edges = np.cumsum([0] + streams)
    units, longest = int(edges[-1]), []
    for b in range(sms):
        lo, hi = b * units // sms, (b + 1) * units // sms
        longest.append(int((np.minimum(edges[1:], hi) - np.maximum(edges[:-1], lo)).max()))
    return longest


def lengths(seed, n, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi, n).tolist()


CASES = [
    # hq, hkv, block, cached tokens, drafts, scale
    (32, 8, 16, lengths(1, 24, 2000, 5000), lengths(2, 24, 1, 33), None),       # one row tile
    (16, 8, 256, [4096, 3968, 4097, 4095, 4000, 4224] * 3, [16] * 18, None),    # whole last tiles and not
    (32, 8, 256, lengths(3, 14, 3000, 5000), [64] * 14, None),                  # two row tiles
    (32, 8, 16, lengths(4, 20, 2000, 4500), [64, 3, 40, 32, 33] * 4, None),     # both in one CTA
    (32, 8, 12, lengths(5, 20, 2000, 4500), [8, 64, 20, 50] * 5, None),         # gathered
    (4, 4, 1, lengths(6, 20, 3500, 5000), [100, 130, 1, 128, 200] * 4, None),   # one head a KV head
    (16, 1, 16, lengths(7, 10, 18000, 33000), [8, 16, 9, 3, 40] * 2, None),     # sixteen, row groups
    (32, 8, 16, lengths(8, 20, 2000, 4500), [20, 64] * 10, 0.5),                # maxima that grow often
    (32, 8, 16, lengths(9, 20, 2000, 4500), [20, 64] * 10, -0.2),               # the scores' sign turned
]


@pytest.mark.parametrize("hq,hkv,bs,ctx,sizes,scale", CASES)
def test_many_tiles_of_a_stream_in_a_cta(hq, hkv, bs, ctx, sizes, scale):
    t = Trees(hq, hkv, bs, ctx, sizes, seed=len(ctx) * 100 + bs)
    # a tile is one step, or two for two row tiles; the loop takes a piece's steps behind the
    # first four up to the last two, so pieces below eight steps never reach it
    assert np.median(longest_pieces(t)) >= 12
    d = t.device()
    scale = t.scale if scale is None else scale
    out = t.call(pkv, d, scale=scale)
    assert pkv.get_device_errors() == 0
    ref, spread = reference(t, d, scale)
    # the bound of assert_tree_close; the part of the scores' fp32 error grows with the scale
    err = (out.double() - ref).abs()
    grow = max(1.0, abs(scale) * 128 ** 0.5)
    assert bool((err <= HALF_BF16 * (spread + ref.abs()) + grow * 2.0 ** -10 * spread).all())
    assert torch.equal(out, t.call(pkv, d, scale=scale))
