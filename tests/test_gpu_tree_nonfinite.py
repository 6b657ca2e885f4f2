"""pkv_tree_decode on queries and keys that are not finite: what the softmax of the formula
gives in 64 bits, wherever the key tiles of a sequence are divided."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import HALF_BF16, Trees

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def check(t, out):
    """NaN exactly where the formula has it, and elsewhere the bound of assert_tree_close
    (nothing else of it changes: a NaN row takes no part in the others)."""
    ref, spread = t.reference()
    got = out[:ref.shape[0]].double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), \
        (int(torch.isnan(got).sum()), int(torch.isnan(ref).sum()))
    ok = ~torch.isnan(ref)
    bound = HALF_BF16 * (spread + ref.abs()) + 2.0 ** -10 * spread + 1e-30
    assert bool(((got - ref).abs() <= bound)[ok].all())


# one tile, the drafts in a tile of their own, a few tiles, a sequence cut over the GPU
CONTEXTS = [100, 128, 300, 9000]
# drafts: one row tile; two row tiles (over 32 rows of 4 query heads a KV head)
DRAFTS = [6, 40]


@pytest.mark.parametrize("drafts", DRAFTS)
@pytest.mark.parametrize("ctx", CONTEXTS)
def test_a_query_row_with_a_nan(ctx, drafts):
    t = Trees(8, 2, 16, [ctx, 50], [drafts, 3], seed=31)
    t.q[2, 1, 5] = NAN
    t.q[drafts - 1, 7] = NAN
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert bool(torch.isnan(out[2, 1]).all()) and bool(torch.isnan(out[drafts - 1, 7]).all())
    check(t, out)


@pytest.mark.parametrize("tree", ["chain", "star"])
@pytest.mark.parametrize("drafts", DRAFTS)
@pytest.mark.parametrize("ctx", CONTEXTS)
def test_a_seen_draft_whose_key_has_a_nan(ctx, drafts, tree):
    # beside finite drafts (every later row of the chain) or alone in its tile (one row of
    # the star, from 128 cached tokens on); rows 0 .. 2 do not see it
    mask = {"chain": lambda n: np.tril(np.ones((n, n), bool)), "star": lambda n: np.eye(n, dtype=bool)}
    t = Trees(8, 2, 16, [ctx, 50], [drafts, 3], seed=32, masks=[mask[tree](n) for n in (drafts, 3)])
    t.key[3, 1, 77] = NAN
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert bool(torch.isnan(out[3:drafts if tree == "chain" else 4, 4:]).all())
    check(t, out)


@pytest.mark.parametrize("drafts", DRAFTS)
@pytest.mark.parametrize("first,last", [(0, 128), (128, 256), (4992, 5000), (0, 9000), (3000, 6000)])
def test_a_run_of_cached_keys_with_nans(first, last, drafts):
    # whole tiles, whole pieces, or some keys of one tile; the other sequence and the other
    # KV head see none of them
    t = Trees(8, 2, 16, [9000, 50], [drafts, 3], seed=33)
    p = np.arange(first, last)
    t.k_cache[t.tables[0, p // 16], p % 16, 0, 9] = NAN
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert bool(torch.isnan(out[:drafts, :4]).all())
    check(t, out)


@pytest.mark.parametrize("ctx", CONTEXTS)
def test_a_key_with_an_infinity(ctx):
    # scores of +inf (a NaN by the formula) and of -inf (a weight of 0), by the query's sign
    t = Trees(8, 2, 16, [ctx, 50], [6, 3], seed=34)
    t.k_cache[t.tables[0, 0], 3, 0, 9] = INF
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    check(t, out)


def test_a_nan_query_that_sees_nothing_is_zero():
    masks = [np.zeros((5, 5), bool), np.eye(3, dtype=bool)]
    t = Trees(8, 2, 16, [0, 300], [5, 3], seed=35, masks=masks)
    t.q[1] = NAN
    out = t.call(pkv, t.device())
    assert pkv.get_device_errors() == 0
    assert torch.count_nonzero(out[:5]) == 0
    check(t, out)


@pytest.mark.parametrize("bad", [NAN, -INF])
@pytest.mark.parametrize("bs", [16, 6])
@pytest.mark.parametrize("ctx", [0, 100, 300, 9000])
def test_values_of_drafts_that_two_row_tiles_do_not_see(ctx, bs, bad):
    # both warpgroups multiply the same V tile, whose odd rows nobody sees
    masks = []
    for n in (64, 33, 50):
        m = np.tril(np.ones((n, n), bool))
        m[:, 1::2] = False
        masks.append(m)
    t = Trees(8, 2, bs, [ctx, 50, 128], [64, 33, 50], seed=36, masks=masks)
    for a, b in zip(t.cu[:-1], t.cu[1:]):
        t.value[a + 1:b:2] = bad
    d = t.device()
    outs = [t.call(pkv, d) for _ in range(20)]
    assert pkv.get_device_errors() == 0
    check(t, outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("at", [0, 31, 32, 63])
def test_a_value_that_some_rows_of_two_row_tiles_see(at):
    # the rows of both row tiles that see the draft get its infinity, no others
    t = Trees(8, 2, 16, [300], [64], seed=37, masks=[np.tril(np.ones((64, 64), bool))])
    t.value[at, 1, 40] = INF
    d = t.device()
    outs = [t.call(pkv, d) for _ in range(20)]
    assert pkv.get_device_errors() == 0
    hit = torch.zeros(outs[0].shape, dtype=torch.bool)
    hit[at:, 4:, 40] = True
    out = outs[0].cpu()
    assert bool((out[hit] == INF).all()) and bool(torch.isfinite(out[~hit]).all())
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("ctx", [0, 20, 128, 300, 9000])
def test_rows_whose_scores_are_all_minus_infinity(ctx):
    # a softmax of nothing but -inf is NaN, a row that sees nothing is zero, and one finite
    # score takes all the weight
    masks = [np.tril(np.ones((6, 6), bool)), np.zeros((4, 4), bool), np.eye(3, dtype=bool)]
    masks[0][3] = False
    t = Trees(8, 2, 16, [ctx, 0, 300], [6, 4, 3], seed=38, masks=masks)
    t.q[:, :, 5] = t.q[:, :, 5].abs() + 0.125
    p = np.arange(ctx)
    t.k_cache[t.tables[0, p // 16], p % 16, :, 5] = -INF
    t.key[:5, :, 5] = -INF                       # but not draft 5, which row 5 sees
    d = t.device()
    d["tree_mask"][6:10] |= -1 << 4              # bits beyond the tree are nobody's
    out = t.call(pkv, d)
    assert pkv.get_device_errors() == 0
    nan = torch.isnan(out).flatten(1).all(1).tolist()
    assert nan[:6] == [True, True, True, ctx > 0, True, False]
    assert torch.count_nonzero(out[6:10]) == 0
    check(t, out)
