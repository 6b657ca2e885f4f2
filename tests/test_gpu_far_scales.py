"""Decode over the fp8 cache with block scales at the ends of the scales' range: products that leave
fp32's range only before all their factors are in, and values down to the smallest scale, to a relative
bound."""
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import HALF_BF16
from window_testutil import HALF_F16, Window

pytestmark = pytest.mark.gpu


def relative(w, got):
    """Every element to the roundings alone, with nothing fixed added: 2^-10 of the weighted sum of |V|
    for the scores and half a step of f16 for the weights; half a step of bf16 of the result; and
    for weights below f16's normal range half of its fixed step 2^-24, where a weight times the scale
    of its value is held relative to the largest such product, which stands at 2^7 or above: 2^-32 of that
    product for each token and unit of code (at most 448)."""
    ref, spread, _ = w.reference()
    small = torch.zeros_like(ref)
    for i, c in enumerate(w.ctx):
        sl = w.slots(i, range(c))
        k = w.rows_of(w.k_cache, w.k_scales, sl).repeat_interleave(w.hq // w.hkv, 1)
        vs = w.v_scales.double()[sl // w.bs].repeat_interleave(w.hq // w.hkv, 1)
        p = torch.softmax(torch.einsum("hd,xhd->hx", w.q[i].double(), k) * w.scale, -1) * vs.T
        small[i] = 2.0 ** -32 * 448 * c * p.amax(1)[:, None]
    bound = (HALF_F16 + 2.0 ** -10) * spread + HALF_BF16 * ref.abs() + small
    return ((got.double().cpu() - ref).abs() <= bound).all()


@pytest.mark.parametrize("bs", [16, 8, 6])
@pytest.mark.parametrize("e", [-120, -119, -113, -100, 60, 110])
@pytest.mark.parametrize("ctx", [[1, 5], [90, 17], [6000]], ids=str)
def test_values_of_one_far_scale(bs, e, ctx):
    """[6000] is cut over ranges, so that its records are merged."""
    w = Window(8, 2, bs, ctx, 0, 0, fp8=True, seed=5)
    w.v_scales[:] = 2.0 ** e
    got = w.call(pkv, w.device())
    assert got.isfinite().all() and relative(w, got)


def test_values_under_a_maximum_that_they_do_not_have():
    """The token of the largest score has the smallest scale and others far behind it large ones."""
    w = Window(2, 1, 16, [200], 0, 0, fp8=True, seed=6)
    w.q[:] = 1.0
    w.k_cache[:] = 0x38                                      # 1.0: scores 128 * scale of the block * 128^-0.5
    w.k_scales[:] = 2.0 ** -120
    w.v_scales[:] = 2.0 ** -120
    w.k_scales[int(w.tables[0, 3]), 0] = 4.0                 # 45: the others have weights of 2^-65
    w.v_scales[int(w.tables[0, 9]), 0] = 2.0 ** -60
    got = w.call(pkv, w.device())
    assert got.isfinite().all() and relative(w, got)


@pytest.mark.parametrize("bs", [16, 6])
@pytest.mark.parametrize("up,down", [(116, -120), (120, -120), (100, -104), (-104, 100), (-118, 114)])
def test_queries_and_keys_of_opposite_size(bs, up, down):
    """Keys all alike, so that every weight is the same: the output is the mean of the values however
    far the scores are from 0."""
    w = Window(4, 2, bs, [50, 17], 0, 0, fp8=True, seed=4)
    w.q[:] = 2.0 ** up
    w.k_cache[:] = 0x7E                                      # 448
    w.k_scales[:] = 2.0 ** down
    ref, spread, _ = w.reference()
    assert ref.isfinite().all()
    got = w.call(pkv, w.device())
    assert got.isfinite().all() and relative(w, got)


@pytest.mark.parametrize("bs", [16, 6])
def test_zero_keys_of_a_large_scale_under_large_queries(bs):
    """Scores of exactly 0 where query and scale alone leave fp32's range."""
    w = Window(4, 2, bs, [50, 17], 0, 0, fp8=True, seed=4)
    w.q[:] = 2.0 ** 120
    w.k_cache[:] = 0
    w.k_scales[:] = 2.0 ** 110
    got = w.call(pkv, w.device())
    assert got.isfinite().all() and relative(w, got)
