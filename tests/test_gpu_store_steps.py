"""Blocks of the fp8 cache with block scales that are filled a token at a time: codes and scales of K and
of V after every call, and against one call."""
import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32, normal
from test_gpu_fp8_block import Store
from window_testutil import store_reference

pytestmark = pytest.mark.gpu


def steps(full, x):
    """The rows of `full` a token a call; yields (caches, scales, held references) after each."""
    caches = [torch.from_numpy(c).cuda() for c, _ in full.pools]
    scales = [torch.from_numpy(s).float().cuda() for _, s in full.pools]
    held = [tuple(p) for p in full.pools]
    tables, xg = i32(full.tables), [t.cuda() for t in x]
    longest = max(full.after)
    for t in range(longest):
        rows = [r for r, a in enumerate(full.after) if t < a]
        at = [int(full.cu[r]) + t for r in rows]
        after = [t + 1] * len(rows)
        pkv.store_kvcache_fp8_block(xg[0][at], xg[1][at], *caches, *scales, tables[rows].contiguous(),
                                    i32(range(len(rows) + 1)), i32(after))
        held = [store_reference(s[at], *h, full.tables[rows], list(range(len(rows) + 1)), after)
                for s, h in zip(x, held)]
        yield caches, scales, held


@pytest.mark.parametrize("bs", [16, 7, 64])
@pytest.mark.parametrize("order", ["any", "growing"])
def test_every_step_is_exact(bs, order):
    full = Store(2, bs, [0, 0, 0], [40, 17, 70], seed=11)
    x = full.x
    if order == "growing":                                   # scales that grow in nearly every call
        x = [(t.float() * torch.exp2(torch.arange(t.shape[0]) % 37 - 18.0)[:, None, None]).to(torch.bfloat16) for t in x]
    for caches, scales, held in steps(full, x):
        for c, s, h in zip(caches, scales, held):
            assert np.array_equal(s.double().cpu().numpy(), h[1])
            assert np.array_equal(c.cpu().numpy(), h[0])
    assert pkv.get_device_errors() == 0


def test_largest_row_first_is_one_store():
    """Where each block's first row holds its largest value of every head, no scale grows behind it, and
    the codes of K and of V are those of one call."""
    full = Store(2, 16, [0, 0], [40, 17], seed=12, size=0.0)
    x = [t.clone() for t in full.x]
    for t in x:
        for r, n in enumerate(full.after):
            rows = t[full.cu[r]:full.cu[r] + n]
            for p in range(0, n, 16):
                rows[p, :, 0] = rows[p:p + 16].abs().amax((0, 2))
    whole_c, whole_s = full.check(x)
    for caches, scales, _ in steps(full, x):
        pass
    for i in range(2):
        live = full.tables[full.tables >= 0]
        assert np.array_equal(scales[i].double().cpu().numpy()[live], whole_s[i][live])
        assert np.array_equal(caches[i].cpu().numpy()[live], whole_c[i][live])
