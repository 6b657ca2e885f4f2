"""A block id outside the pool, in the decode and the prefill behind a window and in the decode over the
fp8 cache with block scales: reported, and its tokens count as zero keys and values, however the block
size lets the rows come in and whichever way a row is computed."""
import copy

import numpy as np
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32
from window_testutil import Window, assert_window_close

pytestmark = pytest.mark.gpu


def zeroed(w, i, j):
    """w's reference with entry j of sequence i at a block of zeros (a spare one of the pool)."""
    spare = next(b for b in range(w.num_blocks) if b not in w.tables)
    z = copy.copy(w)
    z.tables = w.tables.copy()
    z.tables[i, j] = spare
    z.k_cache, z.v_cache = w.k_cache.clone(), w.v_cache.clone()
    z.k_cache[spare] = 0
    z.v_cache[spare] = 0
    return z


@pytest.mark.parametrize("bs", [16, 8, 6, 1, 48])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bad", ["behind the pool", "negative"])
def test_decode(bs, fp8, bad):
    w = Window(8, 2, bs, [100, 40], 60, 2, fp8=fp8, seed=bs)
    d = w.device()
    j = 70 // bs                                             # seen: 0, 1 and 40 .. 99
    tables = w.tables.copy()
    tables[0, j] = w.num_blocks if bad == "behind the pool" else -3
    out = w.call(pkv, {**d, "block_tables": i32(tables)})
    assert pkv.get_device_errors() == 2
    assert_window_close(out, zeroed(w, 0, j))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("bs", [16, 6])
def test_decode_that_sees_nothing_else(fp8, bs):
    w = Window(4, 2, bs, [5, 30], 40, 0, fp8=fp8)
    d = w.device()
    tables = w.tables.copy()
    tables[0, 0] = w.num_blocks
    out = w.call(pkv, {**d, "block_tables": i32(tables)})
    assert pkv.get_device_errors() == 2
    assert_window_close(out, zeroed(w, 0, 0))
    assert (out[0] == 0).all()


@pytest.mark.parametrize("bs", [16, 256, 6, 1])
@pytest.mark.parametrize("again", [False, True], ids=["tiles alone", "rows computed again"])
def test_prefill(bs, again):
    w = Window(4, 2, bs, [420, 40], 60, 3, q_lens=[200, 40], seed=bs)
    if again:                                                # seen by rows 310 .. 369; rows beside them are computed again
        w.v_cache.view(-1, 2, 128)[w.slots(0, [310]), :, 6] = float("nan")
    d = w.device()
    j = (255 if bs == 256 else 290) // bs                    # tokens near 290 for small blocks, 0 .. 255 for large ones
    tables = w.tables.copy()
    tables[0, j] = w.num_blocks + 5
    out = w.call(pkv, {**d, "block_tables": i32(tables)})
    assert pkv.get_device_errors() == 2
    z = zeroed(w, 0, j)
    ref, spread, _ = z.reference()
    got = out.double().cpu()
    assert torch.equal(got.isnan(), ref.isnan()) and bool(ref.isnan().any()) == again
    fine = ~ref.isnan()
    bound = 2.0 ** -8 * (spread + ref.abs()) + 2.0 ** -10 * spread      # as in assert_window_close
    assert ((got - ref).abs()[fine] <= bound[fine]).all()
