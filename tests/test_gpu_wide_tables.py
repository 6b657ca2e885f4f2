"""Bounds beyond 32 bits in the windowed calls and the decode over the fp8 cache with block scales: tables
wide enough for more than 2^31 tokens, and explicit bounds past it."""
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32
from window_testutil import Window, assert_window_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1 << 31, (1 << 32) + 4096])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_over_a_table_for_more_than_2_31_tokens(tokens, fp8):
    bs = 4096
    w = Window(4, 2, bs, [5000], 4500, 3, fp8=fp8)
    d = w.device()
    wide = torch.full((1, tokens // bs), -1, dtype=torch.int32, device="cuda")
    wide[:, :w.tables.shape[1]] = d["block_tables"]
    out = w.call(pkv, {**d, "block_tables": wide}, max_context_len=None)
    assert pkv.get_device_errors() == 0
    assert_window_close(out, w)


@pytest.mark.parametrize("most", [1 << 31, (1 << 32) + 50, -(1 << 32) + 50])
def test_bounds_past_32_bits_are_refused(most):
    for fp8 in (False, True):
        w = Window(4, 2, 16, [40], 30, 3, fp8=fp8)
        with pytest.raises(pkv.PkvError):
            w.call(pkv, w.device(), max_context_len=most)
    w = Window(4, 2, 16, [40], 30, 3, q_lens=[9])
    d = w.device()
    for bounds in ((most, 40), (9, most)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_prefill_window(d["q"], d["k_cache"], d["v_cache"], d["cu_seqlens_q"], d["cu_seqlens_k"],
                                     d["block_tables"], w.scale, 30, 3, *bounds)
    assert pkv.get_device_errors() == 0


@pytest.mark.parametrize("over", [dict(window=-(1 << 32) + 9), dict(sinks=-(1 << 32) + 2)], ids=str)
def test_negative_windows_past_32_bits_are_refused(over):
    for fp8, q_lens in ((False, None), (True, None), (False, [9])):
        w = Window(4, 2, 16, [40], 30, 3, q_lens=q_lens, fp8=fp8)
        w.window, w.sinks = over.get("window", 30), over.get("sinks", 3)
        with pytest.raises(pkv.PkvError):
            w.call(pkv, w.device())
