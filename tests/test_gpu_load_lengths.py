"""Read-back of sequences whose length does not fit their table: every row of theirs is left as it was,
and the length is reported whichever rows the call has."""
import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from draft_testutil import i32
from test_gpu_fp8_block import Load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", ["one over", "far over", "negative"])
@pytest.mark.parametrize("where", [0, 1, 2])
@pytest.mark.parametrize("rows", ["all", "up to the table's end", "none of it"])
def test_rows_of_a_bad_length_are_left(bad, where, rows):
    w = Load(2, 16, [40, 33, 20])
    cap = w.tables.shape[1] * 16
    w.tables = w.tables.copy()
    w.tables[where] = w.tables[where].max()                  # every entry a block of the pool
    a = w.args()
    lens = list(w.ctx)
    lens[where] = {"one over": cap + 1, "far over": 1 << 30, "negative": -1}[bad]
    a[5] = i32(lens)
    room = {"all": cap + 1, "up to the table's end": 24, "none of it": 0}[rows]
    starts, at = [], 0
    for i, c in enumerate(w.ctx):
        starts.append(at)
        at += room if i == where else c
    out = [torch.full((at, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkv.load_kvcache_fp8_block(*a, i32(starts), key_out=out[0], value_out=out[1])
    assert pkv.get_device_errors() == 4
    for which in range(2):
        want = torch.full((at, 2, 128), 7.0, dtype=torch.bfloat16)
        for i, c in enumerate(w.ctx):
            if i != where:
                want[starts[i]:starts[i] + c] = w.rows(which, i)
        assert torch.equal(out[which].cpu(), want)


def test_a_length_of_the_whole_table_is_fine():
    w = Load(2, 16, [40, 9])
    w.tables = w.tables[:, :3].copy()
    w.tables[1, 1:] = w.tables[1, 0]
    w.ctx = [40, 48]
    got = pkv.load_kvcache_fp8_block(*w.args(), i32([0, 40]), num_rows=88)
    for which in range(2):
        assert torch.equal(got[which].cpu(), torch.cat([w.rows(which, 0), w.rows(which, 1)]))
    assert pkv.get_device_errors() == 0
