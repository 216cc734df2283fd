"""Groups of sa_shared_prefixes whose offsets decrease: a group begins where those
before it have ended, so that every sequence has one answer, and rows attended
with it have theirs."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_shared import Shared, _i32, _run

pytestmark = pytest.mark.gpu


def _plan(r, status):
    ws = sa.Workspace(r.prob, rows=True)
    members, prefix = (torch.full((r.B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sa.shared_prefixes(r.prob, r.table, r.lens, r.offsets, r.group_offsets, members, prefix, ws)
    torch.cuda.synchronize()
    assert ws.status() == status
    return members, prefix


@pytest.mark.parametrize("offsets", [
    [0, 5, 3, 8], [0, 8, 3], [4, 1, 6], [0, 3, 3, 2, 8, 8], [8, 0], [0, 8, 0, 8, 0, 8], [-4, 2, -1, 5], [3, 20, 4], [7, 6, 5, 4, 3]])
def test_offsets_that_decrease(offsets):
    r = Shared([(4, 30), (4, 12)], [1, 2, 1, 1, 3, 1, 1, 2], [5, 0, 40, 17, 3, 8, 200, 1], 8, 2, seed=1)
    r.table[:, :6] = r.table[0, :6]             # the first pages are everybody's
    # what they say when each is cut to where the ones before it end
    cut = np.maximum.accumulate(np.clip(offsets, 0, r.B)).tolist()
    r.group_offsets = _i32(cut)
    want = _plan(r, sa.SA_OK)
    assert [x.tolist() for x in r.prefixes()] == [x.tolist() for x in want]
    r.group_offsets = _i32(offsets)
    for _ in range(3):
        plan = _plan(r, sa.SA_ERR_INVALID_ARG)
        assert torch.equal(plan[0], want[0]) and torch.equal(plan[1], want[1])
    out, lse = _run(r, plan=plan)
    ref = R.attention(r)
    R.assert_within(out, ref["out"], ref["tol"], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


def test_many_groups():
    # more groups than a block has threads, the last ones' offsets too small
    B = 700
    r = Shared([(1, 2)] * B, [1] * B, [i % 5 for i in range(B)], 1, 1, seed=2)
    r.table[:, :2] = r.table[0, :2]
    cut = list(range(0, B, 2)) + [B]
    r.group_offsets = _i32(cut)
    want = _plan(r, sa.SA_OK)
    assert want[0].tolist() == [2, 0] * (B // 2) and want[1].tolist() == [32] * B
    cut = cut[:300] + [7] * 50
    r.group_offsets = _i32(cut)
    got = _plan(r, sa.SA_ERR_INVALID_ARG)
    assert got[0].tolist() == [2, 0] * 299 + [0] * (B - 598) and got[1].tolist() == [32] * 598 + [0] * (B - 598)
