"""sa_shared_prefixes records what is wrong with a sequence's offsets or length
whether it is of a group or not; a page outside the pool ends a prefix."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests.test_gpu_shared import Shared, _i32

pytestmark = pytest.mark.gpu


def _status(r):
    ws = sa.Workspace(r.prob, rows=True)
    members, prefix = (torch.full((r.B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sa.shared_prefixes(r.prob, r.table, r.lens, r.offsets, r.group_offsets, members, prefix, ws)
    torch.cuda.synchronize()
    return ws.status(), members.tolist(), prefix.tolist()


@pytest.mark.parametrize("groups", [[2, 4], [0], [0, 0], [4, 6], [0, 6]])
@pytest.mark.parametrize("b", [0, 3, 5])
def test_a_length_behind_the_table(groups, b):
    r = Shared([(6, 9)], [1] * 6, [4] * 6, 1, 1, seed=1)
    r.group_offsets = _i32(groups)
    good = _status(r)
    assert good[0] == sa.SA_OK
    r.lens[b] = r.mpp * 16 + 1
    assert _status(r) == (sa.SA_ERR_CAPACITY, *good[1:])


@pytest.mark.parametrize("groups", [[2, 4], [0], [0, 6]])
@pytest.mark.parametrize("b", [0, 3, 5])
def test_row_offsets_that_decrease(groups, b):
    r = Shared([(6, 9)], [2] * 6, [4] * 6, 1, 1, seed=2)
    r.group_offsets = _i32(groups)
    r.offsets[b + 1] = int(r.offsets[b]) - 1
    assert _status(r)[0] == sa.SA_ERR_INVALID_ARG


def test_a_page_outside_the_pool_ends_a_prefix():
    r = Shared([(3, 9)], [1] * 3, [4] * 3, 1, 1, seed=3)
    r.table[:, 5] = 2 ** 30
    assert _status(r) == (sa.SA_OK, [3, 0, 0], [80] * 3)
