"""What a plan records is decided by the pages: a shortage where there is one
and nothing where there is none; the copies of a short plan."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_pages import _i32, _plan, _random_table

pytestmark = pytest.mark.gpu
P = 16


@pytest.mark.parametrize("B,mpp", [(1, 1), (3, 5), (8, 40), (64, 33), (200, 30), (1024, 4)])
@pytest.mark.parametrize("more", [-3, -1, 0, 1, 7])
def test_a_shortage_is_recorded_and_nothing_else(B, mpp, more):
    rng = np.random.RandomState(B + mpp)
    old = [int(rng.randint(0, mpp * P + 1)) for _ in range(B)]
    used = sum(-(-x // P) for x in old)
    table = _random_table(rng, B, mpp, used, old)
    parent = [int(x) for x in rng.randint(-1, B, B)]
    keep = [0 if p < 0 else int(rng.randint(0, old[p] + 1)) for p in parent]
    lens = [int(rng.choice([k, min(mpp * P, k + 1), rng.randint(k, mpp * P + 1)])) for k in keep]
    lens[0] = mpp * P
    # a pool of exactly what the plan needs, and some more or fewer
    big = used + B * (mpp + 1)
    pages = big - R.plan_pages(table, parent, keep, lens, big)[2] + more
    if pages < max(1, used):
        table[table >= max(1, pages)] = 0         # another table of this smaller pool: needs are counted again below
        pages = max(1, pages)
    left = R.plan_pages(table, parent, keep, lens, pages)[2]
    kept_bad = any(p >= 0 and (table[p, :-(-k // P)] < 0).any() for p, k in zip(parent, keep))
    assert not kept_bad
    assert _plan(table, parent, keep, lens, pages)[0] == (sa.SA_ERR_CAPACITY if left < 0 else sa.SA_OK)


def test_the_copies_of_a_short_plan():
    # two beams on one tail page, a third row that takes the last page: the copy finds none
    t = np.array([[0, 1, -1], [2, -1, -1], [-1, -1, -1]])
    status, want = _plan(t, [0, 0, 1], [20, 20, 16], [21, 21, 16], 3)
    assert status == sa.SA_ERR_CAPACITY and want[1, 1] == -1
    prob = R.problem(3, 2, 2, 3, 3)
    ws = sa.Workspace(prob, rows=True)
    out, src, dst, counts = _i32(np.zeros((3, 3))), _i32([0] * 3), _i32([0] * 3), _i32([0, 0])
    sa.plan_pages(prob, _i32(t), _i32([0, 0, 1]), _i32([20, 20, 16]), _i32([21, 21, 16]), out, src, dst, counts, ws)
    assert ws.status() == sa.SA_ERR_CAPACITY and counts.tolist() == [1, -1]
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(3, 2, P, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    sa.copy_pages(prob, k, v, src, dst, counts, ws)
    assert ws.status() == sa.SA_ERR_BAD_PAGE      # its target is -1: left out
    assert torch.equal(k, k0) and torch.equal(v, v0)
