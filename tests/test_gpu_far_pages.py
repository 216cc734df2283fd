"""Pools whose last pages lie more than 2^32 values behind their first: rows over
selected blocks and behind shared prefixes, all of whose pages are there."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z
from tests.test_gpu_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pools():
    # 8 KV heads: 2^18 pages are 2^32 values
    n = (1 << 18) + 4000
    yield [torch.zeros(n, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.empty_cache()


def _move(r, pools):
    """The rows' pages to the end of a large pool."""
    few = r.k_pool.shape[0]
    assert few <= 4000
    at = pools[0].shape[0] - few
    assert at * 8 * 16 * 128 >= 1 << 32
    for mine, theirs in zip((r.k_pool, r.v_pool), pools):
        theirs[at:] = mine
    r.table = torch.where((r.table >= 0) & (r.table < few), r.table + at, torch.full_like(r.table, -1))
    r.k_pool, r.v_pool = pools
    r.prob = R.problem(r.B, r.Hq, r.Hk, r.mpp, pools[0].shape[0])
    return r


def test_selected_blocks(pools):
    r = _move(R.Rows([70, 3, 1], [900, 20000, 17], 16, 8, seed=1), pools)
    prob = Z.problem(r, [8, 16, 32, 64] * 2, 9, 4, 64)
    idx, cnt = Z.lists(r, prob, 1)
    # a value that some rows see alone: their sums are made again from the pools
    r.v_pool[int(r.table[0, 55]), 3, 2, 9] = float("inf")
    ws = sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    out, lse = torch.zeros_like(r.q), torch.zeros(r.n_rows, 16, device="cuda")
    sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK
    ref = Z.attention(r, prob, idx, cnt)
    assert bool(torch.isinf(ref["out"]).any())
    R.assert_within(out, ref["out"], ref["tol"], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


@pytest.mark.parametrize("groups,rows", [([(3, 60), (2, 9)], [1, 5, 1, 30, 2]), ([(8, 11)] * 6, [1] * 48)])
def test_shared_prefixes(pools, groups, rows):
    # few sequences, and more of them than blocks: own tokens attended where the parts are joined
    r = _move(Shared(groups, rows, [(i * 37) % 150 for i in range(len(rows))], 16, 8, seed=2), pools)
    ws = sa.Workspace(r.prob, rows=True, max_rows=r.n_rows)
    members, prefix = (torch.zeros(r.B, dtype=torch.int32, device="cuda") for _ in range(2))
    out, lse = torch.zeros_like(r.q), torch.zeros(r.n_rows, 16, device="cuda")
    sa.shared_prefixes(r.prob, r.table, r.lens, r.offsets, r.group_offsets, members, prefix, ws)
    sa.shared_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, members, prefix, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK and bool((prefix > 0).all())
    ref = R.attention(r)
    R.assert_within(out, ref["out"], ref["tol"], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


@pytest.mark.parametrize("rows", [5, 2000])
def test_rows_of_nobody_alone(rows):
    # a batch without a row of its own: nothing is written
    r = R.Rows([0, 0, 0], [300, 0, 40], 8, 2, seed=3, extra_rows=rows)
    prob = Z.problem(r, 16, 5, 4, 64)
    ws = sa.Workspace(prob, rows=True, max_rows=rows)
    seven = lambda *s, **kw: torch.full(s, 7, device="cuda", **kw)  # noqa: E731
    idx, cnt = seven(rows, 8, 5, dtype=torch.int32), seven(rows, 8, dtype=torch.int32)
    out, lse = seven(rows, 8, 128, dtype=torch.bfloat16), seven(rows, 8, dtype=torch.float32)
    members, prefix = seven(3, dtype=torch.int32), seven(3, dtype=torch.int32)
    group_offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    sa.select_rows(prob, r.q, torch.zeros(prob.summary_shape(), dtype=torch.bfloat16, device="cuda"), r.lens, r.offsets, idx, cnt, ws)
    sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, out, ws, lse=lse)
    sa.shared_prefixes(prob, r.table, r.lens, r.offsets, group_offsets, members, prefix, ws)
    sa.shared_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, members, prefix, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK
    assert members.tolist() == prefix.tolist() == [0, 0, 0]
    for x in (idx, cnt, out, lse):
        assert bool((x == 7).all())
