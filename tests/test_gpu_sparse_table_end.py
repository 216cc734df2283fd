"""Attention over selected blocks where the page table ends inside a block
(sa_sparse_row_attention): rows behind the table, whose windows do not reach it
either, see of the block what the table holds, and nothing else enters."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z

pytestmark = pytest.mark.gpu


def _check(r, prob, idx, cnt, status):
    ws = sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    ws.buf[256:].fill_(255)
    out = torch.full((r.n_rows, r.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((r.n_rows, r.Hq), 7.0, device="cuda")
    sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == status
    ref = Z.attention(r, prob, idx, cnt)
    R.assert_within(out, ref["out"], ref["tol"], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


def _last_block(rows, prefix, Hq, Hk, bs, mpp, S, W, seed):
    """Every row's list ends with the block in which the table does."""
    r = R.Rows(rows, prefix, Hq, Hk, seed=seed, mpp=mpp)
    prob = Z.problem(r, bs, 6, S, W)
    last = (mpp * 16 - 1) // bs
    rng = np.random.RandomState(seed)
    idx = np.stack([np.append(np.sort(rng.choice(last, 5, replace=False)), last) for _ in range(r.n_rows * Hq)])
    idx = torch.from_numpy(idx.reshape(r.n_rows, Hq, 6)).int().cuda()
    return r, prob, idx, torch.full((r.n_rows, Hq), 6, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
@pytest.mark.parametrize("bs,mpp", [(64, 29), (64, 30), (64, 31), (32, 31), (64, 33), (64, 1001), (32, 1001)])
def test_behind_a_table_that_ends_inside_a_block(Hq, Hk, bs, mpp):
    # 64 + 64 tokens behind the table and more
    args = _last_block([70, 3], [mpp * 16 + 130, mpp * 16 + 500], Hq, Hk, bs, mpp, 4, 64, seed=mpp + bs)
    _check(*args, status=sa.SA_ERR_CAPACITY)


def test_around_the_end_of_such_a_table():
    # rows ahead of the end, at it, with it in their window, and behind
    args = _last_block([64, 64, 64, 200, 1], [400, 448, 479, 470, 2000], 8, 2, 64, 30, 5, 70, seed=3)
    _check(*args, status=sa.SA_ERR_CAPACITY)
