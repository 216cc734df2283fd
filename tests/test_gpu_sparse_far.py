"""Attention over selected blocks at the ends of int32 (sa_sparse_row_attention):
lengths near 2^31 behind a short table, under windows as wide, and rows ahead of
the cache under them."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 - 1


def _check(r, prob, status):
    idx, cnt = Z.lists(r, prob, seed=1)
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
    return out


@pytest.mark.parametrize("S", [0, 5, FAR])
@pytest.mark.parametrize("W", [64, 2 ** 30, 2 ** 30 + 1, FAR - 60, FAR - 300, FAR])
@pytest.mark.parametrize("L", [FAR, 2 ** 30 + 77, FAR - 9])
def test_lengths_and_windows_near_the_largest(L, W, S):
    r = R.Rows([40, 3], [600, 700], 8, 2, seed=3, mpp=35)
    prob = Z.problem(r, [16, 32], 5, S, W)
    r.lens[0] = L
    _check(r, prob, sa.SA_ERR_CAPACITY)


@pytest.mark.parametrize("W", [64, FAR])
@pytest.mark.parametrize("n,L", [(70, 3), (200, 150), (33, 0)])
def test_rows_ahead_of_the_cache(n, L, W):
    r = R.Rows([n, 5], [0, 300], 8, 2, seed=4)
    prob = Z.problem(r, 16, 5, 4, W)
    r.lens[0] = L
    out = _check(r, prob, sa.SA_OK)
    assert bool((out[:n - L] == 0).all())
