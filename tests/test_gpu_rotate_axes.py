"""Rotations over several axes turn any number of dims: sections whose sum is
no multiple of eight, odd ones among them, with a lane's dims on both sides of
the middle and of the end."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_rotate import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [[20, 30], [1, 2], [1, 0], [0, 7], [4, 4, 4], [21, 22], [31, 32], [10, 10, 10, 33], [5, 8], [9, 0, 50]])
@pytest.mark.parametrize("layout", [sa.ROPE_HALVES, sa.ROPE_PAIRS])
@pytest.mark.parametrize("norm", [0, 1, 2, 3])
def test_sections_of_any_sum(pairs, layout, norm):
    r = R.Rows([6, 1, 20], [11, 0, 40], 8, 2, seed=2)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(-3000, 200000, (len(pairs), r.n_rows), generator=g).to(torch.int32).cuda()
    assert _run(r, r.n_rows, 0, pairs, layout, pos, norm) == sa.SA_OK


@pytest.mark.parametrize("Hq,Hk", [(32, 8), (5, 1), (7, 7)])
@pytest.mark.parametrize("layout", [sa.ROPE_HALVES, sa.ROPE_PAIRS])
def test_heads_and_slices(Hq, Hk, layout):
    r = R.Rows([3, 0, 130], [7, 9, 100], Hq, Hk, seed=3, lead=1, extra_rows=2)
    pos = torch.arange(2 * r.n_rows, dtype=torch.int32).cuda().view(2, -1)
    assert _run(r, r.n_rows, 8, [20, 30], layout, pos, 3) == sa.SA_OK


def test_in_place_and_what_does_not_turn():
    # dims from R on are scaled by the norm alone; an infinite one does not reach the others without a norm
    r = R.Rows([9], [4], 8, 2, seed=4)
    pos = torch.arange(2 * r.n_rows, dtype=torch.int32).cuda().view(2, -1)
    for layout in (sa.ROPE_HALVES, sa.ROPE_PAIRS):
        assert _run(r, 9, 0, [20, 30], layout, pos, 3, in_place=True) == sa.SA_OK
        q, k, v = (torch.ones(9, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))
        q[..., 100:] = float("inf")
        out, ws = torch.zeros_like(q), sa.Workspace(r.prob, rows=True)
        freq = torch.ones(50, device="cuda")
        sa.qk_norm_rope(r.prob, q, k, v, r.offsets, r.lens, r.table, out, r.k_pool, r.v_pool, ws,
                        rope=sa.Rope([20, 30], layout), inv_freq=freq, positions=pos)
        assert ws.status() == sa.SA_OK
        assert bool(torch.isfinite(out[..., :100]).all()) and bool(torch.isinf(out[..., 100:]).all())
