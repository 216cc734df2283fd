"""A value that a row sees counts wherever the cache is cut: an infinite one
shows in the result however small its weight is, as where one block takes the
whole cache."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_rows_attention import _run

pytestmark = pytest.mark.gpu
P = 16


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4), (64, 8)])
@pytest.mark.parametrize("L", [300, 3000, 20000])
def test_a_seen_infinity_is_not_lost(Hq, Hk, L):
    r = R.Rows([4], [L], Hq, Hk, seed=L + Hq)
    g = torch.Generator(device="cuda").manual_seed(1)
    way = torch.randn(Hk, 128, generator=g, device="cuda")
    r.q.copy_((way[:, None] + 0.1 * torch.randn(4, Hk, Hq // Hk, 128, generator=g, device="cuda")).reshape(4, Hq, 128))
    # token 250 scores about 113 more than the others: their weights are below the smallest fp32
    page = int(r.table[0, 250 // P])
    r.k_pool[page, :, 250 % P] = 10 * way
    first = int(r.table[0, 0])
    r.v_pool[first, :, 3, 5::16] = float("inf")
    out, lse = _run(r)
    assert not bool(torch.isfinite(out[..., 5::16]).any())
    r.v_pool[first, :, 3, 5::16] = 1.0
    ref = R.attention(r)
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[5::16] = False
    R.assert_within(out[..., rest], ref["out"][..., rest], ref["tol"][..., rest], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")
