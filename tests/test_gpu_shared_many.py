"""Rows behind shared prefixes of more sequences than the attention kernel weighs in
shared memory (10239): against the formulas in 64 bits, all sequences at once."""
import math

import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
P, D = 16, 128


@pytest.mark.parametrize("B,most", [(10239, 40), (10240, 40), (10300, 40), (10300, 300)])
def test_more_sequences_than_shared_memory_holds(B, most):
    Hq, Hk, per, pages = 2, 1, 25, 3
    g = torch.Generator(device="cuda").manual_seed(B + most)
    groups = -(-B // per)
    b = torch.arange(B, device="cuda")
    n = 1 + (b % 7 == 3).long() - (b % 11 == 5).long()                # rows: one, two or none
    lens = pages * P + n + torch.randint(0, most, (B,), generator=g, device="cuda")
    mpp = -(-(pages * P + 2 + most) // P)
    own = mpp - pages
    table = torch.empty(B, mpp, dtype=torch.int32, device="cuda")
    table[:, :pages] = (b // per * pages)[:, None] + torch.arange(pages, device="cuda")
    table[:, pages:] = groups * pages + (b * own)[:, None] + torch.arange(own, device="cuda")
    pool = groups * pages + B * own
    k_pool, v_pool = (torch.randn(pool, Hk, P, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n.cumsum(0)]).int()
    rows = int(offsets[-1])
    q = torch.randn(rows, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
    group_offsets = torch.arange(0, groups + 1, device="cuda").mul(per).clamp(max=B).int()
    prob = R.problem(B, Hq, Hk, mpp, pool)
    ws = sa.Workspace(prob, rows=True, max_rows=rows)
    members, prefix = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    out, lse = torch.zeros_like(q), torch.zeros(rows, Hq, device="cuda")
    lens = lens.int()
    sa.shared_prefixes(prob, table, lens, offsets, group_offsets, members, prefix, ws)
    sa.shared_attention(prob, q, k_pool, v_pool, table, lens, offsets, members, prefix, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK and bool((prefix == pages * P).all())

    seq = torch.repeat_interleave(b, n)
    at = lens.long()[seq] - n[seq] + torch.arange(rows, device="cuda") - offsets.long()[seq]      # a row's position
    for r0 in range(0, rows, 1000):
        s, p = seq[r0:r0 + 1000], at[r0:r0 + 1000]
        k, v = (x[table[s].long(), 0].flatten(1, 2).double() for x in (k_pool, v_pool))           # [rows][tokens][D]
        q64 = q[r0:r0 + 1000].double()
        seen = (torch.arange(k.shape[1], device="cuda") <= p[:, None])[:, None]
        z = torch.einsum("rhd,rtd->rht", q64, k) * prob.scale
        z = torch.where(seen, z, torch.full_like(z, -math.inf))
        ref_lse = torch.logsumexp(z, -1)
        w = torch.exp(z - ref_lse[..., None])
        ref = torch.einsum("rht,rtd->rhd", w, v)
        # as rows_ref.attention: one rounding of the result and one of each weight to bf16, scores in fp32
        mag = (torch.einsum("rhd,rtd->rht", q64.abs(), k.abs()) * prob.scale * seen).amax(-1)
        dz = 128 * 2.0 ** -23 * mag + 2.0 ** -22 + 2.0 ** -22 * z.amax(-1).abs()
        A = torch.einsum("rht,rtd->rhd", w, v.abs())
        tol = R.BF16 * ref.abs() + (R.BF16 * 1.01 + 2 * dz[..., None]) * A + 1e-30
        R.assert_within(out[r0:r0 + 1000], ref, tol, "out")
        R.assert_within(lse[r0:r0 + 1000], ref_lse, dz + 2.0 ** -22 * ref_lse.abs() + k.shape[1] * 2.0 ** -24, "lse")
