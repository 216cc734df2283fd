"""Norm, rotation and append of packed rows (sa_qk_norm_rope) against the
formulas in 64 bits: rows of any length, one row a sequence, strided slices,
pairings, axes, partial rotations, far and negative positions, in place, and
what must stay untouched."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
D, P = 128, 16


def _reference(x, w, pairs, layout, pos, freq, eps):
    """(value, tolerance): one rounding to bf16; before it fp32 sums of 128
    squares, a reciprocal root, sines off by 2^-21 (an angle to 2^-32 of a
    turn, its fp32 form to 2^-24 of half a turn) and a handful of products."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    mag = x.abs()
    y, size = x.clone(), mag.clone()
    r = sum(pairs)
    if r:
        axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).to(x.device)
        ang = (pos.double()[axis].t() * freq.double()[None])[:, None]
        i = torch.arange(r, device=x.device)
        a, b = (i, i + r) if layout == sa.ROPE_HALVES else (2 * i, 2 * i + 1)
        y[..., a] = x[..., a] * torch.cos(ang) - x[..., b] * torch.sin(ang)
        y[..., b] = x[..., b] * torch.cos(ang) + x[..., a] * torch.sin(ang)
        size[..., a] = size[..., b] = mag[..., a] + mag[..., b]
    return y, R.BF16 * y.abs() + 2.0 ** -18 * size + 1e-30


def _run(r: R.Rows, n, slices, pairs, layout, pos, norm, seed=0, eps=1e-5, in_place=False, ws=None, default_pos=False):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed + 77)
    Hq, Hk = r.Hq, r.Hk
    if slices:
        width = (Hq + 2 * Hk) * D + slices
        qkv = torch.randn(n, width, generator=g, device=dev).to(torch.bfloat16)
        q = qkv[:, :Hq * D].view(n, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D)
        v = qkv[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(n, Hk, D)
    else:
        q, k, v = (torch.randn(n, h, D, generator=g, device=dev).to(torch.bfloat16) for h in (Hq, Hk, Hk))
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if norm & b else None for b in (1, 2))
    rope = sa.Rope(pairs, layout) if pairs else None
    freq = torch.tensor([10000.0 ** (-j / max(1, sum(pairs))) for j in range(sum(pairs))], device=dev) if pairs else None
    q0 = q.clone()
    q_out = q if in_place else torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    kp, vp = r.k_pool.clone(), r.v_pool.clone()
    ws = ws or sa.Workspace(r.prob, rows=True)
    sa.qk_norm_rope(r.prob, q, k, v, r.offsets, r.lens, r.table, q_out, kp, vp, ws, rope=rope, inv_freq=freq,
                    positions=None if default_pos else pos, q_weight=qw, k_weight=kw, eps=eps)
    torch.cuda.synchronize()
    want, tol = _reference(q0, qw, pairs, layout, pos, freq, eps)
    mine = R.owned(r)
    R.assert_within(q_out[mine.cuda()], want[mine.cuda()], tol[mine.cuda()], "q")
    if not in_place and not bool(mine.all()):
        assert bool((q_out[~mine.cuda()] == 7.0).all()), "rows of nobody were written"
    wk, tk = _reference(k, kw, pairs, layout, pos, freq, eps)
    kr, vr = r.k_pool.double(), r.v_pool.clone()
    tol_k = torch.zeros_like(kr)
    for b in range(r.B):
        for i in range(r.rows[b]):
            t, row = r.prefix[b] + i, int(r.offsets[b]) + i
            if t < 0 or t >= r.mpp * P:
                continue
            page = int(r.table[b, t // P])
            if not 0 <= page < kp.shape[0]:
                continue
            kr[page, :, t % P], tol_k[page, :, t % P] = wk[row], tk[row]
            vr[page, :, t % P] = v[row]
    R.assert_within(kp, kr, tol_k, "k pool")
    assert torch.equal(vp.view(torch.int16), vr.view(torch.int16)), "v pool"
    return ws.status()


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4), (8, 8), (8, 1), (32, 8), (1, 1)])
@pytest.mark.parametrize("rows,prefix", [([1], [0]), ([1, 1, 1], [4095, 15, 16]), ([5, 0, 17, 33], [3, 9, 0, 100]), ([129], [7])])
def test_rows_and_heads(Hq, Hk, rows, prefix):
    r = R.Rows(rows, prefix, Hq, Hk, seed=1)
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(prefix, rows)]).to(torch.int32).cuda()[None].contiguous()
    for norm, layout, default in ((3, sa.ROPE_HALVES, True), (0, sa.ROPE_PAIRS, False)):
        assert _run(r, r.n_rows, 8, [64], layout, pos, norm, default_pos=default) == sa.SA_OK


@pytest.mark.parametrize("pairs", [[64], [32], [8], [16], [56], [16, 24, 24], [8, 0, 56], [20, 12, 16, 8], []])
@pytest.mark.parametrize("layout", [sa.ROPE_HALVES, sa.ROPE_PAIRS])
@pytest.mark.parametrize("norm", [0, 1, 2, 3])
def test_pairs_axes_and_norms(pairs, layout, norm):
    r = R.Rows([6, 1, 20], [11, 0, 40], 8, 2, seed=2)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(-3000, 200000, (max(1, len(pairs)), r.n_rows), generator=g).to(torch.int32).cuda()
    assert _run(r, r.n_rows, 0, pairs, layout, pos, norm) == sa.SA_OK


def test_far_positions_lose_nothing():
    r = R.Rows([8], [0], 8, 2, seed=3)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 6, 123456789, -1, 0, 1]], dtype=torch.int32).cuda()
    # the reduction's own error at 2^31: the frequency in turns is held to 2^-53 relative, 2^31 / 2 pi turns to 2^-25 of one
    assert _run(r, 8, 0, [64], sa.ROPE_HALVES, pos, 0) == sa.SA_OK


def test_in_place_strided_by_one_and_rows_of_nobody():
    r = R.Rows([7, 3], [1, 30], 8, 2, seed=4, extra_rows=5, lead=2)
    pos = torch.arange(r.n_rows, dtype=torch.int32).cuda()[None].contiguous()
    assert _run(r, r.n_rows, 0, [64], sa.ROPE_HALVES, pos, 3) == sa.SA_OK
    r = R.Rows([7, 3], [1, 30], 8, 2, seed=4)
    assert _run(r, r.n_rows, 0, [64], sa.ROPE_HALVES, pos[:, :10].contiguous(), 3, in_place=True) == sa.SA_OK


def test_no_rows():
    r = R.Rows([0, 0], [5, 0], 8, 2)
    assert _run(r, 0, 0, [64], sa.ROPE_HALVES, torch.zeros(1, 0, dtype=torch.int32).cuda(), 3) == sa.SA_OK


def test_many_sequences_and_a_zero_row():
    rows = [(i * 7) % 4 for i in range(300)]
    r = R.Rows(rows, [(i * 13) % 50 for i in range(300)], 8, 2, seed=6)
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(r.prefix, rows)]).to(torch.int32).cuda()[None].contiguous()
    assert _run(r, r.n_rows, 8, [64], sa.ROPE_HALVES, pos, 3) == sa.SA_OK


def test_pages_and_positions_that_are_not_there():
    # a page outside the pool: its rows are not appended, everything else is
    r = R.Rows([40], [3], 8, 2, seed=7)
    r.table[0, 1] = r.k_pool.shape[0]
    r.table[0, 2] = -4
    pos = torch.arange(40, dtype=torch.int32).cuda()[None].contiguous()
    assert _run(r, 40, 0, [64], sa.ROPE_HALVES, pos, 3) == sa.SA_ERR_BAD_PAGE
    # a length behind the table: the rows that have no entry are left out
    r = R.Rows([20, 4], [20, 2], 8, 2, seed=8, mpp=2)
    pos = torch.arange(24, dtype=torch.int32).cuda()[None].contiguous()
    assert _run(r, 24, 0, [64], sa.ROPE_HALVES, pos, 3) == sa.SA_ERR_CAPACITY
    # more rows than tokens: the first have no position
    r = R.Rows([6], [0], 8, 2, seed=9)
    r.lens[0] = 4
    r.prefix[0] = -2
    assert _run(r, 6, 0, [64], sa.ROPE_HALVES, pos[:, :6].contiguous(), 3) == sa.SA_OK


def test_bad_offsets_are_cut():
    r = R.Rows([4, 4], [0, 0], 8, 2, seed=10)
    r.offsets = torch.tensor([0, 4, 100], dtype=torch.int32).cuda()
    q, k, v = (torch.randn(8, h, D).to(torch.bfloat16).cuda() for h in (8, 2, 2))
    ws = sa.Workspace(r.prob, rows=True)
    out = torch.zeros_like(q)
    sa.qk_norm_rope(r.prob, q, k, v, r.offsets, r.lens, r.table, out, r.k_pool, r.v_pool, ws)
    assert ws.status() == sa.SA_ERR_INVALID_ARG
    assert torch.equal(out, q)      # no norm, no rotation: copied
