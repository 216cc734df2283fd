"""Attention of packed rows over sinks, window and selected blocks
(sa_sparse_row_attention) against the formulas in 64 bits, and against
sa_sparse_decode a row at a time.  Pools are NaN wherever no token lies."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z

pytestmark = pytest.mark.gpu
P = 16


def _run(r, prob, idx, cnt, status=sa.SA_OK, ws=None, with_lse=True):
    ws = ws or sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    ws.buf[256:].fill_(255)      # scratch of an earlier call
    out = torch.full((r.n_rows, r.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((r.n_rows, r.Hq), 7.0, device="cuda") if with_lse else None
    sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == status
    return out, lse


def _check(r, prob, idx, cnt, **kw):
    out, lse = _run(r, prob, idx, cnt, **kw)
    ref = Z.attention(r, prob, idx, cnt)
    mine = R.owned(r).cuda()
    R.assert_within(out[mine], ref["out"][mine], ref["tol"][mine], "out")
    if lse is not None:
        R.assert_within(lse[mine], ref["lse"][mine], ref["tol_lse"][mine], "lse")
        assert bool((lse[~mine] == 7.0).all())
    assert bool((out[~mine] == 7.0).all()), "rows of nobody were written"
    return out, lse


def _case(rows, prefix, Hq, Hk, bs, k, S, W, seed=0, extra=0.0, **kw):
    r = R.Rows(rows, prefix, Hq, Hk, seed=seed, **kw)
    prob = Z.problem(r, bs, k, S, W)
    return (r, prob, *Z.lists(r, prob, seed, extra))


HEADS = [(8, 2), (28, 4), (8, 1), (8, 8), (12, 4), (5, 1)]


@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("S,W", [(0, 64), (4, 64), (16, 65), (37, 200), (8, 100)])
def test_one_sequence(bs, S, W):
    _check(*_case([200], [300], 8, 2, bs, 6, S, W, seed=bs + S))


@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_ragged(Hq, Hk):
    bs = [(8, 64, 16, 32)[h % 4] for h in range(Hk)]
    _check(*_case([100, 1, 0, 33, 7, 130], [0, 700, 50, 300, 1500, 128], Hq, Hk, bs, 9, 5, 70, seed=1))


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 64, 65, 127, 128])
@pytest.mark.parametrize("prefix", [0, 1, 63, 500, 4090])
def test_lengths(n, prefix):
    _check(*_case([n], [prefix], 8, 2, [16, 64], 5, 4, 64, seed=n + prefix))


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
def test_entries_that_are_ignored(Hq, Hk):
    _check(*_case([150, 20], [200, 3000], Hq, Hk, [8, 32, 64, 16][:Hk], 12, 20, 90, seed=3, extra=0.7))


def test_short_lists_and_counts():
    r, prob, idx, cnt = _case([64], [900], 8, 2, 16, 10, 4, 64, seed=4)
    cnt[5:20] = 0
    _check(r, prob, idx, cnt)
    cnt[20:25] = -3
    _check(r, prob, idx, cnt)
    idx[30:40] = torch.arange(10, device="cuda").int() + 3
    cnt[30:40] = 1000        # cut to what the list holds
    _check(r, prob, idx, cnt.clone())


def test_long_and_cut():
    # few rows over many blocks: the work of an item is cut over blocks
    _check(*_case([8, 3], [30000, 12000], 8, 2, 16, 200, 4, 1024, seed=5))
    _check(*_case([1], [60000], 8, 1, 64, 300, 4, 64, seed=6), with_lse=False)
    _check(*_case([30, 30], [9000, 5000], 28, 4, [64, 8, 16, 32], 40, 0, 500, seed=7))


def test_everything_selected_is_dense():
    r = R.Rows([170], [700], 8, 2, seed=8)
    prob = Z.problem(r, 32, 64, 4, 64)
    idx = torch.arange(64, dtype=torch.int32, device="cuda").expand(r.n_rows, 8, 64).contiguous()
    cnt = torch.full((r.n_rows, 8), 64, dtype=torch.int32, device="cuda")
    out, lse = _run(r, prob, idx, cnt)
    ref = R.attention(r)
    R.assert_within(out, ref["out"], ref["tol"], "out")
    R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


def test_window_of_everything():
    _check(*_case([100], [50], 8, 2, 16, 2, 0, 2 ** 31 - 1, seed=9))
    _check(*_case([100], [50], 8, 2, 16, 2, 2 ** 31 - 1, 64, seed=9))


def test_many_sequences():
    rows = [(i * 5) % 7 for i in range(150)]
    _check(*_case(rows, [(i * 37) % 400 for i in range(150)], 8, 2, [16, 8], 4, 4, 64, seed=10))


def test_many_items_taken_whole():
    # more items than eight a block: each block takes the next, and none is cut
    r, prob, idx, cnt = _case([1 + i % 3 for i in range(180)], [(i * 53) % 700 for i in range(180)], 8, 8, [16, 64, 8, 32] * 2, 5, 4, 64, seed=21)
    out, lse = _check(r, prob, idx, cnt)
    ws = sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    o, x = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, o, ws, lse=x)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(x, lse) and ws.status() == sa.SA_OK


def test_rows_of_nobody_and_rows_that_see_nothing():
    _check(*_case([40, 5], [100, 3], 8, 2, 16, 3, 4, 64, seed=11, extra_rows=21, lead=6))
    r, prob, idx, cnt = _case([40, 5], [0, 3], 8, 2, 16, 3, 4, 64, seed=12)
    r.lens[0] = 25
    out, lse = _check(r, prob, idx, cnt)
    assert bool((out[:15] == 0).all()) and bool(torch.isneginf(lse[:15]).all())


def test_table_too_short_and_bad_pages():
    r, prob, idx, cnt = _case([100], [500], 8, 2, 16, 8, 4, 64, seed=13, mpp=30)
    _check(r, prob, idx, cnt, status=sa.SA_ERR_CAPACITY)
    r, prob, idx, cnt = _case([100, 7], [500, 2000], 28, 4, 16, 8, 4, 64, seed=14)
    r.table[0, 3] = -1
    r.table[0, 33] = 2 ** 30
    r.table[1, 125] = r.k_pool.shape[0]
    _check(r, prob, idx, cnt, status=sa.SA_ERR_BAD_PAGE)


@pytest.mark.parametrize("long", [False, True])
def test_what_a_row_does_not_see_cannot_change_it(long):
    # values that only some rows of an item see: infinite and NaN V, NaN K
    r, prob, idx, cnt = _case([60, 4] if not long else [6, 4], [500, 900] if not long else [20000, 900], 8, 2, 16, 8, 4, 64, seed=15)
    want = Z.attention(r, prob, idx, cnt)
    page = int(idx[3, 1, 0]) if int(cnt[3, 1]) else 2
    r.v_pool[int(r.table[0, page]), 0, 4, 9] = float("inf")
    r.v_pool[int(r.table[0, 20]), 1, 7] = float("nan")
    r.k_pool[int(r.table[0, 17]), 1, 3, 5] = float("nan")
    out, lse = _run(r, prob, idx, cnt)
    # NaN in K: the formulas give NaN to rows that see it and leave the others
    kn = r.k_pool[int(r.table[0, 17]), 1, 3, 5].clone()
    r.k_pool[int(r.table[0, 17]), 1, 3, 5] = 0
    ref = Z.attention(r, prob, idx, cnt)
    n0 = int(r.offsets[1])
    p = int(r.lens[0]) - n0 + torch.arange(n0, device="cuda")
    t = 17 * 16 + 3
    sees = ((idx[:n0] == 17) & (torch.arange(prob.kcap, device="cuda") < cnt[:n0, :, None])).any(-1) & (t <= p)[:, None]
    sees |= ((t > p - 64) & (t <= p))[:, None]
    sees[:, :4] = False          # the other KV head
    assert bool(sees.any()) or long
    assert bool(torch.isnan(out[:n0][sees]).all()) and bool(torch.isnan(lse[:n0][sees]).all())
    keep = torch.ones(r.n_rows, 8, dtype=torch.bool, device="cuda")
    keep[:n0] = ~sees
    R.assert_within(out[keep], ref["out"][keep], ref["tol"][keep], "out")
    R.assert_within(lse[keep], ref["lse"][keep], ref["tol_lse"][keep], "lse")
    assert kn.isnan() and bool(torch.isfinite(want["out"]).all())


def test_as_the_decode_step_a_row_at_a_time():
    Hq, Hk, S, W = 8, 2, 4, 64
    r = R.Rows([9], [700], Hq, Hk, seed=16)
    r.k_pool.nan_to_num_(0), r.v_pool.nan_to_num_(0)
    r.table[r.table >= r.k_pool.shape[0]] = 0
    prob = Z.problem(r, [16, 32], 7, S, W)
    summ = torch.zeros(prob.summary_shape(), dtype=torch.bfloat16, device="cuda")
    ws = sa.Workspace(prob, rows=True, max_rows=9)
    sa.block_summarize(prob, r.k_pool, r.table, r.lens, summ, ws)
    idx = torch.full((9, Hq, 7), -5, dtype=torch.int32, device="cuda")
    cnt = torch.full((9, Hq), -5, dtype=torch.int32, device="cuda")
    sa.select_rows(prob, r.q, summ, r.lens, r.offsets, idx, cnt, ws)
    out, lse = _run(r, prob, idx, cnt, ws=ws)
    for i in range(9):
        L = torch.tensor([701 + i], dtype=torch.int32, device="cuda")
        si, sc = torch.full_like(idx[:1], -5), torch.full_like(cnt[:1], -5)
        o, z = torch.zeros(1, Hq, 128, device="cuda"), torch.zeros(1, Hq, device="cuda")
        s1 = torch.zeros_like(summ)
        sa.block_summarize(prob, r.k_pool, r.table, L, s1, ws)
        q = r.q[i:i + 1].contiguous()
        sa.select_topk(prob, q, s1, L, si, sc, ws)
        assert torch.equal(si[0], idx[i]) and torch.equal(sc[0], cnt[i])
        sa.sparse_decode(prob, q, r.k_pool, r.v_pool, r.table, L, si, sc, o, z, ws)
        ref = Z.attention(r, prob, idx, cnt)
        R.assert_within(out[i], o[0].double().cpu().cuda(), ref["tol"][i] + 2e-3, "out")
        R.assert_within(lse[i], z[0].double(), ref["tol_lse"][i] + 2e-3, "lse")


def test_the_same_bits_captured_and_on_two_streams():
    cs = [_case([200, 1, 40], [300, 9000, 2000], 28, 4, [16, 64, 8, 32], 20, 4, 128, seed=17),
          _case([8] * 5, [5000, 20000, 1, 77, 3000], 8, 2, 16, 60, 4, 256, seed=18)]
    want = [_run(*c) for c in cs]
    wss = [sa.Workspace(c[1], rows=True, max_rows=c[0].n_rows) for c in cs]
    got = [(torch.zeros_like(o), torch.zeros_like(x)) for o, x in want]

    def call(c, ws, o, x):
        r, prob, idx, cnt = c
        sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, o, ws, lse=x)

    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, (o, x), st in zip(cs, wss, got, streams):
            with torch.cuda.stream(st):
                call(c, ws, o, x)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # captured, and replayed on other lists
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cs[0], wss[0], *got[0])
    r, prob, idx, cnt = cs[0]
    i2, c2 = Z.lists(r, prob, seed=99)
    idx.copy_(i2), cnt.copy_(c2)
    graph.replay()
    torch.cuda.synchronize()
    ref = Z.attention(r, prob, idx, cnt)
    R.assert_within(got[0][0], ref["out"], ref["tol"], "out")
    assert wss[0].status() == sa.SA_OK


def test_room():
    r, prob, idx, cnt = _case([4], [100], 8, 2, 16, 2, 4, 64, seed=19)
    out = torch.zeros_like(r.q)
    for ws in (sa.Workspace(prob, rows=True), sa.Workspace(prob, rows=True, max_rows=3)):
        with pytest.raises(ValueError, match="max_rows"):
            sa.sparse_row_attention(prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, idx, cnt, out, ws)
        with pytest.raises(ValueError, match="max_rows"):
            sa.select_rows(prob, r.q, torch.zeros(prob.summary_shape(), dtype=torch.bfloat16, device="cuda"), r.lens, r.offsets, idx, cnt, ws)
