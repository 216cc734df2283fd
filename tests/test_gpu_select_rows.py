"""The selection of packed rows (sa_select_rows) against the canonical scores
step by step in 32 bits and a sort, entry for entry."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z

pytestmark = pytest.mark.gpu


def _rows(rows, prefix, Hq, Hk, seed=0, **kw):
    """Rows without pools that matter: the selection reads summaries alone."""
    r = R.Rows([0] * len(rows), [0] * len(rows), Hq, Hk, seed=seed)
    r.rows, r.prefix = list(rows), list(prefix)
    lead, extra = kw.get("lead", 0), kw.get("extra", 0)
    r.n_rows = lead + sum(rows) + extra
    g = torch.Generator(device="cuda").manual_seed(seed)
    r.q = torch.randn(r.n_rows, Hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    r.offsets = torch.tensor(np.concatenate([[0], np.cumsum(rows)]) + lead, dtype=torch.int32, device="cuda")
    lens = [a + n for a, n in zip(prefix, rows)]
    r.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    r.mpp = kw.get("mpp") or max(1, max(-(-n // 16) for n in lens))
    return r


def _summaries(prob, seed=0, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    x = torch.randn(prob.summary_shape(), generator=g, device="cuda")
    if kind == "coarse":           # few different values: many scores are equal
        x = x.sign()
    if kind == "equal":
        x = torch.ones_like(x)
    if prob.mode == sa.SUMMARY_MINMAX:
        lo, hi = x.amin(3, keepdim=True), x.amax(3, keepdim=True)
        x = torch.cat([lo, hi], 3)
    return x.to(torch.bfloat16).contiguous()


def _run(r, prob, summ, status=sa.SA_OK, ws=None):
    ws = ws or sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    ws.buf[256:].fill_(255)
    idx = torch.full((r.n_rows, r.Hq, prob.kcap), -7, dtype=torch.int32, device="cuda")
    cnt = torch.full((r.n_rows, r.Hq), -7, dtype=torch.int32, device="cuda")
    sa.select_rows(prob, r.q, summ, r.lens, r.offsets, idx, cnt, ws)
    torch.cuda.synchronize()
    assert ws.status() == status
    return idx, cnt


def _check(r, prob, summ, **kw):
    idx, cnt = _run(r, prob, summ, **kw)
    want = Z.select(r, prob, summ)
    i, c = idx.cpu().numpy(), cnt.cpu().numpy()
    for (row, h), w in want.items():
        assert c[row, h] == len(w), (row, h)
        assert i[row, h, :len(w)].tolist() == w, (row, h)
        assert (i[row, h, len(w):] == -7).all()
    mine = R.owned(r).numpy()
    assert (i[~mine] == -7).all() and (c[~mine] == -7).all(), "rows of nobody were written"
    return idx, cnt


HEADS = [(8, 2), (28, 4), (8, 1), (4, 4), (12, 4), (5, 1), (12, 2)]


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_ragged(Hq, Hk, mode, group):
    r = _rows([40, 1, 0, 9], [300, 5000, 20, 1200], Hq, Hk, seed=Hq)
    bs = [(16, 8, 64, 32)[h % 4] for h in range(Hk)]
    k = [5] * Hq if group else [(h * 3) % 11 for h in range(Hq)]
    prob = Z.problem(r, bs, k, 4, 64, mode=mode, selection=sa.SELECT_GROUP if group else sa.SELECT_PER_HEAD)
    _check(r, prob, _summaries(prob, Hq))


@pytest.mark.parametrize("kind", ["coarse", "equal"])
@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
def test_ties_go_to_the_lowest(kind, mode):
    r = _rows([20], [3000], 8, 2, seed=3)
    if kind == "coarse":
        r.q.sign_()
    prob = Z.problem(r, [8, 16], 37, 4, 64, mode=mode)
    _check(r, prob, _summaries(prob, 3, kind))


@pytest.mark.parametrize("S,W", [(0, 64), (1, 64), (63, 64), (64, 65), (200, 300)])
@pytest.mark.parametrize("bs", [8, 64])
def test_candidates(S, W, bs):
    r = _rows([150, 3], [230, 600], 8, 2, seed=S)
    prob = Z.problem(r, bs, 3, S, W)
    _check(r, prob, _summaries(prob, 4))


@pytest.mark.parametrize("k", [0, 1, 2, 31, 32, 33, 63, 64, 200, 1000])
def test_budgets(k):
    r = _rows([5], [2000], 4, 2, seed=k)
    prob = Z.problem(r, 16, k, 4, 64)
    _check(r, prob, _summaries(prob, 5))


def test_long():
    r = _rows([2, 3], [150000, 70000], 4, 1, seed=6)
    prob = Z.problem(r, 8, 700, 4, 1024)
    _check(r, prob, _summaries(prob, 6))
    r = _rows([600], [8000], 4, 1, seed=7)
    prob = Z.problem(r, 16, 24, 4, 256, mode=sa.SUMMARY_MEAN)
    _check(r, prob, _summaries(prob, 7))


def test_more_than_the_scratch_holds():
    # the longest lists of candidates there may be: the scores of 32 items at a time
    r = _rows([2, 2, 2, 2, 2, 2], [520000, 3000, 900, 100, 3000, 400000], 8, 8, seed=50, mpp=32768)
    prob = Z.problem(r, 8, 17, 4, 64, mode=sa.SUMMARY_MEAN)
    assert prob.block_slots() == 65536
    g = torch.Generator(device="cuda").manual_seed(51)
    summ = torch.empty(prob.summary_shape(), dtype=torch.bfloat16, device="cuda")
    for b in range(6):
        summ[b] = torch.randn(summ[b].shape, generator=g, device="cuda").to(torch.bfloat16)
    _check(r, prob, summ)


def test_close_scores():
    # scores that differ in the last bits: the order of their sums decides
    r = _rows([64], [4000], 8, 2, seed=8)
    prob = Z.problem(r, 16, 20, 4, 64, mode=sa.SUMMARY_MEAN)
    summ = _summaries(prob, 8)
    summ[:] = summ[:, :, :1]
    perm = torch.randperm(128, generator=torch.Generator().manual_seed(1)).tolist()
    for j in range(0, summ.shape[2], 2):      # every other block with dims swapped in pairs and tiny changes
        summ[:, :, j, perm[j % 128]] *= 1 + 2.0 ** -7
    _check(r, prob, summ)


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
def test_values_at_the_ends(mode):
    # zeros of both signs, the largest and smallest values, infinite summaries
    r = _rows([24], [1000], 8, 2, seed=9)
    r.q[0] = 0.0
    r.q[1] = -0.0
    r.q[2, :, ::2] = 0
    r.q[3] = 0
    r.q[3, :, 5] = 3e38       # one product alone: infinities of both signs would make NaN
    r.q[4] *= 2.0 ** -100
    prob = Z.problem(r, [8, 16], 9, 4, 64, mode=mode)
    summ = _summaries(prob, 9)
    summ[0, 0, 3, ..., 5] = 3e38
    summ[0, 0, 7, ..., 5] = -3e38
    summ[0, 1, 5] *= 2.0 ** -60
    _check(r, prob, summ)
    # an infinity among blocks that rows with positive queries take first
    r.q.abs_().clamp_(min=0.125, max=4)
    summ = summ.clamp(-4, 4)
    (summ[0, 0, 11, 1] if mode == sa.SUMMARY_MINMAX else summ[0, 0, 11])[20] = float("inf")
    idx, cnt = _check(r, prob, summ)
    assert bool((idx[:, :4] == 11).any(-1).all())


def test_rows_of_nobody_and_rows_without_a_position():
    r = _rows([12, 5], [400, 300], 8, 2, seed=10, lead=5, extra=30)
    prob = Z.problem(r, 16, 4, 4, 64)
    _check(r, prob, _summaries(prob, 10))
    r = _rows([300], [0], 8, 2, seed=11)
    r.lens[0] = 270
    prob = Z.problem(r, 16, 4, 4, 64)
    idx, cnt = _check(r, prob, _summaries(prob, 11))
    assert bool((cnt[:30] == 0).all())


def test_behind_the_table():
    r = _rows([40], [700], 8, 2, seed=12, mpp=40)
    prob = Z.problem(r, 16, 4, 4, 64)
    _check(r, prob, _summaries(prob, 12), status=sa.SA_ERR_CAPACITY)


# many rows a sequence: scores of the tensor cores first, canonical ones where they are close

@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("group", [False, True])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_many_rows(Hq, Hk, mode, group):
    r = _rows([260, 1, 0, 140], [900, 3000, 20, 5000], Hq, Hk, seed=Hq + 50)
    bs = [(16, 8, 64, 32)[h % 4] for h in range(Hk)]
    k = [5] * Hq if group else [(h * 3) % 23 for h in range(Hq)]
    prob = Z.problem(r, bs, k, 4, 64, mode=mode, selection=sa.SELECT_GROUP if group else sa.SELECT_PER_HEAD)
    _check(r, prob, _summaries(prob, Hq + 1))


@pytest.mark.parametrize("kind", ["coarse", "equal"])
@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("group", [False, True])
def test_many_rows_with_ties(kind, mode, group):
    r = _rows([100], [3000], 8, 2, seed=33)
    if kind == "coarse":
        r.q.sign_()
    prob = Z.problem(r, [8, 16], 37, 4, 64, mode=mode, selection=sa.SELECT_GROUP if group else sa.SELECT_PER_HEAD)
    _check(r, prob, _summaries(prob, 3, kind))


@pytest.mark.parametrize("k", [0, 1, 2, 31, 63, 100, 118, 119, 1000])
def test_many_rows_budgets(k):
    r = _rows([90], [1950], 4, 2, seed=k + 1)
    prob = Z.problem(r, 16, k, 4, 64)
    _check(r, prob, _summaries(prob, 5))


@pytest.mark.parametrize("eps", [2.0 ** -7, 2.0 ** -8, 0.0])
def test_many_rows_with_close_scores(eps):
    # neighbouring blocks differ by at most one step of bf16 in one dim, or not at all
    r = _rows([130], [4000], 8, 2, seed=38)
    prob = Z.problem(r, 16, 20, 4, 64, mode=sa.SUMMARY_MEAN)
    summ = _summaries(prob, 8)
    summ[:, :, 1::2] = summ[:, :, :-1:2] if summ.shape[2] % 2 == 0 else summ[:, :, :-1:2][:, :, :summ[:, :, 1::2].shape[2]]
    g = torch.Generator().manual_seed(1)
    for j in range(1, summ.shape[2], 2):
        summ[:, :, j, int(torch.randint(0, 128, (1,), generator=g))] *= 1 + eps
    _check(r, prob, summ)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
def test_many_rows_of_other_sizes(size):
    r = _rows([70], [2500], 8, 2, seed=39)
    prob = Z.problem(r, [8, 16], 13, 4, 64)
    summ = _summaries(prob, 9)
    r.q *= size
    _check(r, prob, summ)


def test_many_rows_with_infinities():
    # no bound for a KV head with an infinite summary, or for a row with an infinite query: these are scored as a whole
    r = _rows([70], [2500], 8, 2, seed=40)
    prob = Z.problem(r, [8, 16], 13, 4, 64)
    summ = _summaries(prob, 10)
    r.q.abs_().clamp_(min=0.125)
    summ[0, 1, 77, 1, 5] = float("inf")
    r.q[9, 2, 3] = float("inf")
    summ[0, 0, :, 1, 3] = summ[0, 0, :, 1, 3].abs().clamp(min=0.125)      # infinity times it is infinity: all are equal
    _check(r, prob, summ)


@pytest.mark.parametrize("size", [1.0, 1e-25, 1e-36])
@pytest.mark.parametrize("group", [False, True])
def test_many_rows_whose_products_cancel(size, group):
    # large products that cancel: what is left, and with it the order, is the rounding of the canonical sums
    r = _rows([96], [3000], 8, 2, seed=43)
    prob = Z.problem(r, 16, 12, 4, 64, mode=sa.SUMMARY_MEAN, selection=sa.SELECT_GROUP if group else sa.SELECT_PER_HEAD)
    summ = _summaries(prob, 13)
    big = torch.randn(64, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * 1000
    r.q[:] = r.q.sign() * 0 + 1
    r.q[:, :, 64:] = -1
    summ[:] = 0.001 * summ
    summ += torch.cat([big, big]).to(torch.bfloat16)
    r.q[::3] += (0.01 * torch.randn(r.q[::3].shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")).to(torch.bfloat16)
    r.q *= size
    _check(r, prob, summ)


def test_many_rows_at_once_and_captured():
    rs = [_rows([300, 200], [4000, 900], 8, 2, seed=44), _rows([400], [6000], 28, 4, seed=45)]
    probs = [Z.problem(rs[0], [16, 64], 20, 4, 64), Z.problem(rs[1], [64, 32, 16, 64], 9, 4, 128, mode=sa.SUMMARY_MEAN, selection=sa.SELECT_GROUP)]
    summs = [_summaries(p, 14 + i) for i, p in enumerate(probs)]
    want = [_check(r, p, s) for r, p, s in zip(rs, probs, summs)]
    wss = [sa.Workspace(p, rows=True, max_rows=r.n_rows) for r, p in zip(rs, probs)]
    got = [[torch.full_like(x, -7) for x in w] for w in want]
    streams = [torch.cuda.Stream() for _ in rs]
    torch.cuda.synchronize()
    for _ in range(10):
        for r, p, s, ws, g, st in zip(rs, probs, summs, wss, got, streams):
            with torch.cuda.stream(st):
                sa.select_rows(p, r.q, s, r.lens, r.offsets, *g, ws)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for r, p, s, ws, g in zip(rs, probs, summs, wss, got):
            sa.select_rows(p, r.q, s, r.lens, r.offsets, *g, ws)
    for g in got:
        for x in g:
            x.fill_(-7)
    for r in rs:
        r.q.neg_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for r, p, s, ws, g in zip(rs, probs, summs, wss, got):
        again = _check(r, p, s)
        assert torch.equal(again[0], g[0]) and torch.equal(again[1], g[1])
        assert ws.status() == sa.SA_OK


def test_many_candidates():
    r = _rows([70, 64], [30000, 12000], 8, 2, seed=41)
    prob = Z.problem(r, [16, 32], 100, 4, 512)
    _check(r, prob, _summaries(prob, 11))
    r = _rows([64], [16500], 8, 1, seed=42)
    prob = Z.problem(r, [8], 300, 0, 64, mode=sa.SUMMARY_MEAN)
    _check(r, prob, _summaries(prob, 12))


def test_many_sequences_and_replay():
    _many([(i * 5) % 4 for i in range(300)])
    _many([(i * 5) % 4 + (80 if i < 3 else 0) for i in range(5)])


def _many(rows):
    r = _rows(rows, [200 + (i * 37) % 900 for i in range(len(rows))], 4, 2, seed=13)
    prob = Z.problem(r, [16, 32], 6, 4, 64)
    summ = _summaries(prob, 13)
    idx, cnt = _check(r, prob, summ)
    ws = sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    i2, c2 = torch.full_like(idx, -7), torch.full_like(cnt, -7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.select_rows(prob, r.q, summ, r.lens, r.offsets, i2, c2, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(i2, idx) and torch.equal(c2, cnt)
