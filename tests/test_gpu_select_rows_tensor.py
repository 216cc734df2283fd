"""The form of sa_select_rows that looks for a row's blocks with approximate
scores of the tensor cores and decides close ones by canonical scores: lists
entry for entry against the canonical scores step by step in 32 bits, at sizes
that take this form, and a look at which form ran."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z
from tests.test_gpu_select_rows import _rows, _summaries

pytestmark = pytest.mark.gpu
SHARED, EACH = sa.SELECT_GROUP, sa.SELECT_PER_HEAD


def _canonical(q, x, minmax):
    """[rows][blocks] canonical fp32 scores of query rows [rows][128]: eight lanes of 16 dims, each summed upwards (a
    product of two bf16 is exact in fp32, so a rounding an addition), joined 4, 2 and 1 apart."""
    out = []
    for q1 in q.split(max(1, (1 << 26) // (x.shape[0] * 128))):
        y = torch.where(q1[:, None] >= 0, x[None, :, 1], x[None, :, 0]) if minmax else x[None]
        t = (q1[:, None] * y).unflatten(-1, (8, 16))
        acc = t[..., 0].clone()
        for d in range(1, 16):
            acc = acc + t[..., d]
        acc = acc[..., :4] + acc[..., 4:]
        acc = acc[..., :2] + acc[..., 2:]
        out.append(acc[..., 0] + acc[..., 1] + 0.0)
    return torch.cat(out)


def _select(r, prob, summ):
    """(idx, cnt) of the rows with a sequence, -7 where nothing is written, by the definition."""
    dev = r.q.device
    idx = torch.full((r.n_rows, r.Hq, prob.kcap), -7, dtype=torch.int32, device=dev)
    cnt = torch.full((r.n_rows, r.Hq), -7, dtype=torch.int32, device=dev)
    minmax, shared = prob.mode == sa.SUMMARY_MINMAX, prob.selection == SHARED
    q, x = r.q.float(), summ.float()
    off, lens = r.offsets.tolist(), r.lens.tolist()
    for b in range(r.B):
        o0, o1 = off[b], off[b + 1]
        p = [lens[b] - (o1 - row) for row in range(o0, o1)]
        for kvh in range(r.Hk):
            span = [Z.candidates(prob, kvh, pos) for pos in p]
            j1 = max([e for _, e in span], default=0)
            if o0 == o1:
                continue
            at = torch.arange(j1, device=dev)
            lo, hi = (torch.tensor([s[i] for s in span], device=dev)[:, None] for i in range(2))
            there = (at >= lo) & (at < hi)
            total = None
            for g in range(r.G):
                h = kvh * r.G + g
                z = _canonical(q[o0:o1, h], x[b, kvh, :j1], minmax) if j1 > 0 else torch.zeros(o1 - o0, 0, device=dev)
                total = z if total is None else total + z
                if shared and g < r.G - 1:
                    continue
                assert not bool(torch.isnan(total if shared else z)[there].any())
                # those that are no candidates behind all others; equal ones in order
                order = torch.argsort(torch.where(there, -(total if shared else z), torch.full_like(z, float("nan"))), dim=1, stable=True)
                n = torch.minimum((hi - lo)[:, 0].clamp(min=0), torch.tensor(prob.k_per_head[h], device=dev))
                k = min(j1, prob.k_per_head[h])
                take = torch.where(torch.arange(k, device=dev) < n[:, None], order[:, :k], torch.full_like(order[:, :k], 1 << 30)).sort(1).values
                for y in range(r.G if shared else 1):
                    h1 = kvh * r.G + y if shared else h
                    idx[o0:o1, h1, :k] = torch.where(take < 1 << 30, take, torch.full_like(take, -7)).int()
                    cnt[o0:o1, h1] = n.int()
    return idx, cnt


def _check(r, prob, summ, tensor=True, status=sa.SA_OK):
    ws = sa.Workspace(prob, rows=True, max_rows=r.n_rows)
    ws.buf[256:].fill_(255)
    idx = torch.full((r.n_rows, r.Hq, prob.kcap), -7, dtype=torch.int32, device="cuda")
    cnt = torch.full((r.n_rows, r.Hq), -7, dtype=torch.int32, device="cuda")
    sa.select_rows(prob, r.q, summ, r.lens, r.offsets, idx, cnt, ws)
    torch.cuda.synchronize()
    assert ws.status() == status
    # the form with the tensor cores keeps the summaries' norms behind the header, the other one nothing
    norms = ws.buf[256:256 + 4 * r.B * r.Hk].view(torch.int32)
    assert bool((norms != -1).all()) if tensor else bool((norms == -1).all()), "the other form ran"
    want = _select(r, prob, summ)
    assert torch.equal(cnt, want[1])
    bad = (idx != want[0]).any(-1)
    assert not bool(bad.any()), f"{int(bad.sum())} lists differ, the first of row and head {torch.nonzero(bad)[0].tolist()}"
    return idx, cnt


def _problem(r, bs, k, S=4, W=64, mode=sa.SUMMARY_MINMAX, selection=EACH):
    return Z.problem(r, bs, k, S, W, mode=mode, selection=selection)


def test_the_definition_here_is_the_one_there():
    r = _rows([30, 0, 5], [700, 10, 2000], 8, 2, seed=1)
    for mode in (sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN):
        for selection in (EACH, SHARED):
            prob = _problem(r, [8, 32], 9, mode=mode, selection=selection)
            idx, cnt = _check(r, prob, _summaries(prob, 1), tensor=False)
            for (row, h), w in Z.select(r, prob, _summaries(prob, 1)).items():
                assert idx[row, h, :int(cnt[row, h])].tolist() == w


# query rows and heads for which this form takes less: 128 of them an item and a KV head
HEADS = [(8, 2, 1), (28, 4, 1), (8, 1, 1), (4, 4, 2), (12, 4, 1), (5, 1, 3), (12, 2, 1), (64, 8, 1)]


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("selection", [EACH, SHARED])
@pytest.mark.parametrize("Hq,Hk,times", HEADS)
def test_heads(Hq, Hk, times, selection, mode):
    r = _rows([900 * times, 1, 0, 1140 * times], [900, 3000, 20, 5000], Hq, Hk, seed=Hq + 50)
    bs = [(16, 8, 64, 32)[h % 4] for h in range(Hk)]
    k = [5] * Hq if selection == SHARED else [(h * 3) % 23 for h in range(Hq)]
    prob = _problem(r, bs, k, mode=mode, selection=selection)
    _check(r, prob, _summaries(prob, Hq + 1))


@pytest.mark.parametrize("kind", ["coarse", "equal"])
@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("selection", [EACH, SHARED])
def test_ties(kind, mode, selection):
    # more equal ones at the border than are scored one by one: rows scored again as a whole
    r = _rows([1400], [3000], 8, 2, seed=33)
    if kind == "coarse":
        r.q.sign_()
    prob = _problem(r, [8, 16], 37, mode=mode, selection=selection)
    _check(r, prob, _summaries(prob, 3, kind))


@pytest.mark.parametrize("k", [0, 1, 2, 31, 39, 40])
@pytest.mark.parametrize("prefix", [100, 1950, 6000])
def test_budgets(k, prefix):
    # candidates that all are kept, that lie in TMEM (256) and that go through the scratch
    r = _rows([2800], [prefix], 4, 2, seed=k + 1)
    prob = _problem(r, 16, k)
    _check(r, prob, _summaries(prob, 5))


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("k", [41, 63, 64, 100, 200])
@pytest.mark.parametrize("bs,prefix", [(64, 7000), (16, 6500), (8, 9000)])
def test_long_lists(k, mode, bs, prefix):
    r = _rows([2300], [prefix], 64, 8, seed=k)
    prob = _problem(r, bs, k, mode=mode, selection=SHARED)
    _check(r, prob, _summaries(prob, 6))


@pytest.mark.parametrize("kind", ["coarse", "equal"])
def test_long_lists_with_ties(kind):
    r = _rows([2300], [3000], 64, 8, seed=34)
    r.q.sign_()
    prob = _problem(r, 16, 70, selection=SHARED)
    _check(r, prob, _summaries(prob, 7, kind))


@pytest.mark.parametrize("eps", [2.0 ** -7, 2.0 ** -8, 0.0])
@pytest.mark.parametrize("selection,k,Hq,Hk", [(EACH, 20, 8, 2), (SHARED, 20, 8, 2), (SHARED, 50, 64, 8)])
def test_close_scores(eps, selection, k, Hq, Hk):
    # neighbouring blocks differ by at most one step of bf16 in one dim, or not at all
    r = _rows([1500 if Hq == 8 else 2300], [4000], Hq, Hk, seed=38)
    prob = _problem(r, 16, k, mode=sa.SUMMARY_MEAN, selection=selection)
    summ = _summaries(prob, 8)
    n = summ.shape[2] // 2
    summ[:, :, 1:2 * n:2] = summ[:, :, 0:2 * n:2]
    g = torch.Generator().manual_seed(1)
    for j in range(1, 2 * n, 2):
        summ[:, :, j, int(torch.randint(0, 128, (1,), generator=g))] *= 1 + eps
    _check(r, prob, summ)


@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e-12, 1e12, 1e30])
@pytest.mark.parametrize("selection", [EACH, SHARED])
def test_sizes_of_values(size, selection):
    r = _rows([1500], [2500], 8, 2, seed=39)
    prob = _problem(r, [8, 16], 13, selection=selection)
    summ = _summaries(prob, 9)
    r.q *= size
    _check(r, prob, summ)


@pytest.mark.parametrize("selection", [EACH, SHARED])
def test_infinities(selection):
    # no bound for a KV head with an infinite summary, or for a row with an infinite query: these are scored as a whole
    r = _rows([1500], [2500], 8, 2, seed=40)
    prob = _problem(r, [8, 16], 13, selection=selection)
    summ = _summaries(prob, 10)
    r.q.abs_().clamp_(min=0.125)
    summ[0, 1, 77, 1, 5] = float("inf")
    r.q[9, 2, 3] = r.q[700, 1, 3] = float("inf")
    summ[0, 0, :, 1, 3] = summ[0, 0, :, 1, 3].abs().clamp(min=0.125)      # infinity times it is infinity: all are equal
    _check(r, prob, summ)


@pytest.mark.parametrize("size", [1.0, 1e-25, 1e-36])
@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("selection,Hq,Hk", [(EACH, 8, 2), (SHARED, 8, 2), (SHARED, 16, 2)])
def test_products_that_cancel(size, mode, selection, Hq, Hk):
    # large products that cancel: what is left, and with it the order, is the rounding of the canonical sums.  Groups have
    # heads of both signs, so that the sum's positive and negative parts both are multiplied.
    r = _rows([1500], [3000], Hq, Hk, seed=43)
    prob = _problem(r, 16, 12, mode=mode, selection=selection)
    g = torch.Generator(device="cuda").manual_seed(2)
    summ = 0.001 * torch.randn(prob.summary_shape(), generator=g, device="cuda")
    big = 1000 * torch.randn(64, generator=g, device="cuda")
    summ = (summ + torch.cat([big, big])).to(torch.bfloat16)
    if mode == sa.SUMMARY_MINMAX:
        summ = torch.stack([summ.amin(3), summ.amax(3)], 3).contiguous()
    r.q[:] = 1
    r.q[:, :, 64:] = -1
    if selection == SHARED:
        r.q[:, 1::2] *= -1
    r.q[::3] += (0.01 * torch.randn(r.q[::3].shape, generator=g, device="cuda")).to(torch.bfloat16)
    r.q *= size
    _check(r, prob, summ)


@pytest.mark.parametrize("selection", [EACH, SHARED])
def test_rows_without_a_position_or_a_sequence(selection):
    r = _rows([1700], [0], 8, 2, seed=11, lead=3, extra=9)
    r.lens[0] = 1650
    prob = _problem(r, 16, 6, selection=selection)
    idx, cnt = _check(r, prob, _summaries(prob, 11))
    assert bool((cnt[3:53] == 0).all())


def test_behind_the_table():
    r = _rows([1500], [700], 8, 2, seed=12, mpp=70)
    prob = _problem(r, [16, 64], 6)
    _check(r, prob, _summaries(prob, 12), status=sa.SA_ERR_CAPACITY)


@pytest.mark.parametrize("selection", [EACH, SHARED])
def test_many_candidates(selection):
    r = _rows([700, 640, 300], [60000, 12000, 30], 8, 2, seed=41)
    prob = _problem(r, [16, 32], 40, W=512, selection=selection)
    _check(r, prob, _summaries(prob, 11))


def test_at_once_captured_and_on_other_values():
    rs = [_rows([900, 800], [4000, 900], 8, 2, seed=44), _rows([900], [6000], 28, 4, seed=45)]
    probs = [_problem(rs[0], [16, 64], 20), _problem(rs[1], [64, 32, 16, 64], 9, W=128, mode=sa.SUMMARY_MEAN, selection=SHARED)]
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
