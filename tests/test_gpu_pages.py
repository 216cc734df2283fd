"""The pages' bookkeeping against the definitions, page by page: forks, frees,
truncation, growth, copy on write, packing, copies, accepted rows."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
P = 16


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _plan(table, parent, keep, lens, pages, Hk=2):
    B, mpp = table.shape
    prob = R.problem(B, Hk, Hk, mpp, pages)
    ws = sa.Workspace(prob, rows=True)
    out = torch.full((B, mpp), -9, dtype=torch.int32, device="cuda")
    src, dst, counts = _i32([-9] * B), _i32([-9] * B), _i32([-9, -9])
    sa.plan_pages(prob, _i32(table), _i32(parent), _i32(keep), _i32(lens), out, src, dst, counts, ws)
    torch.cuda.synchronize()
    want, copies, left = R.plan_pages(table, parent, keep, lens, pages)
    assert np.array_equal(out.cpu().numpy(), want)
    n = len(copies)
    assert counts.tolist() == [n, left]
    assert src.tolist() == [a for a, _ in copies] + [-1] * (B - n)
    assert dst.tolist() == [b for _, b in copies] + [-1] * (B - n)
    return ws.status(), want


def _random_table(rng, B, mpp, pages, lens, share=0.5):
    perm = rng.permutation(pages)
    at, table = 0, np.full((B, mpp), -1, np.int64)
    for b in range(B):
        n = -(-lens[b] // P)
        k = 0
        if b and rng.rand() < share:
            c = rng.randint(0, b)
            k = min(n, -(-lens[c] // P))
            k = rng.randint(0, k + 1)
            table[b, :k] = table[c, :k]
        table[b, k:n] = perm[at:at + n - k]
        at += n - k
    return table


@pytest.mark.parametrize("B,mpp", [(1, 1), (3, 5), (8, 40), (64, 33), (200, 300), (1024, 4)])
@pytest.mark.parametrize("seed", range(4))
def test_plan_random(B, mpp, seed):
    rng = np.random.RandomState(100 * seed + B)
    old = [int(rng.randint(0, mpp * P + 1)) for _ in range(B)]
    used = sum(-(-x // P) for x in old)
    pages = used + int(rng.randint(B, 3 * B + mpp * B + 2))
    table = _random_table(rng, B, mpp, pages, old)
    parent = [int(x) for x in rng.randint(-1, B, B)]
    keep = [0 if p < 0 else int(rng.choice([0, old[p], rng.randint(0, old[p] + 1), old[p] // P * P])) for p in parent]
    lens = [int(rng.choice([k, min(mpp * P, k + 1), rng.randint(k, mpp * P + 1), max(0, k - 3)])) for k in keep]
    status, _ = _plan(table, parent, keep, lens, pages)
    assert status in (sa.SA_OK, sa.SA_ERR_CAPACITY)


def test_plan_cases():
    # two beams go on from the same row: the lower keeps the tail page, the other copies
    t = np.array([[5, 3, -1], [2, -1, -1], [-1, -1, -1]])
    assert _plan(t, [0, 0, 1], [20, 20, 16], [21, 21, 17], 8)[0] == sa.SA_OK
    # a reader and a writer of the same tail: the writer copies, lowest or not
    assert _plan(t, [0, 0, -1], [20, 32, 0], [21, 32, 0], 8)[0] == sa.SA_OK
    # cut inside a page that another row holds whole
    assert _plan(t, [0, 0, -1], [32, 5, 0], [32, 6, 0], 8)[0] == sa.SA_OK
    # everything freed, then everything taken
    assert _plan(t, [-1, -1, -1], [0, 0, 0], [48, 48, 32], 8)[0] == sa.SA_OK
    # too few pages: the first rows get theirs
    assert _plan(t, [-1, -1, -1], [0, 0, 0], [48, 48, 48], 8)[0] == sa.SA_ERR_CAPACITY
    # a copy that finds no page
    assert _plan(t, [0, 0, 1], [20, 20, 16], [21, 21, 16], 3)[0] in (sa.SA_ERR_CAPACITY, sa.SA_ERR_BAD_PAGE)
    # the same row twice, nothing grows: shared, no copy
    status, out = _plan(t, [0, 0, 0], [20, 20, 7], [20, 20, 7], 8)
    assert status == sa.SA_OK and out[0, 0] == out[1, 0] == out[2, 0] == 5


def test_plan_refuses_on_the_device():
    t = np.array([[5, 3, -1], [2, 99, -1]])
    assert _plan(t, [2, 0], [3, 20], [4, 21], 8)[0] == sa.SA_ERR_INVALID_ARG     # no such parent
    assert _plan(t, [-2, 0], [3, 20], [4, 21], 8)[0] == sa.SA_ERR_INVALID_ARG
    assert _plan(t, [0, 0], [49, 20], [4, 21], 8)[0] == sa.SA_ERR_INVALID_ARG    # behind the table
    assert _plan(t, [0, 0], [-1, 20], [4, 21], 8)[0] == sa.SA_ERR_INVALID_ARG
    assert _plan(t, [0, 0], [20, 20], [49, 21], 8)[0] == sa.SA_ERR_INVALID_ARG
    assert _plan(t, [1, 0], [20, 20], [22, 21], 8)[0] == sa.SA_ERR_BAD_PAGE      # a kept page outside the pool
    assert _plan(t, [1, 0], [15, 20], [22, 21], 8)[0] == sa.SA_OK                # not kept: nobody looks


@pytest.mark.parametrize("B,mpp,slack", [(1, 1, 0), (4, 20, 7), (32, 50, 0), (32, 50, 3000), (128, 64, 9000), (600, 3, 1)])
@pytest.mark.parametrize("seed", range(3))
def test_compact_and_copy(B, mpp, slack, seed):
    rng = np.random.RandomState(7 * seed + B)
    lens = [int(rng.randint(0, mpp * P + 1)) for _ in range(B)]
    pages = max(1, sum(-(-x // P) for x in lens)) + slack
    table = _random_table(rng, B, mpp, pages, lens)
    Hk = 2
    prob = R.problem(B, Hk, Hk, mpp, pages)
    ws = sa.Workspace(prob, rows=True)
    out = torch.full((B, mpp), -9, dtype=torch.int32, device="cuda")
    src, dst, counts = _i32([-9] * pages), _i32([-9] * pages), _i32([-9, -9])
    sa.compact_pages(prob, _i32(table), _i32(lens), out, src, dst, counts, ws)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(pages, Hk, P, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    sa.copy_pages(prob, k, v, src, dst, counts, ws)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK
    want, moves, live = R.compact_pages(table, lens, pages)
    assert np.array_equal(out.cpu().numpy(), want)
    n = len(moves)
    assert counts.tolist() == [n, live]
    assert src.tolist() == [a for a, _ in moves] + [-1] * (pages - n)
    assert dst.tolist() == [b for _, b in moves] + [-1] * (pages - n)
    for a, b in moves:
        k0[b], v0[b] = k0[a], v0[a]
    assert torch.equal(k.view(torch.int16), k0.view(torch.int16)) and torch.equal(v.view(torch.int16), v0.view(torch.int16))


def test_compact_bad_rows():
    prob = R.problem(2, 2, 2, 3, 8)
    ws = sa.Workspace(prob, rows=True)
    t = np.array([[7, 9, -1], [2, 6, -1]])
    out, src, dst, counts = _i32(np.zeros((2, 3))), _i32([0] * 8), _i32([0] * 8), _i32([0, 0])
    sa.compact_pages(prob, _i32(t), _i32([20, 32]), out, src, dst, counts, ws)
    want, moves, live = R.compact_pages(t, [20, 32], 8)
    assert ws.status() == sa.SA_ERR_BAD_PAGE
    assert np.array_equal(out.cpu().numpy(), want) and counts.tolist() == [len(moves), live]
    sa.compact_pages(prob, _i32(t), _i32([-1, 49]), out, src, dst, counts, ws)
    assert ws.status() == sa.SA_ERR_INVALID_ARG
    assert bool((out == -1).all()) and counts.tolist() == [0, 0]


@pytest.mark.parametrize("Hk", [1, 2, 8])
@pytest.mark.parametrize("n", [0, 1, 5, 700])
def test_copy_pages(Hk, n):
    pages = 2 * n + 3
    rng = np.random.RandomState(n + Hk)
    perm = rng.permutation(pages)
    src, dst = perm[:n].astype(np.int64), perm[n:2 * n].astype(np.int64)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn(pages, Hk, P, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    k0[dst], v0[dst] = k0[src], v0[src]
    prob = R.problem(1, Hk, Hk, 1, pages)
    ws = sa.Workspace(prob, rows=True)
    tail = [pages + 5] * 3     # behind the count: not looked at
    sa.copy_pages(prob, k, v, _i32(list(src) + tail), _i32(list(dst) + tail), _i32([n]), ws)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK
    assert torch.equal(k.view(torch.int16), k0.view(torch.int16)) and torch.equal(v.view(torch.int16), v0.view(torch.int16))
    # a page that is not there is left out and recorded; a count above the list is cut to it
    sa.copy_pages(prob, k, v, _i32([pages, 0, -1]), _i32([0, pages, 1]), _i32([1000]), ws)
    assert ws.status() == sa.SA_ERR_BAD_PAGE
    sa.copy_pages(prob, k, v, _i32([0]), _i32([1]), _i32([-5]), ws)
    assert ws.status() == sa.SA_OK
    assert torch.equal(k.view(torch.int16), k0.view(torch.int16)) and torch.equal(v.view(torch.int16), v0.view(torch.int16))


@pytest.mark.parametrize("Hk", [1, 2, 8])
def test_accept_rows(Hk):
    base = [0, 15, 16, 37, 200, 5, 9]
    paths = [[0, 1, 2], [63], [0, 3, 7, 20, 41], list(range(64)), [], [5, 9, 9, 2], [1]]
    B, most, nodes = len(base), 64, 64
    r = R.Rows([nodes] * B, base, Hk, Hk, seed=3)
    path = np.zeros((B, most), np.int64) - 1
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    k, v = r.k_pool.clone(), r.v_pool.clone()
    ws = sa.Workspace(r.prob, rows=True)
    sa.accept_rows(r.prob, k, v, r.table, _i32(base), _i32(path), _i32([len(x) for x in paths]), ws)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK
    kr, vr = r.k_pool.clone(), r.v_pool.clone()
    t = r.table.cpu().numpy()
    for b, x in enumerate(paths):
        for i, node in enumerate(x):
            s, d = base[b] + node, base[b] + i
            kr[t[b, d // P], :, d % P] = r.k_pool[t[b, s // P], :, s % P]
            vr[t[b, d // P], :, d % P] = r.v_pool[t[b, s // P], :, s % P]
    assert torch.equal(k.view(torch.int16), kr.view(torch.int16)) and torch.equal(v.view(torch.int16), vr.view(torch.int16))


def test_accept_rows_refuses_on_the_device():
    r = R.Rows([16], [20], 2, 2, seed=4)
    ws = sa.Workspace(r.prob, rows=True)

    def go(base, path, cnt, table=None):
        k, v = r.k_pool.clone(), r.v_pool.clone()
        sa.accept_rows(r.prob, k, v, r.table if table is None else table, _i32([base]), _i32([path]), _i32([cnt]), ws)
        status = ws.status()
        assert torch.equal(k.view(torch.int16), r.k_pool.view(torch.int16))
        assert torch.equal(v.view(torch.int16), r.v_pool.view(torch.int16))
        return status

    assert go(20, [0, 2, 3], 4) == sa.SA_ERR_INVALID_ARG        # a count above the list's width
    assert go(20, [0, 2, 3], -1) == sa.SA_ERR_INVALID_ARG
    assert go(20, [0, -2, 3], 3) == sa.SA_ERR_INVALID_ARG
    assert go(20, [0, 28, 3], 3) == sa.SA_ERR_INVALID_ARG       # behind the table (48 tokens)
    assert go(-1, [0, 2, 3], 3) == sa.SA_ERR_INVALID_ARG
    assert go(47, [0, 0, 0], 3) == sa.SA_ERR_INVALID_ARG
    bad = r.table.clone()
    bad[0, 1] = 1000
    assert go(20, [0, 12, 13], 3, bad) == sa.SA_ERR_BAD_PAGE
    assert go(20, [0, 12, 13], 0, bad) == sa.SA_OK
