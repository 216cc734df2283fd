"""Attention of packed rows over the paged cache (sa_prompt_attention,
sa_tree_attention) against the formulas in 64 bits.  The pools are NaN wherever
no token of a sequence lies, so a look at a masked place shows."""
import math

import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
P = 16


def _run(r, words=None, ws=None, with_lse=True, status=sa.SA_OK):
    ws = ws or sa.Workspace(r.prob, rows=True)
    out = torch.full((r.n_rows, r.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((r.n_rows, r.Hq), 7.0, device="cuda") if with_lse else None
    if words is None:
        sa.prompt_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, out, ws, lse=lse)
    else:
        full = np.zeros(r.n_rows, np.uint64)
        full[int(r.offsets[0]):int(r.offsets[0]) + len(words)] = words
        mask = torch.from_numpy(full.view(np.int64)).cuda()
        sa.tree_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, mask, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert ws.status() == status
    return out, lse


def _check(r, words=None, **kw):
    out, lse = _run(r, words, **kw)
    ref = R.attention(r, words)
    mine = R.owned(r).cuda()
    R.assert_within(out[mine], ref["out"][mine], ref["tol"][mine], "out")
    if lse is not None:
        R.assert_within(lse[mine], ref["lse"][mine], ref["tol_lse"][mine], "lse")
        assert bool((lse[~mine] == 7.0).all())
    assert bool((out[~mine] == 7.0).all()), "rows of nobody were written"
    return out, lse


HEADS = [(8, 2), (28, 4), (8, 1), (8, 8), (12, 4), (5, 1), (12, 2)]


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (7, 1), (8, 1), (2, 2)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 300])
def test_prompt_one_sequence(Hq, Hk, n):
    _check(R.Rows([n], [0], Hq, Hk, seed=n))


@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_prompt_ragged(Hq, Hk):
    _check(R.Rows([200, 1, 0, 33, 97, 130], [0, 0, 50, 300, 17, 128], Hq, Hk, seed=1))


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 111, 127, 128, 1000, 4090])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_prompt_behind_a_prefix(prefix, n):
    _check(R.Rows([n], [prefix], 8, 2, seed=prefix + n))


def test_prompt_long():
    _check(R.Rows([2500, 700], [600, 0], 8, 2, seed=2))
    _check(R.Rows([1111, 3], [64, 9000], 28, 4, seed=3), with_lse=False)


def test_prompt_many_sequences():
    rows = [(i * 5) % 7 for i in range(150)]
    _check(R.Rows(rows, [(i * 37) % 400 for i in range(150)], 8, 2, seed=4))


def test_prompt_rows_that_see_nothing():
    # more rows than tokens: the first have no position and see nothing
    r = R.Rows([40, 5], [0, 3], 8, 2, seed=5)
    r.lens[0] = 25
    out, lse = _check(r)
    assert bool((out[:15] == 0).all()) and bool(torch.isneginf(lse[:15]).all())
    r = R.Rows([3, 4], [0, 0], 8, 2, seed=6)
    r.lens[:] = 0
    out, lse = _check(r)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_rows_of_nobody_and_no_rows():
    _check(R.Rows([20, 30], [5, 0], 8, 2, seed=7, lead=3, extra_rows=9))
    _check(R.Rows([0, 0], [5, 0], 8, 2, seed=7, extra_rows=4))
    r = R.Rows([0], [5], 8, 2, seed=7)
    _run(r)
    _run(r, np.zeros(0, np.uint64))


@pytest.mark.parametrize("Hq,Hk", HEADS)
@pytest.mark.parametrize("rows,prefix", [([1], [0]), ([1], [1]), ([16], [4080]), ([64, 1, 7], [200, 3000, 0]),
                                         ([33, 0, 64, 20], [130, 77, 0, 1029])])
def test_tree(Hq, Hk, rows, prefix):
    _check(R.Rows(rows, prefix, Hq, Hk, seed=8), R.tree_words(rows, 1))


def test_tree_any_words():
    # words without the row itself, empty words, bits behind the rows, all bits
    rows = [10, 64, 5]
    w = np.array([0, 1, 2, 3, 1 << 9, 1 << 10, (1 << 64) - 1, 5, 0, 1 << 63] + [(1 << 64) - 1, 0] * 32 + [0] * 5, dtype=np.uint64)
    r = R.Rows(rows, [0, 300, 0], 8, 2, seed=9)
    out, lse = _check(r, w)
    assert bool(torch.isneginf(lse[0]).all()) and bool((out[0] == 0).all())


def test_tree_is_the_causal_rows_for_a_chain():
    rows, prefix = [5, 64, 1, 30], [500, 20, 4000, 0]
    r = R.Rows(rows, prefix, 8, 2, seed=10)
    w = np.array([(1 << (i + 1)) - 1 for n in rows for i in range(n)], dtype=np.uint64)
    a, la = _run(r, w)
    b, lb = _run(r)
    ref = R.attention(r)
    R.assert_within(a, ref["out"], ref["tol"], "chain")
    R.assert_within(la, ref["lse"], ref["tol_lse"], "chain lse")
    R.assert_within(b, ref["out"], ref["tol"], "causal")


def test_tree_too_many_rows():
    r = R.Rows([65, 4], [10, 20], 8, 2, seed=11)
    words = R.tree_words([64, 1, 4], 2)
    out, lse = _run(r, words, status=sa.SA_ERR_CAPACITY)
    assert bool((out[:65] == 7.0).all()) and bool((lse[:65] == 7.0).all())
    ref = R.attention(r, words)
    R.assert_within(out[65:], ref["out"][65:], ref["tol"][65:], "out")


@pytest.mark.parametrize("kind", ["nan", "inf", "-inf", "mixed"])
def test_later_values_cannot_change_a_row(kind):
    # non-finite values at a position: rows before it stay exact, rows from it on carry them
    r = R.Rows([150, 20], [40, 3], 8, 2, seed=12)
    for b, t in ((0, 44), (0, 60), (0, 170), (1, 10)):
        page = int(r.table[b, t // P])
        v = {"nan": math.nan, "inf": math.inf, "-inf": -math.inf, "mixed": math.inf}[kind]
        r.v_pool[page, :, t % P, 5::7] = v
        if kind == "mixed" and t == 60:
            r.v_pool[page, :, t % P, 5::14] = -math.inf
    _check(r)
    words = R.tree_words([50, 20], 4)
    r = R.Rows([50, 20], [140, 3], 8, 2, seed=13)
    for b, t in ((0, 143), (0, 160), (0, 189), (1, 10)):
        r.v_pool[int(r.table[b, t // P]), :, t % P, 3::5] = math.nan if kind == "nan" else math.inf
    _check(r, words)


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
def test_later_values_over_a_split_cache(Hq, Hk):
    # the same where the item's KV range is cut over blocks, with one and two query tiles
    for rows, prefix in (([40, 7], [1500, 2000]), ([64], [3000])):
        r = R.Rows(rows, prefix, Hq, Hk, seed=25)
        words = R.tree_words(rows, 9)
        for b, n in enumerate(rows):
            for t in (prefix[b] + n // 2, prefix[b] + n - 1):
                r.v_pool[int(r.table[b, t // P]), :, t % P, 1::9] = math.inf
        _check(r)
        _check(r, words)


def test_later_keys_cannot_change_a_row():
    r = R.Rows([100], [30], 8, 2, seed=14)
    base, _ = _run(r)
    page = int(r.table[0, 100 // P])
    r.k_pool[page, :, 100 % P] = math.nan
    got, _ = _run(r)
    assert torch.equal(got[:70].view(torch.int16), base[:70].view(torch.int16))     # positions 30 .. 99
    assert bool(torch.isnan(got[70:]).all())


def test_large_scores_and_the_lowest_value():
    r = R.Rows([70], [100], 8, 2, seed=15)
    r.q.mul_(40)
    _check(r)
    # keys of the type's lowest value: scores of a few times 1e38, or infinite
    r = R.Rows([20], [0], 8, 2, seed=16)
    r.k_pool[int(r.table[0, 0]), :, 3] = -3.0e38
    r.q.abs_().mul_(0.001)
    _check(r)


def test_bad_pages_are_left_out():
    r = R.Rows([60, 40], [400, 0], 8, 2, seed=17)
    r.table[0, 3] = r.k_pool.shape[0]
    r.table[0, 26] = -1
    r.table[1, 1] = 2 ** 30
    _check(r, status=sa.SA_ERR_BAD_PAGE)
    _check(r, R.tree_words([60, 40], 5), status=sa.SA_ERR_BAD_PAGE)


def test_a_length_behind_the_table():
    r = R.Rows([30], [50], 8, 2, seed=18, mpp=4)
    _check(r, status=sa.SA_ERR_CAPACITY)
    _check(r, R.tree_words([30], 6), status=sa.SA_ERR_CAPACITY)
    # all rows behind the table: they see what the table has, and it ends inside a tile
    r = R.Rows([30, 9], [170, 300], 8, 2, seed=23, mpp=5)
    _check(r, status=sa.SA_ERR_CAPACITY)
    _check(r, R.tree_words([30, 9], 6), status=sa.SA_ERR_CAPACITY)


def test_tree_rows_that_are_more_than_the_tokens():
    r = R.Rows([20, 6], [0, 5], 8, 2, seed=24)
    r.lens[0] = 7
    _check(r, R.tree_words([20, 6], 8))


def test_bad_offsets_are_cut():
    r = R.Rows([10, 10], [20, 20], 8, 2, seed=19)
    ref = R.attention(r)
    r.offsets = torch.tensor([0, 10, 500], dtype=torch.int32).cuda()
    out, _ = _run(r, status=sa.SA_ERR_INVALID_ARG)
    R.assert_within(out, ref["out"], ref["tol"], "out")
    r.offsets = torch.tensor([0, 10, 5], dtype=torch.int32).cuda()
    out, _ = _run(r, status=sa.SA_ERR_INVALID_ARG)
    R.assert_within(out[:10], ref["out"][:10], ref["tol"][:10], "out")
    assert bool((out[10:] == 7.0).all())


def test_the_same_call_twice_gives_the_same_bits():
    r = R.Rows([500, 30, 1], [100, 5000, 9000], 28, 4, seed=20)
    ws = sa.Workspace(r.prob, rows=True)
    a, la = _run(r, ws=ws)
    b, lb = _run(r, ws=ws)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


def test_other_stream_and_graphs():
    # two captured graphs of two calls on one workspace, replayed in order, with new contents
    r = R.Rows([40, 3], [700, 90], 8, 2, seed=21)
    words = R.tree_words(r.rows, 7)
    mask = torch.from_numpy(words.view(np.int64)).cuda()
    ws = sa.Workspace(r.prob, rows=True)
    outs = [torch.zeros(r.n_rows, r.Hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros(r.n_rows, r.Hq, device="cuda") for _ in range(2)]
    calls = [lambda: sa.prompt_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, outs[0], ws, lse=lses[0]),
             lambda: sa.tree_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, mask, outs[1], ws, lse=lses[1])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
    side.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    for seed in (1, 2):
        r.q.copy_(torch.randn(r.q.shape, generator=torch.Generator().manual_seed(seed)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, w in ((0, None), (1, words)):
            ref = R.attention(r, w)
            R.assert_within(outs[i], ref["out"], ref["tol"], "out")
            R.assert_within(lses[i], ref["lse"], ref["tol_lse"], "lse")
    assert ws.status() == sa.SA_OK


def test_binding_refuses():
    r = R.Rows([4], [10], 8, 2, seed=26)
    out = torch.zeros_like(r.q)
    small, ws = sa.Workspace(r.prob), sa.Workspace(r.prob, rows=True)
    go = lambda **kw: sa.prompt_attention(**{**dict(prob=r.prob, q=r.q, k_pool=r.k_pool, v_pool=r.v_pool, page_table=r.table,  # noqa: E731
                                                    seq_lens=r.lens, row_offsets=r.offsets, out=out, ws=ws), **kw})
    go()
    with pytest.raises(ValueError, match="rows=True"):
        go(ws=small)
    with pytest.raises(TypeError):
        go(q=r.q.float())
    with pytest.raises(ValueError):
        go(out=out[:3])
    with pytest.raises(ValueError):
        go(row_offsets=r.offsets[:1])
    with pytest.raises(ValueError):
        go(q=torch.zeros(8, 4, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1))
    with pytest.raises(sa.SAError) as e:
        go(out=r.q)
    assert e.value.code == sa.SA_ERR_INVALID_ARG
    more = R.problem(1, 8, 2, r.mpp, r.k_pool.shape[0] + 1)     # a pool of more pages than the workspace is for
    with pytest.raises(ValueError, match="as many pages"):
        go(prob=more, k_pool=torch.zeros(more.num_pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda"),
           v_pool=torch.zeros(more.num_pages, 2, 16, 128, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_scale(scale):
    r = R.Rows([50], [60], 8, 2, seed=22)
    r.prob = R.problem(1, 8, 2, r.mpp, r.k_pool.shape[0], scale=scale)
    _check(r)
