"""Rows behind prefixes that groups of sequences share (sa_shared_prefixes,
sa_shared_attention): the prefixes against a walk over the table, the attention
against the formulas in 64 bits over each sequence's own row of the table."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
P = 16


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Shared(R.Rows):
    """Rows whose groups hold their first `pages` pages in common.  groups: (sequences, pages) of neighbours."""

    def __init__(self, groups, rows, own, Hq, Hk, seed=0, **kw):
        assert sum(m for m, _ in groups) == len(rows) == len(own)
        pages = [p for m, p in groups for _ in range(m)]
        super().__init__(rows, [p * P + o for p, o in zip(pages, own)], Hq, Hk, seed=seed, **kw)
        self.groups = [m for m, _ in groups]
        at = 0
        for m, p in groups:
            self.table[at + 1:at + m, :p] = self.table[at, :p]
            at += m
        self.group_offsets = _i32(np.concatenate([[0], np.cumsum(self.groups)]))

    def prefixes(self, min_tokens=0):
        """(members, prefix_lens) by the definition."""
        table, lens, off = self.table.cpu().numpy(), self.lens.cpu().numpy(), self.offsets.cpu().numpy()
        go, pool = self.group_offsets.cpu().numpy(), self.k_pool.shape[0]
        members, prefix = np.zeros(self.B, np.int64), np.zeros(self.B, np.int64)
        for b0, b1 in zip(go[:-1], go[1:]):
            some = [b for b in range(b0, b1) if off[b + 1] > off[b]]
            if len(some) < 2:
                continue
            n = min(max(0, int(lens[b]) - int(off[b + 1] - off[b])) // P for b in some)
            n = min(n, self.mpp)
            j = 0
            while j < n and all(table[b, j] == table[some[0], j] for b in some) and 0 <= table[some[0], j] < pool:
                j += 1
            if j * P < max(1, min_tokens):
                continue
            prefix[b0:b1] = j * P
            members[some[0]] = b1 - some[0]
        return members, prefix


def _plan(r, min_tokens=0, status=sa.SA_OK, ws=None):
    ws = ws or sa.Workspace(r.prob, rows=True)
    members, prefix = (torch.full((r.B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    sa.shared_prefixes(r.prob, r.table, r.lens, r.offsets, r.group_offsets, members, prefix, ws, min_tokens=min_tokens)
    torch.cuda.synchronize()
    assert ws.status() == status
    return members, prefix


def _check_plan(r, **kw):
    members, prefix = _plan(r, **kw)
    want = r.prefixes(kw.get("min_tokens", 0))
    assert members.tolist() == want[0].tolist()
    assert prefix.tolist() == want[1].tolist()
    return members, prefix


def _mask(r, words):
    full = np.zeros(r.n_rows, np.uint64)
    full[int(r.offsets[0]):int(r.offsets[0]) + len(words)] = words
    return torch.from_numpy(full.view(np.int64)).cuda()


def _run(r, words=None, plan=None, status=sa.SA_OK, ws=None, with_lse=True):
    members, prefix = plan if plan is not None else _check_plan(r)
    ws = ws or sa.Workspace(r.prob, rows=True, max_rows=r.n_rows)
    ws.buf[256:].fill_(255)     # scratch of an earlier call: NaN
    out = torch.full((r.n_rows, r.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((r.n_rows, r.Hq), 7.0, device="cuda") if with_lse else None
    sa.shared_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, members, prefix, out, ws, lse=lse,
                        tree_mask=None if words is None else _mask(r, words))
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


HEADS = [(8, 2), (28, 4), (8, 1), (8, 8), (12, 4), (5, 1)]


@pytest.mark.parametrize("Hq,Hk", HEADS)
@pytest.mark.parametrize("pages", [0, 1, 7, 8, 9, 100])
def test_single_tokens(Hq, Hk, pages):
    _check(Shared([(5, pages), (1, 3), (2, 17)], [1] * 8, [0, 5, 16, 200, 33, 7, 1, 140], Hq, Hk, seed=pages))


@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_trees(Hq, Hk):
    rows = [16, 1, 64, 33, 7, 0, 12, 5]
    r = Shared([(4, 20), (3, 60), (1, 5)], rows, [0, 3, 16, 77, 0, 9, 300, 1], Hq, Hk, seed=3)
    _check(r, R.tree_words(rows, 3))


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
def test_prompts_behind_a_prefix(Hq, Hk):
    _check(Shared([(3, 12), (2, 70)], [300, 41, 129, 64, 500], [0, 10, 130, 1, 16], Hq, Hk, seed=4))


def test_long_prefix_is_cut():
    # few rows over a long prefix: its tokens are cut over blocks, and so are some sequences' own
    _check(Shared([(4, 1250)], [1, 1, 1, 1], [20, 2500, 90, 5000], 8, 2, seed=5))
    _check(Shared([(3, 900), (2, 1100)], [8, 3, 16, 1, 1], [0, 700, 64, 3000, 5], 28, 4, seed=6), with_lse=False)


def test_large_groups():
    # rows of a group fill several items of the prefix
    _check(Shared([(150, 40)], [1] * 150, [(i * 13) % 90 for i in range(150)], 8, 2, seed=7))
    _check(Shared([(70, 9), (80, 30)], [1 + i % 3 for i in range(150)], [(i * 7) % 40 for i in range(150)], 16, 2, seed=8))


def test_nothing_shared():
    r = Shared([(1, 9), (1, 4), (1, 0)], [1, 5, 40], [3, 0, 12], 8, 2, seed=9)
    members, prefix = _check_plan(r)
    assert not bool(members.any()) and not bool(prefix.any())
    out, lse = _check(r)
    ws = sa.Workspace(r.prob, rows=True)
    same = torch.empty_like(out)
    sa.prompt_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, same, ws)
    R.assert_within(out, same.double(), 2 * R.BF16 * same.double().abs() + 1e-3, "against prompt_attention")


def test_sequences_without_rows():
    # a finished sequence in a group, its table gone, takes nothing from the others
    r = Shared([(5, 30), (3, 8)], [0, 1, 0, 1, 1, 1, 1, 0], [0, 5, 0, 9, 2, 0, 40, 0], 8, 2, seed=10)
    r.table[0], r.table[2], r.table[7] = -1, 2 ** 31 - 1, -1
    r.lens[0] = r.lens[2] = r.lens[7] = 0
    members, prefix = _check_plan(r)
    assert members.tolist() == [0, 4, 0, 0, 0, 3, 0, 0] and prefix.tolist() == [480] * 5 + [128] * 3
    _check(r)


def test_rows_of_nobody():
    _check(Shared([(3, 10)], [1, 2, 1], [4, 4, 4], 8, 2, seed=11, extra_rows=40, lead=9))


def test_large_batch():
    m = 330
    groups = [(i % 7 + 1, i % 11) for i in range(90)]
    n = sum(x for x, _ in groups)
    assert n > m
    _check(Shared(groups, [1 if i % 9 else 0 for i in range(n)], [(i * 31) % 50 for i in range(n)], 8, 2, seed=12))


def _many_few(Hq, Hk, seed, tree):
    """More sequences than blocks, few rows and mostly few tokens of their own: those are attended where the parts are joined."""
    B = -(-320 // Hk)
    rng = np.random.RandomState(seed)
    rows = [int(rng.choice((1, 1, 1, 2, 3, 4, 5, 0))) for _ in range(B)]
    rows[7] = 12
    own = [int(rng.randint(0, 190)) for _ in range(B)]
    own[:8] = [0, 156, 157, 159, 160, 161, 15, 3]
    groups, left = [], B
    while left:
        m = min(left, int(rng.randint(1, 40)))
        groups.append((m, int(rng.randint(0, 14))))
        left -= m
    r = Shared(groups, rows, own, Hq, Hk, seed=seed)
    assert r.n_rows <= 4 * B
    return r, R.tree_words(rows, seed) if tree else None


@pytest.mark.parametrize("Hq,Hk", [(2, 2), (4, 2), (6, 2), (8, 2), (10, 2), (12, 2), (14, 2), (16, 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_many_sequences_of_few_tokens(Hq, Hk, tree):
    r, words = _many_few(Hq, Hk, Hq, tree)
    _check(r, words)


def test_many_sequences_unseen_values_and_bad_pages():
    r, _ = _many_few(8, 2, 3, False)
    plan = _plan(r)
    two = [b for b in range(r.B) if r.rows[b] >= 2 and int(plan[1][b]) > 0 and int(r.lens[b]) - int(plan[1][b]) < 100]
    b, c, d = two[0], two[1], two[2]
    # the newest token is seen by the sequence's last row alone
    L = int(r.lens[b])
    r.v_pool[int(r.table[b, (L - 1) // P]), 0, (L - 1) % P, 9] = float("inf")
    L = int(r.lens[c])
    r.v_pool[int(r.table[c, (L - 1) // P]), 1, (L - 1) % P] = float("nan")
    out, lse = _check(r, plan=plan)
    assert bool(torch.isposinf(out[int(r.offsets[b + 1]) - 1, :4, 9]).all())
    assert bool(torch.isnan(out[int(r.offsets[c + 1]) - 1, 4:]).all())
    r.table[d, int(plan[1][d]) // P] = -1
    _check(r, plan=plan, status=sa.SA_ERR_BAD_PAGE)


def test_many_sequences_bits_and_replay():
    r, _ = _many_few(28, 4, 5, False)
    plan = _plan(r)
    out, lse = _run(r, plan=plan)
    ws = sa.Workspace(r.prob, rows=True, max_rows=r.n_rows)
    o, x = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.shared_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, *plan, o, ws, lse=x)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(x, lse)


def test_prefix_by_hand():
    # less than what is shared, and none for some: the result is the same attention
    r = Shared([(4, 40), (3, 25)], [1] * 7, [9, 0, 100, 31, 16, 2, 5], 8, 2, seed=13)
    for members, prefix in (([4, 0, 0, 0, 3, 0, 0], [640, 640, 640, 640, 16, 16, 16]), ([2, 0, 2, 0, 0, 0, 0], [320] * 2 + [128] * 2 + [0] * 3),
                            ([0] * 7, [0] * 7), ([1] * 7, [16] * 7), ([99, 0, 0, 0, 0, 0, 0], [16] * 4 + [16] * 3)):
        if members[0] == 99:      # more sequences than there are: up to the last
            r.table[4:, 0] = r.table[0, 0]
        _check(r, plan=(_i32(members), _i32(prefix)))


@pytest.mark.parametrize("bad", [-16, 8, 656, 2 ** 30])
def test_bad_prefix(bad):
    # no multiple of a page, negative or over the row itself: reported, and that sequence read on its own
    r = Shared([(2, 40)], [1, 1], [0, 5], 8, 2, seed=14)
    _check(r, plan=(_i32([0, 0]), _i32([bad, 0])), status=sa.SA_ERR_INVALID_ARG)


def test_too_many_drafts():
    rows = [4, 65, 3, 2]
    r = Shared([(4, 20)], rows, [0, 1, 2, 3], 8, 2, seed=15)
    words = np.concatenate([R.tree_words([4], 1), np.zeros(65, np.uint64), R.tree_words([3, 2], 2)])
    out, lse = _run(r, words, status=sa.SA_ERR_CAPACITY)
    assert bool((out[4:69] == 7.0).all()) and bool((lse[4:69] == 7.0).all())
    ref = R.attention(r, words)
    keep = torch.ones(r.n_rows, dtype=torch.bool, device="cuda")
    keep[4:69] = False
    R.assert_within(out[keep], ref["out"][keep], ref["tol"][keep], "out")


def test_what_nobody_sees_is_not_read():
    # a non-finite value that one sequence's rows do not see, and one in the prefix that all see
    r = Shared([(3, 11)], [1, 1, 1], [20, 3, 150], 8, 2, seed=16)
    r.v_pool[int(r.table[0, 2]), 0, 5, 17] = float("inf")
    r.v_pool[int(r.table[2, 13]), 1, 2, 40] = float("nan")
    r.k_pool[int(r.table[1, 11]), 1, 1] = float("nan")     # seen by sequence 1's second KV head: its result is NaN
    out, _ = _run(r)
    assert bool(torch.isposinf(out[:, :4, 17]).all())
    assert bool(torch.isnan(out[2, 4:, 40]).all()) and bool(torch.isfinite(out[2, 4:, 41:]).all())
    assert bool(torch.isfinite(out[0]).sum() == 8 * 128 - 4)
    assert bool(torch.isnan(out[1, 4:]).all())


def test_bad_page_in_the_prefix():
    r = Shared([(3, 20)], [1, 2, 1], [9, 0, 30], 8, 2, seed=17)
    plan = _plan(r)
    r.table[:, 4] = 2 ** 31 - 1
    _check(r, plan=plan, status=sa.SA_ERR_BAD_PAGE)
    members, prefix = _check_plan(r)
    assert prefix.tolist() == [64] * 3 and members.tolist() == [3, 0, 0]


@pytest.mark.parametrize("mpp", [None, 700])
def test_plan_finds_where_tables_part(mpp):
    rng = np.random.RandomState(1)
    groups = [(9, 300), (1, 40), (17, 257), (2, 600), (40, 3), (8, 0)]
    n = sum(m for m, _ in groups)
    r = Shared(groups, [int(rng.randint(0, 4)) for _ in range(n)], [int(rng.randint(0, 60)) for _ in range(n)], 1, 1, seed=18, mpp=mpp)
    _check_plan(r)
    for b, j in ((3, 299), (12, 256), (20, 0), (27, 1), (28, 599), (40, 2)):
        r.table[b, j] = (r.table[b, j] + 1) % r.k_pool.shape[0]
        _check_plan(r)
    for t in (1, 16, 17, 48, 49, 5000):
        _check_plan(r, min_tokens=t)


def test_plan_offsets():
    r = Shared([(3, 5), (3, 7)], [1] * 6, [2] * 6, 1, 1, seed=19)
    r.group_offsets = _i32([1, 3, 5])         # sequences of no group
    _check_plan(r)
    r.group_offsets = _i32([0])               # no group at all
    _check_plan(r)
    r.group_offsets = _i32([3, 9])
    members, prefix = _plan(r, status=sa.SA_ERR_INVALID_ARG)
    assert members.tolist() == [0, 0, 0, 3, 0, 0] and prefix.tolist() == [0] * 3 + [112] * 3
    r.lens[4] = 2 ** 30                       # behind the table
    r.group_offsets = _i32([3, 6])
    members, prefix = _plan(r, status=sa.SA_ERR_CAPACITY)
    assert prefix.tolist() == [0] * 3 + [112] * 3


def test_after_a_fork_captured():
    """A step of beam search: pages planned and copied, the new token appended, what the beams share found and read
    once; captured once and replayed on other contents."""
    Hq, Hk, beams = 8, 2, 6
    r = Shared([(beams, 25)], [1] * beams, [14] * beams, Hq, Hk, seed=20, spare=30, mpp=40)
    r.table[r.table >= r.k_pool.shape[0]] = -1
    r.k_pool.nan_to_num_(0), r.v_pool.nan_to_num_(0)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(beams, Hk, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    freq = torch.tensor([10000.0 ** (-j / 64) for j in range(64)], device="cuda")
    ws = sa.Workspace(r.prob, rows=True, max_rows=beams)
    parent, keep = _i32([0, 0, 2, 2, 5, 1]), r.lens - 1
    table2, src, dst, counts = torch.zeros_like(r.table), _i32([0] * beams), _i32([0] * beams), _i32([0, 0])
    members, prefix, out, q_out = _i32([0] * beams), _i32([0] * beams), torch.zeros_like(r.q), torch.zeros_like(r.q)

    def step():
        sa.plan_pages(r.prob, r.table, parent, keep, r.lens, table2, src, dst, counts, ws)
        sa.copy_pages(r.prob, r.k_pool, r.v_pool, src, dst, counts, ws)
        sa.qk_norm_rope(r.prob, r.q, k, v, r.offsets, r.lens, table2, q_out, r.k_pool, r.v_pool, ws, rope=sa.Rope(), inv_freq=freq)
        sa.shared_prefixes(r.prob, table2, r.lens, r.offsets, r.group_offsets, members, prefix, ws)
        sa.shared_attention(r.prob, q_out, r.k_pool, r.v_pool, table2, r.lens, r.offsets, members, prefix, out, ws)

    start = r.k_pool.clone(), r.v_pool.clone()
    step()
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK and prefix.tolist() == [400] * beams and members.tolist() == [beams] + [0] * (beams - 1)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for again in range(3):
        r.k_pool.copy_(start[0]), r.v_pool.copy_(start[1])
        if again == 1:      # other contents
            parent.copy_(_i32([3, 3, 3, 1, 0, 0]))
            r.q.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert ws.status() == sa.SA_OK
        if again == 0:
            assert torch.equal(out, want)
        keep_table, keep_q = r.table, r.q
        r.table, r.q = table2, q_out
        ref = R.attention(r)
        R.assert_within(out, ref["out"], ref["tol"], "out")
        r.table, r.q = keep_table, keep_q


def test_the_same_bits_again_and_on_two_streams():
    rs = [Shared([(6, 300), (4, 20)], [1, 1, 8, 1, 1, 1, 2, 1, 1, 30], [(i * 29) % 200 for i in range(10)], 28, 4, seed=21),
          Shared([(64, 60)], [1] * 64, [(i * 5) % 60 for i in range(64)], 8, 2, seed=22)]
    plans = [_plan(r) for r in rs]
    want = [_run(r, plan=p) for r, p in zip(rs, plans)]
    wss = [sa.Workspace(r.prob, rows=True, max_rows=r.n_rows) for r in rs]
    got = [(torch.zeros_like(o), torch.zeros_like(x)) for o, x in want]
    streams = [torch.cuda.Stream() for _ in rs]
    torch.cuda.synchronize()
    for _ in range(20):
        for r, p, ws, (o, x), st in zip(rs, plans, wss, got, streams):
            with torch.cuda.stream(st):
                sa.shared_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, *p, o, ws, lse=x)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_room():
    r = Shared([(2, 4)], [3, 1], [1, 1], 8, 2, seed=23)
    plan = _plan(r)
    for ws in (sa.Workspace(r.prob, rows=True), sa.Workspace(r.prob, rows=True, max_rows=3)):
        with pytest.raises(ValueError, match="max_rows"):
            sa.shared_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, *plan, torch.zeros_like(r.q), ws)
