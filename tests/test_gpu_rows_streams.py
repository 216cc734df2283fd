"""Calls at once: two streams, each with a workspace of its own, give what one
after the other gives, bit for bit; and the smallest calls there are."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_rotate import _run as rotate
from tests.test_gpu_rows_attention import _check

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Step:
    """Rows appended, attended as a prompt and as a tree, forked, packed, and a path accepted: all outputs."""

    def __init__(self, rows, prefix, Hq, Hk, seed):
        self.r = r = R.Rows(rows, prefix, Hq, Hk, seed=seed, spare=40)
        r.table[r.table >= r.k_pool.shape[0]] = -1
        r.k_pool.nan_to_num_(0), r.v_pool.nan_to_num_(0)
        self.ws = sa.Workspace(r.prob, rows=True)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.randn(r.n_rows, Hk, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.freq = torch.tensor([10000.0 ** (-j / 64) for j in range(64)], device="cuda")
        self.mask = torch.from_numpy(R.tree_words(rows, seed).view(np.int64)).cuda()
        B, pages = r.B, r.k_pool.shape[0]
        self.parent, self.keep = _i32([0] * B), _i32([int(r.lens[0]) - 3] * B)
        self.room, self.base = self.keep + 1, _i32(prefix)
        self.path, self.cnt = _i32([[1, 2]] * B), _i32([2] * B)
        self.out = [torch.zeros_like(r.q) for _ in range(3)]
        self.lse = [torch.zeros(r.n_rows, Hq, device="cuda") for _ in range(2)]
        self.tables = [torch.zeros_like(r.table) for _ in range(2)]
        self.lists = [_i32([0] * n) for n in (B, B, 2, pages, pages, 2)]
        self.start = [x.clone() for x in (r.k_pool, r.v_pool)]

    def __call__(self):
        r, ws = self.r, self.ws
        r.k_pool.copy_(self.start[0]), r.v_pool.copy_(self.start[1])
        sa.qk_norm_rope(r.prob, r.q, self.k, self.v, r.offsets, r.lens, r.table, self.out[0], r.k_pool, r.v_pool, ws,
                        rope=sa.Rope(), inv_freq=self.freq)
        sa.prompt_attention(r.prob, self.out[0], r.k_pool, r.v_pool, r.table, r.lens, r.offsets, self.out[1], ws, lse=self.lse[0])
        sa.tree_attention(r.prob, self.out[0], r.k_pool, r.v_pool, r.table, r.lens, r.offsets, self.mask, self.out[2], ws,
                          lse=self.lse[1])
        sa.accept_rows(r.prob, r.k_pool, r.v_pool, r.table, self.base, self.path, self.cnt, ws)
        a, b, c, d, e, f = self.lists
        sa.plan_pages(r.prob, r.table, self.parent, self.keep, self.room, self.tables[0], a, b, c, ws)
        sa.copy_pages(r.prob, r.k_pool, r.v_pool, a, b, c, ws)
        sa.compact_pages(r.prob, self.tables[0], self.room, self.tables[1], d, e, f, ws)
        sa.copy_pages(r.prob, r.k_pool, r.v_pool, d, e, f, ws)

    def results(self):
        r = self.r
        return [x.clone() for x in (r.k_pool, r.v_pool, *self.out, *self.lse, *self.tables, *self.lists)]


def test_two_streams():
    steps = [Step([40, 3, 64, 17], [700, 2000, 30, 5], 8, 2, 1), Step([64, 64, 9], [9000, 40, 300], 28, 4, 2)]
    want = []
    for s in steps:
        s()
        torch.cuda.synchronize()
        want.append(s.results())
        assert s.ws.status() == sa.SA_OK
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(s.results(), w):
            assert torch.equal(a, b)
        assert s.ws.status() == sa.SA_OK


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 1), (3, 3)])
@pytest.mark.parametrize("prefix", [0, 15])
def test_one_row_one_page(Hq, Hk, prefix):
    r = R.Rows([1], [prefix], Hq, Hk, seed=3, spare=0)
    _check(r)
    _check(r, R.tree_words([1]))
    assert rotate(r, 1, 0, [64], sa.ROPE_PAIRS, _i32([[prefix]]), 3) == sa.SA_OK
