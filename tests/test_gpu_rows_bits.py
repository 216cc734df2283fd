"""A row's result is its own: what other rows of its tile hold (the next
sequence's queries, rows of nobody, what an earlier call left in shared
memory) does not change a bit of it, and a row that sees nothing stays zero
beside one whose maximum grows."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_rows_attention import _check, _run

pytestmark = pytest.mark.gpu


def _equal(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("Hq,Hk", [(32, 8), (8, 8), (56, 8), (24, 8)])
@pytest.mark.parametrize("n", [1, 5, 37])
@pytest.mark.parametrize("tree", [False, True])
def test_neighbours_do_not_change_a_row(Hq, Hk, n, tree):
    # 20000 tokens and 8 KV heads: a block's piece has several tiles, over which the neighbours' scores grow
    r = R.Rows([n], [20000], Hq, Hk, seed=n + Hq, extra_rows=256)
    words = R.tree_words([n], 3) if tree else None
    outs = []
    for scale in (1.0, 60.0, 0.01):
        r.q[n:].mul_(scale)
        outs.append(_run(r, words))
    for out, lse in outs[1:]:
        assert _equal(out[:n], outs[0][0][:n]) and torch.equal(lse[:n], outs[0][1][:n])


@pytest.mark.parametrize("G", [3, 5, 6, 7])
def test_what_lies_in_shared_memory_does_not_change_a_row(G):
    # tiles of 128 // G * G rows: the lanes behind them hold nothing of this call
    n = 2 * (128 // G)
    r = R.Rows([n], [20000], 8 * G, 8, seed=G)
    other = R.Rows([32], [20000], 64, 8, seed=1)     # fills both query tiles of every block
    outs = []
    for scale in (1.0, 200.0, 1e-4):
        other.q.mul_(scale)
        _run(other)
        outs.append(_run(r))
    for out, lse in outs[1:]:
        assert _equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (7, 1)])
def test_an_empty_row_beside_one_whose_maximum_grows(Hq, Hk):
    # the prefix has no pages, so a row with an empty word sees nothing; another sees drafts of two tiles, the
    # later one with a score far above the earlier
    r = R.Rows([64], [240], Hq, Hk, seed=5)
    words = R.tree_words([64], 2)
    words[2], words[3], words[5] = 1 << 0 | 1 << 20, 0, 0
    r.table[0, :15] = -1
    for kvh in range(Hk):
        t = 240 + 20
        r.k_pool[int(r.table[0, t // 16]), kvh, t % 16] = 4 * r.q[2, kvh * (Hq // Hk)]
    out, lse = _check(r, words, status=sa.SA_ERR_BAD_PAGE)
    assert bool((out[[3, 5]] == 0).all()) and bool(torch.isneginf(lse[[3, 5]]).all())
