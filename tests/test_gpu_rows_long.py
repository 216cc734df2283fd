"""The row and page calls at the sizes where their work is divided otherwise
than in a small call: a warp of the rotation with many heads and several rows,
trees and prompts cut by weight, blocks with many pieces, pools of many
chunks.  And every token of a long cache marked once: a row whose query is
the token's key has the token's value as its result."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests.test_gpu_pages import _plan, _random_table, test_compact_and_copy as compact_and_copy
from tests.test_gpu_rotate import _run as rotate
from tests.test_gpu_rows_attention import _check

pytestmark = pytest.mark.gpu
D, P = 128, 16


@pytest.mark.parametrize("Hq,Hk", [(32, 8), (28, 4), (8, 2), (64, 8)])
@pytest.mark.parametrize("rows,prefix", [([7000, 1, 0, 295], [5, 90, 3, 0])])
def test_rotation_of_many_rows(Hq, Hk, rows, prefix):
    r = R.Rows(rows, prefix, Hq, Hk, seed=Hq, lead=2)
    pos = torch.arange(3 * r.n_rows, dtype=torch.int32).cuda().view(3, -1)
    assert rotate(r, r.n_rows, 8, [16, 24, 24], sa.ROPE_HALVES, pos, 3) == sa.SA_OK
    assert rotate(r, r.n_rows, 0, [32], sa.ROPE_PAIRS, pos[:1].contiguous(), 2) == sa.SA_OK
    assert rotate(r, r.n_rows, 8, [20, 30], sa.ROPE_HALVES, pos[:2].contiguous(), 1) == sa.SA_OK


@pytest.mark.parametrize("Hq,Hk", [(28, 4), (8, 2), (8, 1), (8, 8)])
def test_trees_cut_by_weight(Hq, Hk):
    rng = np.random.RandomState(Hq + Hk)
    rows = [int(rng.choice([0, 1, 64, rng.randint(1, 65)])) for _ in range(45)]     # more than 32 sequences
    prefix = [int(np.exp(rng.uniform(0, np.log(4000)))) for _ in rows]
    _check(R.Rows(rows, prefix, Hq, Hk, seed=1), R.tree_words(rows, 1))


def test_trees_of_a_long_even_batch():
    rows = [32] * 6
    _check(R.Rows(rows, [9000 - 16 * b for b in range(6)], 32, 8, seed=2), R.tree_words(rows, 2))


def test_prompt_whose_weight_passes_32_bits_a_block():
    _check(R.Rows([8192, 700], [0, 300], 32, 4, seed=3))


def test_blocks_with_many_pieces():
    # 400 sequences of 8 KV heads: about twenty items a block, some with values that are not finite at their edge
    rows = [1 + i % 5 for i in range(400)]
    prefix = [(i * 37) % 300 for i in range(400)]
    r = R.Rows(rows, prefix, 8, 8, seed=4)
    for b in range(0, 400, 3):
        t = prefix[b] + rows[b] - 1
        r.v_pool[int(r.table[b, t // P]), :, t % P, b % 7::11] = float("inf") if b % 2 else float("nan")
    _check(r)
    _check(r, R.tree_words(rows, 4))


@pytest.mark.parametrize("B,mpp,slack", [(128, 64, 40000), (300, 200, 20000)])
def test_packing_a_large_pool(B, mpp, slack):
    compact_and_copy(B, mpp, slack, 1)


def test_planning_over_a_large_pool():
    rng = np.random.RandomState(5)
    B, mpp, pages = 200, 150, 45000
    old = [int(rng.randint(0, mpp * P + 1)) for _ in range(B)]
    table = _random_table(rng, B, mpp, pages, old)
    parent = [int(x) for x in rng.randint(-1, B, B)]
    keep = [0 if p < 0 else int(rng.randint(0, old[p] + 1)) for p in parent]
    lens = [int(rng.randint(k, mpp * P + 1)) for k in keep]
    assert _plan(table, parent, keep, lens, pages)[0] == sa.SA_OK


# ------------------------------------------------------------------ marked tokens

def _marked(r, at, words=None):
    """Row i, head h looks for token at[i][h]: its query is five times that token's key.

    Keys are N(0, 1), so |k|^2 is 128 with a deviation of 16 and above 60 for every token here; the marked score is
    then above 5 * 60 / sqrt(128) = 26, and another's has a deviation of 5 |k| / sqrt(128), 3.5 at that |k|: 20000 of
    them have e^(9.9 + 3.5^2 / 2) = e^16 in all, against e^26.  That their weight is below 1e-3 is checked in 64 bits.
    The result is the value but for that weight times the largest |v| (below 6, twice) and two roundings of 2^-8, of
    the weight and of the result.  The score itself is a sum of 128 products of at most 5 |k|^2 / sqrt(128) < 100 in
    all, off by less than 1e-3 in fp32."""
    q = torch.zeros(r.n_rows, r.Hq, D, device="cuda")
    v = torch.zeros_like(q, dtype=torch.float64)
    z = torch.zeros(r.n_rows, r.Hq, dtype=torch.float64, device="cuda")
    for b in range(r.B):
        rows = slice(int(r.offsets[b]), int(r.offsets[b + 1]))
        for h in range(r.Hq):
            ks, vs, _ = r.kv(b, h // r.G)
            t = at[rows, h]
            q[rows, h] = (5 * ks[t]).float()
            v[rows, h] = vs[t]
    r.q.copy_(q)
    for b in range(r.B):
        rows = slice(int(r.offsets[b]), int(r.offsets[b + 1]))
        for h in range(r.Hq):
            ks, _, _ = r.kv(b, h // r.G)
            s = r.q[rows, h].double() @ ks.T * r.prob.scale
            z[rows, h] = s.gather(1, at[rows, h][:, None])[:, 0]
            rest = torch.exp(s - z[rows, h][:, None]).sum(1) - 1     # over the whole cache: more than the row sees
            assert float(rest.max()) < 1e-3
    out = torch.zeros_like(r.q)
    lse = torch.zeros(r.n_rows, r.Hq, device="cuda")
    ws = sa.Workspace(r.prob, rows=True)
    if words is None:
        sa.prompt_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, out, ws, lse=lse)
    else:
        mask = torch.from_numpy(words.view(np.int64)).cuda()
        sa.tree_attention(r.prob, r.q, r.k_pool, r.v_pool, r.table, r.lens, r.offsets, mask, out, ws, lse=lse)
    assert ws.status() == sa.SA_OK
    assert float((out.double() - v).abs().sub(2 * R.BF16 * 1.01 * v.abs()).max()) < 2 * 6 * 1e-3
    assert float((lse.double() - z).abs().max()) < 2e-3


@pytest.mark.parametrize("Hq,Hk,rows,prefix", [
    (8, 2, [64], [9000]), (28, 4, [64, 36], [6000, 8100]), (8, 2, [16, 30, 20, 33], [3000, 4095, 4096, 1111]),
    (8, 1, [64], [20000]), (32, 8, [32] * 4, [5000] * 4)])
def test_every_token_of_a_long_cache_counts(Hq, Hk, rows, prefix):
    r = R.Rows(rows, prefix, Hq, Hk, seed=sum(prefix))
    words = np.array([1 << i for n in rows for i in range(n)], dtype=np.uint64)     # a row sees the prefix and itself
    G, cols = Hq // Hk, [n * Hq // Hk for n in rows]
    for call in range(max(-(-p // c) for p, c in zip(prefix, cols))):
        at = torch.zeros(r.n_rows, Hq, dtype=torch.int64, device="cuda")
        for b, (n, p) in enumerate(zip(rows, prefix)):
            o = int(r.offsets[b])
            which = (call * cols[b] + torch.arange(n * G, device="cuda")) % p       # every token once for each KV head
            at[o:o + n] = which.view(n, 1, G).expand(n, Hk, G).reshape(n, Hq)
        _marked(r, at, words)
        if call % 4 == 0:
            _marked(r, at)


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
@pytest.mark.parametrize("rows,prefix", [([900, 300], [0, 2500]), ([2000], [100])])
def test_every_row_of_a_prompt_finds_its_token(Hq, Hk, rows, prefix):
    r = R.Rows(rows, prefix, Hq, Hk, seed=7)
    # the row's own token, the one before, the first, tile and page borders behind and before it, and random ones
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(rows, prefix)]).cuda()[:, None]
    for pick in (lambda x: x, lambda x: x - 1, lambda x: x // 128 * 128, lambda x: x // 128 * 128 - 1, lambda x: x // 16 * 16,
                 lambda x: x * 0, lambda x: (torch.rand(x.shape[0], Hq, generator=g, device="cuda") * (x + 1)).long()):
        _marked(r, pick(pos).clamp(min=0).expand(-1, Hq).contiguous())
