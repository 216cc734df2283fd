"""Prompts over selected blocks as a program runs them: pages planned, rows
rotated and appended, blocks summarised, lists selected and attended, and the
decode step behind them; then the sequence forked and read with its prefix
shared.  Eager and captured."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R
from tests import sparse_ref as Z

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hk", [(8, 2), (28, 4)])
def test_prompt_to_decode_step(Hq, Hk):
    B, S, W, k = 3, 4, 64, 6
    ahead, rows, mpp, pool = [900, 0, 333], [150, 300, 1], 80, 300
    bs = [(16, 32, 64, 8)[h % 4] for h in range(Hk)]
    g = torch.Generator(device="cuda").manual_seed(Hq)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    n = sum(rows)
    prob = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=mpp, num_pages=pool, sink=S, window=W, block_sizes=bs,
                      k_per_head=[k] * Hq, kcap=k)
    ws = sa.Workspace(prob, rows=True, max_rows=n)
    k_pool, v_pool = torch.zeros(pool, Hk, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(pool, Hk, 16, 128, dtype=torch.bfloat16, device="cuda")
    # what the cache holds ahead of the rows
    table0 = torch.full((B, mpp), -1, dtype=torch.int32, device="cuda")
    at = 7
    for b, a in enumerate(ahead):
        u = -(-a // 16)
        table0[b, :u] = torch.arange(at, at + u, device="cuda").int()
        at += u
    k_pool[7:at], v_pool[7:at] = rand(at - 7, Hk, 16, 128), rand(at - 7, Hk, 16, 128)
    lens, keep = _i32([a + m for a, m in zip(ahead, rows)]), _i32(ahead)
    off = _i32(np.concatenate([[0], np.cumsum(rows)]))
    q, kk, vv = rand(n, Hq, 128), rand(n, Hk, 128), rand(n, Hk, 128)
    freq = torch.tensor([10000.0 ** (-j / 64) for j in range(64)], device="cuda")
    table, src, dst, counts = torch.full_like(table0, -1), _i32([0] * B), _i32([0] * B), _i32([0, 0])
    summ = torch.zeros(prob.summary_shape(), dtype=torch.bfloat16, device="cuda")
    q_out, out, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(n, Hq, device="cuda")
    idx, cnt = torch.zeros(n, Hq, k, dtype=torch.int32, device="cuda"), torch.zeros(n, Hq, dtype=torch.int32, device="cuda")
    parent = _i32(range(B))

    def step():
        sa.plan_pages(prob, table0, parent, keep, lens, table, src, dst, counts, ws)
        sa.copy_pages(prob, k_pool, v_pool, src, dst, counts, ws)
        sa.qk_norm_rope(prob, q, kk, vv, off, lens, table, q_out, k_pool, v_pool, ws, rope=sa.Rope(), inv_freq=freq)
        sa.block_summarize(prob, k_pool, table, lens, summ, ws)
        sa.select_rows(prob, q_out, summ, lens, off, idx, cnt, ws)
        sa.sparse_row_attention(prob, q_out, k_pool, v_pool, table, lens, off, idx, cnt, out, ws, lse=lse)

    class Now:       # what the references look at
        pass

    def check():
        torch.cuda.synchronize()
        assert ws.status() == sa.SA_OK
        r = Now()
        r.B, r.Hq, r.Hk, r.G, r.mpp, r.n_rows, r.rows = B, Hq, Hk, Hq // Hk, mpp, n, rows
        r.q, r.table, r.lens, r.offsets, r.k_pool, r.v_pool, r.prob = q_out, table, lens, off, k_pool, v_pool, prob
        r.kv = lambda b, h: R.Rows.kv(r, b, h)
        for (row, h), w in Z.select(r, prob, summ).items():
            assert int(cnt[row, h]) == len(w) and idx[row, h, :len(w)].tolist() == w
        ref = Z.attention(r, prob, idx, cnt)
        R.assert_within(out, ref["out"], ref["tol"], "out")
        R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")
        # the last rows are a decode step's
        last = (off[1:] - 1).long()
        si, sc = torch.zeros(B, Hq, k, dtype=torch.int32, device="cuda"), torch.zeros(B, Hq, dtype=torch.int32, device="cuda")
        o, z = torch.zeros(B, Hq, 128, device="cuda"), torch.zeros(B, Hq, device="cuda")
        sa.decode_step(prob, q_out[last].contiguous(), k_pool, v_pool, table, lens, summ, si, sc, o, z, ws)
        torch.cuda.synchronize()
        assert torch.equal(sc, cnt[last])
        for b in range(B):
            for h in range(Hq):
                m = int(sc[b, h])
                assert torch.equal(si[b, h, :m], idx[last[b], h, :m])
        R.assert_within(out[last], o.double(), ref["tol"][last] + 2e-3, "as the decode step")
        R.assert_within(lse[last], z.double(), ref["tol_lse"][last] + 2e-3, "as the decode step")

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for again in range(2):
        q.copy_(rand(n, Hq, 128)), kk.copy_(rand(n, Hk, 128))
        lens.copy_(_i32([a + m - 7 * again for a, m in zip(ahead, rows)]))      # rows whose first have no position
        keep.copy_(torch.minimum(keep, (lens - (off[1:] - off[:-1])).clamp(min=0)))
        graph.replay()
        if again == 0:
            check()
        else:
            torch.cuda.synchronize()
            assert ws.status() == sa.SA_OK and bool(torch.isfinite(out).all())

    # the first sequence forked three times, a token each behind what they share
    lens1 = _i32([1040] * B)
    sa.plan_pages(prob, table, _i32([0] * B), _i32([1039] * B), lens1, table0, src, dst, counts, ws)
    sa.copy_pages(prob, k_pool, v_pool, src, dst, counts, ws)
    q1, k1, v1 = rand(B, Hq, 128), rand(B, Hk, 128), rand(B, Hk, 128)
    o1, members, prefix = torch.zeros_like(q1), _i32([0] * B), _i32([0] * B)
    off1 = _i32(range(B + 1))
    sa.qk_norm_rope(prob, q1, k1, v1, off1, lens1, table0, q1, k_pool, v_pool, ws, rope=sa.Rope(), inv_freq=freq)
    sa.shared_prefixes(prob, table0, lens1, off1, _i32([0, B]), members, prefix, ws)
    sa.shared_attention(prob, q1, k_pool, v_pool, table0, lens1, off1, members, prefix, o1, ws)
    o2 = torch.zeros_like(q1)
    sa.prompt_attention(prob, q1, k_pool, v_pool, table0, lens1, off1, o2, ws)
    torch.cuda.synchronize()
    assert ws.status() == sa.SA_OK and prefix.tolist() == [1024] * B and members.tolist() == [B, 0, 0]
    # each is within half a step of bf16 of its value and of each weight
    R.assert_within(o1, o2.double(), 2 * R.BF16 * (o2.double().abs() + 1.0), "against prompt_attention")
