"""Attention over selected blocks in a batch most of whose sequences have no rows
(a prompt in a table of many): the same result, and no time for those without."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa

pytestmark = pytest.mark.gpu


def _call(B, at, n, L=4000, Hq=8, Hk=2):
    """Sequence `at` of B has n rows, the others none."""
    g = torch.Generator(device="cuda").manual_seed(1)
    mpp = -(-L // 16)
    table = torch.zeros(B, mpp, dtype=torch.int32, device="cuda")
    table[at] = torch.randperm(mpp, generator=g, device="cuda").int()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[at] = L
    offsets = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    offsets[at + 1:] = n
    q = torch.randn(n, Hq, 128, generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(mpp, Hk, 16, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    prob = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=mpp, num_pages=mpp, sink=4, window=256, block_sizes=[16] * Hk,
                      k_per_head=[8] * Hq, kcap=8)
    idx = torch.randint(0, mpp, (n, Hq, 8), generator=g, device="cuda").sort(-1).values.int()
    cnt = torch.full((n, Hq), 8, dtype=torch.int32, device="cuda")
    ws = sa.Workspace(prob, rows=True, max_rows=n)
    out, lse = torch.zeros_like(q), torch.zeros(n, Hq, device="cuda")

    def run():
        sa.sparse_row_attention(prob, q, k, v, table, lens, offsets, idx, cnt, out, ws, lse=lse)
    return run, out, lse, ws


def _time(run):
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = float("inf")
    for _ in range(5):
        start.record()
        run()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end))
    return best


@pytest.mark.parametrize("n", [1, 130, 2000])
def test_sequences_without_rows_change_nothing(n):
    alone = _call(1, 0, n)
    alone[0]()
    for B, at in ((64, 0), (300, 299), (2000, 1000)):
        run, out, lse, ws = _call(B, at, n)
        run()
        torch.cuda.synchronize()
        assert ws.status() == sa.SA_OK
        assert torch.equal(out, alone[1]) and torch.equal(lse, alone[2])


def test_they_take_no_time():
    # eight times that of the sequence alone is far above what their places cost, and far below a walk over them (80 times)
    alone, many = _call(1, 0, 2000, Hq=32, Hk=8), _call(2000, 0, 2000, Hq=32, Hk=8)
    a, b = _time(alone[0]), _time(many[0])
    assert b < 8 * a, f"{b * 1e3:.0f} us with 1999 sequences without rows, {a * 1e3:.0f} us without them"
