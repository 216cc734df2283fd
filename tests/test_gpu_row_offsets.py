"""Row offsets and lengths that are wrong are recorded by the rotation and the
attention alike, whichever sequence they belong to: one that decreases, one
behind the rows, one without rows."""
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
D = 128

BAD, CAP = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_CAPACITY
MANY = [min(i, 20) for i in range(701)]

CASES = [
    ([0, 15, 10, 20], None, 20, BAD),        # decreases: two sequences claim rows 10 .. 14
    ([0, 10, 5], None, 10, BAD),             # decreases at the end
    ([0, 10, 12, 15], None, 10, BAD),        # begins at and behind the last row
    ([0, 4, 100], None, 8, BAD),
    ([-3, 4, 8], None, 8, BAD),
    ([0, 10, 10], [12, 500], 10, CAP),       # a sequence without rows, longer than the table
    ([0, 10, 20], [12, 500], 20, CAP),
    (MANY[:651] + [3] + MANY[652:], None, 20, BAD),
    (MANY, [30] * 650 + [500] + [30] * 49, 20, CAP),
    (MANY, None, 20, sa.SA_OK),
    ([0, 10, 10, 20], [30, 0, 30], 20, sa.SA_OK),
]


@pytest.mark.parametrize("offsets,lens,n,want", CASES)
@pytest.mark.parametrize("call", ["rotation", "prompt", "tree"])
def test_every_sequence_is_checked(call, offsets, lens, n, want):
    B, Hq, Hk, mpp = len(offsets) - 1, 8, 2, 4
    prob = R.problem(B, Hq, Hk, mpp, 4 * B)
    ws = sa.Workspace(prob, rows=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
    kp, vp = (torch.zeros(4 * B, Hk, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(4 * B, dtype=torch.int32, device="cuda").view(B, mpp)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    length = torch.tensor(lens or [30] * B, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    if call == "rotation":
        sa.qk_norm_rope(prob, q, k, v, off, length, table, out, kp, vp, ws)
    elif call == "prompt":
        sa.prompt_attention(prob, q, kp, vp, table, length, off, out, ws)
    else:
        mask = torch.ones(n, dtype=torch.int64, device="cuda")
        sa.tree_attention(prob, q, kp, vp, table, length, off, mask, out, ws)
    assert ws.status() == want
    if call == "rotation":
        assert torch.equal(out, q)       # neither norm nor rotation, and every row belongs to some sequence
