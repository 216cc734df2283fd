"""What the decode step keeps by sequence after a fork: block summaries taken
from the parents' rows, and made again only from the kept tokens on, are those
of the whole cache; a step of beam search needs no more than its own refresh."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
D, P = 128, 16
B, Hq, Hk, MPP, PAGES = 6, 8, 2, 30, 256


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class State:
    def __init__(self, mode, bs):
        g = torch.Generator(device="cuda").manual_seed(1)
        self.bs = bs
        self.prob = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=MPP, num_pages=PAGES, sink=4, window=64, mode=mode,
                               block_sizes=bs, k_per_head=[MPP * 2] * Hq, kcap=MPP * 2)
        self.ws = sa.Workspace(self.prob, rows=True)
        self.kp, self.vp = (torch.randn(PAGES, Hk, P, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.lens = [300, 77, 16, 400, 129, 255]
        perm = np.random.RandomState(2).permutation(PAGES)
        self.table = np.full((B, MPP), -1)
        at = 0
        for b, L in enumerate(self.lens):
            n = -(-L // P)
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.table = _i32(self.table)
        self.summ = self.summaries()

    def summaries(self, into=None, begin=0):
        s = torch.zeros(self.prob.summary_shape(), dtype=torch.bfloat16, device="cuda") if into is None else into
        sa.block_summarize(self.prob, self.kp, self.table, _i32(self.lens), s, self.ws, block_begin=begin)
        return s

    def plan(self, parent, keep, lens):
        out, src, dst, counts = torch.empty_like(self.table), _i32([0] * B), _i32([0] * B), _i32([0, 0])
        sa.plan_pages(self.prob, self.table, _i32(parent), _i32(keep), _i32(lens), out, src, dst, counts, self.ws)
        sa.copy_pages(self.prob, self.kp, self.vp, src, dst, counts, self.ws)
        self.table, self.lens = out, list(lens)
        self.summ = self.summ[_i32(parent).long().clamp(min=0)].contiguous()

    def same(self):
        full = self.summaries()
        for b, L in enumerate(self.lens):
            for h in range(Hk):
                n = -(-L // self.bs[h])
                assert torch.equal(self.summ[b, h, :n], full[b, h, :n]), (b, h)


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
@pytest.mark.parametrize("bs", [[16, 16], [32, 64], [8, 16]])
def test_summaries_follow_the_parents(mode, bs):
    s = State(mode, bs)
    s.same()
    # forked, cut back, one freed; some grow by many tokens
    parent, keep = [3, 3, 0, 1, 5, 4], [400, 123, 300, 70, 255, 128]
    lens = [450, 170, 300, 90, 256, 139]
    s.plan(parent, keep, lens)
    grow = [b - a for a, b in zip(keep, lens)]
    n = sum(grow)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
    off = _i32(np.concatenate([[0], np.cumsum(grow)]))
    sa.qk_norm_rope(s.prob, q, k, v, off, _i32(lens), s.table, torch.empty_like(q), s.kp, s.vp, s.ws)
    s.summaries(s.summ, min(k // max(bs) for k in keep))
    s.same()
    # accepted rows of a draft change the blocks from its base on
    base = [440, 160, 290, 80, 246, 129]
    sa.accept_rows(s.prob, s.kp, s.vp, s.table, _i32(base), _i32([[1, 5, 8]] * B), _i32([3] * B), s.ws)
    s.lens = [x + 3 for x in base]
    s.summaries(s.summ, min(base) // max(bs))
    s.same()
    assert s.ws.status() == sa.SA_OK


@pytest.mark.parametrize("mode", [sa.SUMMARY_MINMAX, sa.SUMMARY_MEAN])
def test_a_step_of_beam_search(mode):
    s = State(mode, [16, 32])
    for step, parent in enumerate(([0, 0, 3, 3, 3, 5], [1, 0, 2, 5, 4, 4], [0, 1, 2, 3, 4, 5])):
        keep = [s.lens[p] for p in parent]
        s.plan(parent, keep, [x + 1 for x in keep])
        g = torch.Generator(device="cuda").manual_seed(step)
        q, k, v = (torch.randn(B, h, D, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
        sel, cnt = torch.empty(B, Hq, 2 * MPP, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, dtype=torch.int32, device="cuda")
        o, lse = torch.empty(B, Hq, D, device="cuda"), torch.empty(B, Hq, device="cuda")
        lens = _i32(s.lens)
        sa.decode_step_append(s.prob, q, k, v, s.kp, s.vp, s.table, lens, s.summ, sel, cnt, o, lse, s.ws)
        s.same()
        # every candidate is selected: the step is the attention of one row a sequence
        r = R.Rows.__new__(R.Rows)
        r.rows, r.Hq, r.Hk, r.G, r.B, r.mpp, r.n_rows, r.prob = [1] * B, Hq, Hk, Hq // Hk, B, MPP, B, s.prob
        r.table, r.offsets, r.lens, r.q, r.k_pool, r.v_pool = s.table, _i32(range(B + 1)), lens, q, s.kp, s.vp
        ref = R.attention(r)
        R.assert_within(o, ref["out"], ref["tol"], "out")
        R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")
        assert s.ws.status() == sa.SA_OK
