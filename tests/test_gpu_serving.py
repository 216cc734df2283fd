"""The calls together, as a serving program uses them: pages for two prompts,
their rows rotated into the cache, prompt attention; each prompt forked, a tree
drafted and verified, a path accepted; the pool packed; then the decode step
over the same pages.  A shadow keeps every sequence's keys and values."""
import numpy as np
import pytest
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

pytestmark = pytest.mark.gpu
D, P = 128, 16
Hq, Hk, B, MPP, PAGES = 8, 2, 4, 40, 128


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Serve:
    def __init__(self, graphs):
        g = self.g = torch.Generator(device="cuda").manual_seed(3)
        self.graphs = graphs
        # k_per_head covers every candidate block: the decode step is then dense
        self.prob = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=MPP, num_pages=PAGES, sink=4, window=64,
                               block_sizes=[P] * Hk, k_per_head=[MPP] * Hq, kcap=MPP)
        self.ws = sa.Workspace(self.prob, rows=True)
        self.kp, self.vp = (torch.full((PAGES, Hk, P, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table, self.lens = torch.full((B, MPP), -1, dtype=torch.int32, device="cuda"), [0] * B
        self.shadow = [(torch.zeros(0, Hk, D), torch.zeros(0, Hk, D)) for _ in range(B)]
        self.freq = torch.tensor([10000.0 ** (-j / 64) for j in range(64)], device="cuda")
        self.qw, self.kw = ((1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))

    def call(self, f):
        """The call, or the same captured and replayed."""
        if not self.graphs:
            return f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        graph.replay()
        torch.cuda.synchronize()

    def pages(self, parent, keep, lens):
        out = torch.empty_like(self.table)
        src, dst, counts = _i32([0] * B), _i32([0] * B), _i32([0, 0])
        pa, ke, le = _i32(parent), _i32(keep), _i32(lens)

        def both():
            sa.plan_pages(self.prob, self.table, pa, ke, le, out, src, dst, counts, self.ws)
            sa.copy_pages(self.prob, self.kp, self.vp, src, dst, counts, self.ws)
        self.call(both)
        assert counts[1] >= 0
        self.table = out
        self.shadow = [tuple(x[:k].clone() for x in self.shadow[p]) if p >= 0 else (torch.zeros(0, Hk, D),) * 2 for p, k in zip(parent, keep)]
        self.lens = list(keep)

    def append(self, rows, positions):
        n = sum(rows)
        qkv = torch.randn(n, (Hq + 2 * Hk) * D, generator=self.g, device="cuda").to(torch.bfloat16)
        q, k, v = (qkv[:, a * D:b * D].view(n, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        off = _i32(np.concatenate([[0], np.cumsum(rows)]).tolist())
        q_out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
        self.lens = [a + b for a, b in zip(self.lens, rows)]
        lens, pos = _i32(self.lens), _i32([positions])
        self.call(lambda: sa.qk_norm_rope(self.prob, q, k, v, off, lens, self.table, q_out, self.kp, self.vp, self.ws,
                                          rope=sa.Rope(), inv_freq=self.freq, positions=pos, q_weight=self.qw, k_weight=self.kw))
        ks, vs = self.read()
        o = 0
        for b, m in enumerate(rows):     # the appended keys are what the rotation made (tested elsewhere), the values are exact
            assert torch.equal(vs[b][self.lens[b] - m:], v[o:o + m].cpu().float())
            self.shadow[b] = (torch.cat([self.shadow[b][0], ks[b][self.lens[b] - m:]]), torch.cat([self.shadow[b][1], vs[b][self.lens[b] - m:]]))
            o += m
        return q_out, off, lens

    def read(self):
        t = self.table.cpu().long()
        kp, vp = self.kp.cpu().float(), self.vp.cpu().float()
        ks, vs = [], []
        for b, L in enumerate(self.lens):
            at = torch.arange(L)
            page = t[b, at // P]
            assert bool((page >= 0).all())
            ks.append(kp[page, :, at % P])
            vs.append(vp[page, :, at % P])
        return ks, vs

    def check(self):
        ks, vs = self.read()
        for b in range(B):
            assert torch.equal(ks[b], self.shadow[b][0]) and torch.equal(vs[b], self.shadow[b][1]), f"sequence {b}"

    def rows(self, rows, q, off):
        """The references' view of the present cache."""
        r = R.Rows.__new__(R.Rows)
        r.rows, r.Hq, r.Hk, r.G, r.B, r.mpp = rows, Hq, Hk, Hq // Hk, B, MPP
        r.table, r.offsets, r.lens, r.q, r.n_rows = self.table, off, _i32(self.lens), q, q.shape[0]
        r.k_pool, r.v_pool, r.prob = self.kp, self.vp, self.prob
        return r

    def attend(self, rows, q, off, lens, words=None):
        out = torch.empty(q.shape[0], Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(q.shape[0], Hq, device="cuda")
        if words is None:
            self.call(lambda: sa.prompt_attention(self.prob, q, self.kp, self.vp, self.table, lens, off, out, self.ws, lse=lse))
        else:
            mask = torch.from_numpy(words.view(np.int64)).cuda()
            self.call(lambda: sa.tree_attention(self.prob, q, self.kp, self.vp, self.table, lens, off, mask, out, self.ws, lse=lse))
        ref = R.attention(self.rows(rows, q, off), words)
        R.assert_within(out, ref["out"], ref["tol"], "out")
        R.assert_within(lse, ref["lse"], ref["tol_lse"], "lse")


@pytest.mark.parametrize("graphs", [False, True])
def test_prompt_fork_draft_accept_pack_decode(graphs):
    s = Serve(graphs)
    if graphs:      # kernels' first launches are not captured
        test_prompt_fork_draft_accept_pack_decode(False)
    # two prompts
    s.pages([-1] * B, [0] * B, [300, 77, 0, 0])
    rows = [300, 77, 0, 0]
    s.attend(rows, *s.append(rows, list(range(300)) + list(range(77))))
    s.check()
    # each goes on as two, with room for a draft of 9
    s.pages([0, 1, 0, 1], [300, 77, 300, 77], [309, 86, 309, 86])
    s.check()
    rows = [9] * 4
    words = R.tree_words(rows, 5)
    depth = [bin(int(w)).count("1") - 1 for w in words]
    q, off, lens = s.append(rows, [L + d for L, dd in zip([300, 77, 300, 77], np.array(depth).reshape(4, 9)) for d in dd])
    s.attend(rows, q, off, lens, words)
    s.check()
    # a path of each is accepted
    path = [[0, 3, 7], [2, 0, 0], [1, 4, 5], [0, 1, 8]]
    cnt = [3, 1, 2, 3]
    base = [300, 77, 300, 77]
    p_d, c_d, b_d = _i32(path), _i32(cnt), _i32(base)
    s.call(lambda: sa.accept_rows(s.prob, s.kp, s.vp, s.table, b_d, p_d, c_d, s.ws))
    for b in range(B):
        at = torch.cat([torch.arange(base[b]), torch.tensor([base[b] + path[b][i] for i in range(cnt[b])])])
        s.shadow[b] = tuple(x[at] for x in s.shadow[b])
        s.lens[b] = base[b] + cnt[b]
    s.check()
    # one is given up, one forked again, the pool packed
    s.pages([0, 3, 3, 1], [s.lens[0], s.lens[3], s.lens[3], s.lens[1]], [s.lens[0] + 1, s.lens[3] + 1, s.lens[3] + 1, s.lens[1] + 1])
    s.check()
    room = _i32([n + 1 for n in s.lens])
    out = torch.empty_like(s.table)
    src, dst, counts = _i32([0] * PAGES), _i32([0] * PAGES), _i32([0, 0])

    def pack():
        sa.compact_pages(s.prob, s.table, room, out, src, dst, counts, s.ws)
        sa.copy_pages(s.prob, s.kp, s.vp, src, dst, counts, s.ws)
    s.call(pack)
    s.table = out
    assert int(s.table.max()) == int(counts[1]) - 1
    s.check()
    # a token a sequence: the framework's own append and decode step over these pages, against the rows' attention
    s.lens = [n + 1 for n in s.lens]
    lens = _i32(s.lens)
    k_new, v_new = (torch.randn(B, Hk, D, generator=s.g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, Hq, D, generator=s.g, device="cuda").to(torch.bfloat16)
    # what no token has been written to must be finite for the block summaries' pages
    sa.append_kv(s.prob, k_new, v_new, s.kp, s.vp, s.table, lens, s.ws)
    s.shadow = [(torch.cat([a, k_new[b:b + 1].cpu().float()]), torch.cat([v, v_new[b:b + 1].cpu().float()])) for b, (a, v) in enumerate(s.shadow)]
    s.check()
    off = _i32(list(range(B + 1)))
    s.attend([1] * B, q, off, lens)
    s.attend([1] * B, q, off, lens, np.ones(B, np.uint64))
    s.kp.nan_to_num_(0)
    s.vp.nan_to_num_(0)
    summ = torch.zeros(s.prob.summary_shape(), dtype=torch.bfloat16, device="cuda")
    sa.block_summarize(s.prob, s.kp, s.table, lens, summ, s.ws)
    sel, n_sel = torch.empty(B, Hq, MPP, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, dtype=torch.int32, device="cuda")
    o, lse = torch.empty(B, Hq, D, device="cuda"), torch.empty(B, Hq, device="cuda")
    sa.decode_step(s.prob, q, s.kp, s.vp, s.table, lens, summ, sel, n_sel, o, lse, s.ws)
    ref = R.attention(s.rows([1] * B, q, off))
    R.assert_within(o, ref["out"], ref["tol"], "decode step")
    assert s.ws.status() == sa.SA_OK
