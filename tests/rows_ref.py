"""Plain references in 64 bits for the packed-row and page calls, and the inputs
that their tests share.  Sequences, heads and pages are taken one at a time."""
import math

import numpy as np
import torch

from sparse_decode_attention_head_gb300 import sa

D, P = 128, 16
BF16 = 2.0 ** -8        # half a step of bf16, relative


class Rows:
    """Packed rows of some sequences over a pool that is NaN where nobody may look."""

    def __init__(self, rows, prefix, Hq, Hk, seed=0, extra_rows=0, lead=0, spare=3, mpp=None, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.rows, self.prefix, self.Hq, self.Hk, self.G = list(rows), list(prefix), Hq, Hk, Hq // Hk
        self.B = len(self.rows)
        lens = [p + n for p, n in zip(self.prefix, self.rows)]
        need = [max(0, -(-L // P)) for L in lens]
        self.mpp = mpp or max(1, max(need))
        pool = sum(need) + spare
        perm = torch.randperm(pool, generator=g, device=device).to(torch.int32)
        self.table = torch.full((self.B, self.mpp), 2 ** 31 - 1, dtype=torch.int32, device=device)
        at = 0
        for b, n in enumerate(need):
            n = min(n, self.mpp)
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.n_rows = lead + sum(self.rows) + extra_rows
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(self.rows)]) + lead, dtype=torch.int32, device=device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.q = torch.randn(self.n_rows, Hq, D, generator=g, device=device).to(torch.bfloat16)
        self.k_pool = torch.full((pool, Hk, P, D), float("nan"), dtype=torch.bfloat16, device=device)
        self.v_pool = torch.full((pool, Hk, P, D), float("nan"), dtype=torch.bfloat16, device=device)
        for b, L in enumerate(lens):
            for t0 in range(0, min(L, self.mpp * P), P):
                page, n = int(self.table[b, t0 // P]), min(P, L - t0)
                self.k_pool[page, :, :n] = torch.randn(Hk, n, D, generator=g, device=device).to(torch.bfloat16)
                self.v_pool[page, :, :n] = torch.randn(Hk, n, D, generator=g, device=device).to(torch.bfloat16)
        self.prob = problem(self.B, Hq, Hk, self.mpp, pool)

    def kv(self, b, kvh):
        """K and V of one KV head of a sequence, in 64 bits (NaN where the page is not there), and which are there."""
        L = int(self.lens[b])
        t = torch.arange(min(L, self.mpp * P), device=self.q.device)
        page = self.table[b].long()[t // P]
        there = (page >= 0) & (page < self.k_pool.shape[0])
        page = page.clamp(0, self.k_pool.shape[0] - 1)
        return self.k_pool[page, kvh, t % P].double(), self.v_pool[page, kvh, t % P].double(), there


def problem(B, Hq, Hk, mpp, num_pages, scale=None):
    return sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=mpp, num_pages=num_pages, sink=4, window=64,
                      block_sizes=[P] * Hk, k_per_head=[1] * Hq, kcap=1, scale=scale)


def tree_words(rows, seed=0, words=None):
    """Random trees: a node's ancestors and itself, as int64."""
    rng = np.random.RandomState(seed)
    out = []
    for n in rows:
        up = []
        for i in range(n):
            parent = int(rng.randint(-1, i)) if i else -1
            up.append((up[parent] if parent >= 0 else 0) | 1 << i)
        out += up
    return np.array(out, dtype=np.uint64)


def attention(r: Rows, words=None):
    """{"out", "lse", "tol", "tol_lse"} of the rows' attention: positions up to
    the row's own, or (words) the prefix and the drafts of its word.

    tol: the result is rounded to bf16 once (half a step of |out|) and so is
    every softmax weight (half a step of each term of sum p |v|); scores are
    sums of 128 exact products in fp32, each addition off by at most 2^-23 of
    the running magnitude, and one exponential is off by 2^-22 relative; a
    weight changes by as much as its score."""
    n = r.n_rows
    dev = r.q.device
    out = torch.zeros(n, r.Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((n, r.Hq), -math.inf, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    scale = r.prob.scale
    for b in range(r.B):
        m, o0 = r.rows[b], int(r.offsets[b])
        a = int(r.lens[b]) - m
        for kvh in range(r.Hk):
            k, v, there = r.kv(b, kvh)
            L = k.shape[0]
            t = torch.arange(L, device=dev)
            if words is None:
                seen = t[None] <= a + torch.arange(m, device=dev)[:, None]
            else:
                w = [int(x) for x in words[o0 - int(r.offsets[0]):o0 - int(r.offsets[0]) + m]]
                bits = np.array([[a + j >= 0 and (x >> j) & 1 for j in range(min(64, m))] for x in w], dtype=bool).reshape(m, min(64, m))
                seen = (t < a)[None].repeat(m, 1)
                lo, hi = max(a, 0), min(L, a + min(64, m))
                if hi > lo:
                    seen[:, lo:hi] = torch.from_numpy(bits).to(dev)[:, lo - a:hi - a]
            seen = seen & there[None]
            for g in range(r.G):
                h = kvh * r.G + g
                q = r.q[o0:o0 + m, h].double()
                kz = torch.where(there[:, None], k, torch.zeros_like(k))
                z = torch.where(seen, (q @ kz.T) * scale, torch.full((m, L), -math.inf, dtype=torch.float64, device=dev))
                some = seen.any(1)
                if L == 0 or not bool(some.any()):
                    continue
                mx = torch.where(some, z.amax(1), torch.zeros(m, dtype=torch.float64, device=dev))
                p = torch.exp(z - mx[:, None])
                l = p.sum(1)
                w = torch.where(seen, p / l[:, None], torch.zeros_like(p))
                # only what is seen enters: a product of zero with NaN is not formed
                fin = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
                o = w @ fin
                bad = ~torch.isfinite(v)
                if bool(bad.any()):
                    for tt in torch.nonzero(bad.any(1)).flatten().tolist():
                        o += torch.where(seen[:, tt, None] & bad[None, tt], v[tt][None], torch.zeros_like(v[tt])[None])
                o = torch.where(some[:, None], o, torch.zeros_like(o))
                out[o0:o0 + m, h] = o
                lse[o0:o0 + m, h] = torch.where(some, mx + torch.log(l), torch.full_like(l, -math.inf))
                mag = (q.abs() @ torch.nan_to_num(kz, 0, 0, 0).abs().T * scale * seen).amax(1)
                dz = 128 * 2.0 ** -23 * mag + 2.0 ** -22 + 2.0 ** -22 * mx.abs()
                A = w @ fin.abs()
                tol[o0:o0 + m, h] = BF16 * torch.nan_to_num(o.abs(), 0, 0, 0) + (BF16 * 1.01 + 2 * dz[:, None]) * A + 1e-30
                tol_lse[o0:o0 + m, h] = dz + 2.0 ** -22 * lse[o0:o0 + m, h].abs() + L * 2.0 ** -24
    return {"out": out, "lse": lse, "tol": tol, "tol_lse": tol_lse}


def owned(r: Rows):
    m = torch.zeros(r.n_rows, dtype=torch.bool)
    m[int(r.offsets[0]):int(r.offsets[-1])] = True
    return m


def assert_within(got, ref, tol, what):
    got, ref, tol = got.double().cpu(), ref.cpu(), tol.cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: other values are finite ({int((torch.isfinite(got) != fin).sum())})"
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN elsewhere"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = (got - ref).abs()[fin]
    over = err > tol[fin]
    assert not bool(over.any()), f"{what}: {int(over.sum())} of {err.numel()} off, worst {float((err / tol[fin].clamp(min=1e-300)).max()):.2f} x the tolerance, err {float(err.max()):.3e}"


# ------------------------------------------------------------------ pages

def plan_pages(table, parent, keep, lens, num_pages):
    """(table_out, copies [(src, dst)], copies, free pages left), by the definition."""
    B, mpp = table.shape
    parent, keep = list(parent), list(keep)
    for b in range(B):
        if not (-1 <= parent[b] < B and 0 <= keep[b] <= mpp * P and lens[b] <= mpp * P):
            parent[b], keep[b] = -1, 0
            lens = [0 if i == b else x for i, x in enumerate(lens)]
        if parent[b] < 0:
            keep[b] = 0
    room = [max(a, b) for a, b in zip(lens, keep)]
    rows = [[int(x) if 0 <= x < num_pages else -1 for x in table[parent[b], :-(-keep[b] // P)]] if parent[b] >= 0 else [] for b in range(B)]
    holders = {}
    for b, r in enumerate(rows):
        for p in r:
            holders[p] = holders.get(p, 0) + 1
    writes = [keep[b] % P != 0 and room[b] > keep[b] for b in range(B)]
    writers = {}
    for b in range(B):
        if writes[b]:
            writers.setdefault(rows[b][-1], []).append(b)
    free = [p for p in range(num_pages) if p not in holders]
    n_free, taken = len(free), 0
    out = np.full((B, mpp), -1, np.int64)
    copies = []

    def take():
        nonlocal taken
        taken += 1
        return free[taken - 1] if taken <= n_free else -1

    for b in range(B):
        r = list(rows[b])
        if writes[b] and r[-1] >= 0:
            page = r[-1]
            if not (len(writers[page]) == holders[page] and min(writers[page]) == b):
                r[-1] = take()
                copies.append((page, r[-1]))
        r += [take() for _ in range(-(-room[b] // P) - len(r))]
        out[b, :len(r)] = r
    return out, copies, n_free - taken


def compact_pages(table, lens, num_pages):
    B, mpp = table.shape
    lens = [x if 0 <= x <= mpp * P else 0 for x in lens]
    rows = [[int(x) if 0 <= x < num_pages else -1 for x in table[b, :-(-lens[b] // P)]] for b in range(B)]
    live = sorted({p for r in rows for p in r if p >= 0})
    n = len(live)
    src = [p for p in live if p >= n]
    dst = sorted(set(range(n)) - set(live))
    to = dict(zip(src, dst))
    out = np.full((B, mpp), -1, np.int64)
    for b, r in enumerate(rows):
        out[b, :len(r)] = [to.get(p, p) for p in r]
    return out, list(zip(src, dst)), n
