"""Plain references for the calls with selected blocks of packed rows: the
canonical scores and their top-k in 32 bits, step by step, and the attention
over what a row sees in 64 bits."""
import math

import numpy as np
import torch

from sparse_decode_attention_head_gb300 import sa
from tests import rows_ref as R

D, P = 128, 16


def problem(r, bs, k, S, W, kcap=None, mode=sa.SUMMARY_MINMAX, selection=sa.SELECT_PER_HEAD):
    ks = [k] * r.Hq if isinstance(k, int) else list(k)
    return sa.Problem(B=r.B, Hq=r.Hq, Hk=r.Hk, max_pages_per_seq=r.mpp, num_pages=r.k_pool.shape[0], sink=S, window=W,
                      block_sizes=[bs] * r.Hk if isinstance(bs, int) else list(bs), k_per_head=ks,
                      kcap=kcap or max(1, max(ks)), mode=mode, selection=selection)


def candidates(prob, kvh, p):
    """Candidate blocks [j0, j1) of a row at position p."""
    size = prob.block_sizes[kvh]
    L = p + 1
    s_end = min(L, prob.sink)
    w_beg = max(L - prob.window, s_end)
    if w_beg <= s_end:
        return 0, 0
    return s_end // size, min(-(-w_beg // size), -(-prob.max_pages_per_seq * P // size))


def scores(q, summ, minmax):
    """[blocks] canonical fp32 scores of one query row (numpy float32)."""
    q = q.astype(np.float32)
    x = summ.astype(np.float32)
    x = np.where(q >= 0, x[:, 1], x[:, 0]) if minmax else x
    t = (q[None] * x).reshape(-1, 8, 16)
    acc = t[..., 0].copy()
    for d in range(1, 16):
        acc = acc + t[..., d]
    acc = acc[:, :4] + acc[:, 4:]
    acc = acc[:, :2] + acc[:, 2:]
    return acc[:, 0] + acc[:, 1] + np.float32(0)


def select(r, prob, summaries):
    """{(row, head): ascending list} by the definition."""
    out = {}
    q, summ = r.q.float().cpu().numpy(), summaries.float().cpu().numpy()
    minmax, group = prob.mode == sa.SUMMARY_MINMAX, prob.selection == sa.SELECT_GROUP
    off, lens = r.offsets.tolist(), r.lens.tolist()
    for b in range(r.B):
        for row in range(off[b], off[b + 1]):
            p = lens[b] - (off[b + 1] - row)
            for kvh in range(r.Hk):
                j0, j1 = candidates(prob, kvh, p)
                z = [scores(q[row, kvh * r.G + g], summ[b, kvh, j0:j1], minmax) for g in range(r.G)] if j1 > j0 else [np.zeros(0)] * r.G
                if group:
                    total = z[0]
                    for g in range(1, r.G):
                        total = total + z[g]
                    z = [total] * r.G
                for g in range(r.G):
                    h = kvh * r.G + g
                    order = np.argsort(-z[g], kind="stable")[:prob.k_per_head[h]]
                    out[row, h] = sorted(int(j) + j0 for j in order)
    return out


def lists(r, prob, seed=0, extra=0.0):
    """Random ascending lists within the budgets; extra: the share of entries that the call ignores."""
    rng = np.random.RandomState(seed)
    idx = np.full((r.n_rows, r.Hq, prob.kcap), 2 ** 31 - 1, np.int64)
    cnt = np.zeros((r.n_rows, r.Hq), np.int64)
    off, lens = r.offsets.tolist(), r.lens.tolist()
    for b in range(r.B):
        for row in range(off[b], off[b + 1]):
            p = lens[b] - (off[b + 1] - row)
            for h in range(r.Hq):
                size = prob.block_sizes[h // r.G]
                j0, j1 = candidates(prob, h // r.G, p)
                n = min(int(rng.randint(0, prob.k_per_head[h] + 1)), j1 - j0)
                got = list(rng.choice(np.arange(j0, j1), n, replace=False)) if n else []
                if extra and rng.rand() < extra:     # in sinks or window, behind the row, twice, below zero
                    got += [int(rng.randint(-3, (p + 200) // size + 2)) for _ in range(min(3, prob.kcap - n))] + got[:1]
                    got = got[:prob.kcap]
                idx[row, h, :len(got)] = sorted(got)
                cnt[row, h] = len(got)
    dev = r.q.device
    return torch.from_numpy(idx).int().to(dev), torch.from_numpy(cnt).int().to(dev)


def attention(r, prob, idx, cnt):
    """As rows_ref.attention (tolerances too), over what each row and head sees."""
    n, dev = r.n_rows, r.q.device
    out = torch.zeros(n, r.Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((n, r.Hq), -math.inf, dtype=torch.float64, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(r.B):
        o0, o1 = int(r.offsets[b]), int(r.offsets[b + 1])
        m = o1 - o0
        if m == 0:
            continue
        a = int(r.lens[b]) - m
        for kvh in range(r.Hk):
            k, v, there = r.kv(b, kvh)
            L, size = k.shape[0], prob.block_sizes[kvh]
            if L == 0:
                continue
            t = torch.arange(L, device=dev)
            p = a + torch.arange(m, device=dev)[:, None]
            for g in range(r.G):
                h = kvh * r.G + g
                e = idx[o0:o1, h].long()
                ok = (torch.arange(prob.kcap, device=dev)[None] < cnt[o0:o1, h, None]) & (e >= 0) & (e <= (L - 1) // size)
                block = torch.zeros(m, (L - 1) // size + 2, dtype=torch.bool, device=dev)
                block.scatter_(1, torch.where(ok, e, torch.full_like(e, (L - 1) // size + 1)), True)
                seen = (block[:, t // size] | (t < prob.sink) | (t > p - prob.window)) & (t <= p) & there[None]
                q = r.q[o0:o1, h].double()
                kz = torch.where(there[:, None], k, torch.zeros_like(k))
                z = torch.where(seen, (q @ kz.T) * prob.scale, torch.full((m, L), -math.inf, dtype=torch.float64, device=dev))
                some = seen.any(1)
                if not bool(some.any()):
                    continue
                mx = torch.where(some, z.amax(1), torch.zeros(m, dtype=torch.float64, device=dev))
                w = torch.exp(z - mx[:, None])
                l = w.sum(1)
                w = torch.where(seen, w / l[:, None], torch.zeros_like(w))
                fin = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
                o = w @ fin
                for tt in torch.nonzero((~torch.isfinite(v)).any(1)).flatten().tolist():
                    bad = ~torch.isfinite(v[tt])
                    o += torch.where(seen[:, tt, None] & bad[None], v[tt][None], torch.zeros_like(v[tt])[None])
                o = torch.where(some[:, None], o, torch.zeros_like(o))
                out[o0:o1, h] = o
                lse[o0:o1, h] = torch.where(some, mx + torch.log(l), torch.full_like(l, -math.inf))
                # as in rows_ref.attention: one rounding of the result and one of each weight to bf16, scores in fp32
                mag = (q.abs() @ torch.nan_to_num(kz, 0, 0, 0).abs().T * prob.scale * seen).amax(1)
                dz = 128 * 2.0 ** -23 * mag + 2.0 ** -22 + 2.0 ** -22 * mx.abs()
                A = w @ fin.abs()
                tol[o0:o1, h] = R.BF16 * torch.nan_to_num(o.abs(), 0, 0, 0) + (R.BF16 * 1.01 + 2 * dz[:, None]) * A + 1e-30
                tol_lse[o0:o1, h] = dz + 2.0 ** -22 * lse[o0:o1, h].abs() + L * 2.0 ** -24
    return {"out": out, "lse": lse, "tol": tol, "tol_lse": tol_lse}
