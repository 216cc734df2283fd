"""Attention of many rows that reads less than all of the cache, as it is measured: a prefix that several sequences
hold in the same pages, found in the page table and read once for all of them; blocks selected for each row by their
summaries, and the attention over them.

Each case is a dict of plain values.  `run` makes the calls of the library where `own` is true and computes the same
thing with elementary torch operations in 32 bits where it is false.
"""
import math

import numpy as np
import torch

own = False

D = 128   # head dim
P = 16    # tokens in a page


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a step of beam search, 8 prompts of 8 beams: what each prompt's beams share, from the page table
        {"name": "prefix_beams", "op": "prefixes", "groups": "8,8,8,8,8,8,8,8", "prefix": "8000,7500,4010,6000,7999,5003,8000,6500",
         "lo": 60, "hi": 90, "rows": 1},
        # a large batch behind 16 system prompts of up to 32K
        {"name": "prefix_batch", "op": "prefixes", "groups": ",".join(["64"] * 16),
         "prefix": "32768,20001,9999,16000,31,32000,12345,8192,30000,1024,25007,65,17000,4097,22222,28000", "lo": 1, "hi": 2000, "rows": 1},
        # four beams of one prompt of a small layer: latency
        {"name": "shared_small", "op": "shared", "Hq": 8, "Hk": 2, "groups": "4", "prefix": "4000", "lo": 20, "hi": 90, "rows": 1, "tree": False},
        # a step of beam search: 8 prompts of 8 beams each, a few generated tokens behind
        {"name": "shared_beams", "op": "shared", "Hq": 32, "Hk": 8, "groups": "8,8,8,8,8,8,8,8", "prefix": "8000,7500,4010,6000,7999,5003,8000,6500",
         "lo": 60, "hi": 90, "rows": 1, "tree": False},
        # 128 conversations behind one system prompt of 32K, ragged
        {"name": "shared_system", "op": "shared", "Hq": 32, "Hk": 8, "groups": "128", "prefix": "32768", "lo": 1, "hi": 2000, "rows": 1, "tree": False},
        # drafted trees of up to 32 tokens for samples of a few documents, some sequences alone, seven heads to a group
        {"name": "shared_trees", "op": "shared", "Hq": 28, "Hk": 4, "groups": "6,1,12,1,8,5", "prefix": "30000,777,16411,12345,8192,25000",
         "lo": 0, "hi": 700, "rows": 32, "tree": True},
        # eight sequences of 32K with eight drafted tokens in a row each, 5 % of the blocks for every head
        {"name": "select_draft", "op": "select", "Hq": 32, "Hk": 8, "rows": "8,8,8,8,8,8,8,8", "prefix": "32760,32760,32760,32760,32760,32760,32760,32760",
         "bs": "16,16,16,16,16,16,16,16", "k": 100, "sink": 4, "window": 1024, "mode": "minmax", "group": False},
        # packed prompts, some behind a prefix, each KV head with its block size, selected for a group of seven heads together
        {"name": "select_packed", "op": "select", "Hq": 28, "Hk": 4, "rows": "4099,1,977,2048,517,63", "prefix": "0,4095,31,0,9024,7",
         "bs": "16,32,64,8", "k": 24, "sink": 3, "window": 200, "mode": "mean", "group": True},
        # one long prompt
        {"name": "select_16k", "op": "select", "Hq": 32, "Hk": 8, "rows": "16384", "prefix": "0", "bs": "64,64,64,64,64,64,64,64",
         "k": 16, "sink": 4, "window": 512, "mode": "minmax", "group": False},
        # the drafted rows of eight sequences of 32K over their selected blocks
        {"name": "sparse_draft", "op": "sparse", "Hq": 32, "Hk": 8, "rows": "8,8,8,8,8,8,8,8", "prefix": "32760,32760,32760,32760,32760,32760,32760,32760",
         "bs": "16,16,16,16,16,16,16,16", "k": 100, "sink": 4, "window": 1024},
        # packed prompts, some behind a prefix, each KV head with its block size, seven heads to a group
        {"name": "sparse_packed", "op": "sparse", "Hq": 28, "Hk": 4, "rows": "4099,1,977,2048,517,63", "prefix": "0,4095,31,0,9024,7",
         "bs": "16,32,64,8", "k": 24, "sink": 3, "window": 200},
        # one long prompt of 32K, 16 blocks of 64 and a window of 512 for every row
        {"name": "sparse_32k", "op": "sparse", "Hq": 32, "Hk": 8, "rows": "32768", "prefix": "0", "bs": "64,64,64,64,64,64,64,64",
         "k": 16, "sink": 4, "window": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(v):
    return ",".join(str(int(x)) for x in v)


def draw(rng):
    op = rng.choice(("prefixes", "shared", "shared", "select", "select", "sparse", "sparse"))
    Hq, Hk = rng.choice(((8, 2), (32, 8), (28, 4), (8, 8), (16, 8), (20, 4), (24, 4), (8, 1)))
    if op in ("prefixes", "shared"):
        n = _log(rng, 1, 12)
        groups = [_log(rng, 1, 80 // n + 1) for _ in range(n)]
        prefix = [_log(rng, 1, 24000) - 1 for _ in groups]
        if op == "prefixes":   # something to find
            groups[:1], prefix[:1] = [groups[0] + 1, 2], [_log(rng, 4000, 24000), _log(rng, 4000, 24000)]
        c = {"op": op, "groups": _text(groups), "prefix": _text(prefix), "lo": rng.randint(0, 40),
             "hi": 40 + _log(rng, 1, 1500), "rows": rng.choice((1, 1, rng.randint(2, 32)))}
        if op == "shared":
            c.update(Hq=Hq, Hk=Hk, tree=c["rows"] > 1 and rng.random() < 0.6)
        return c
    if rng.random() < 0.5:   # drafts and single tokens over long caches
        n = _log(rng, 1, 12)
        rows, prefix = [rng.randint(1, 32) for _ in range(n)], [_log(rng, 1, 60000) - 1 for _ in range(n)]
    else:                    # prompts
        n = rng.randint(1, 6)
        rows, prefix = [_log(rng, 1, 9000 // n) for _ in range(n)], [rng.choice((0, _log(rng, 1, 8000))) for _ in range(n)]
    window, bs, k = rng.choice((64, 128, 500, 1024)), [rng.choice((8, 16, 32, 64)) for _ in range(Hk)], _log(rng, 1, 128)
    if op == "select":   # a choice to make: some row has twice as many candidates as it keeps
        prefix[0] = max(prefix[0], 2000)
        k = min(k, (prefix[0] - window - 64) // max(bs) // 2)
    c = {"op": op, "Hq": Hq, "Hk": Hk, "rows": _text(rows), "prefix": _text(prefix), "bs": _text(bs),
         "k": k, "sink": rng.choice((0, 1, 4, 16, 37)), "window": window}
    if op == "select":
        c.update(mode=rng.choice(("minmax", "mean")), group=rng.random() < 0.3)
    return c


def _ints(text):
    return [int(x) for x in str(text).split(",")]


def _sequences(case):
    """(tokens ahead of the rows, rows) of every sequence, and each one's group."""
    if case["op"] in ("select", "sparse"):
        rows, prefix = _ints(case["rows"]), _ints(case["prefix"])
        return prefix, rows, list(range(len(rows)))
    ahead, rows, group = [], [], []
    for g, (m, p) in enumerate(zip(_ints(case["groups"]), _ints(case["prefix"]))):
        for _ in range(m):
            b = len(ahead)
            ahead.append(p + case["lo"] + b * 37 % (case["hi"] - case["lo"] + 1))
            rows.append(case["rows"] if not case.get("tree") else 1 + (b * 7 + 3) % case["rows"])
            group.append(g)
    return ahead, rows, group


# ------------------------------------------------------------------ inputs

def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    ahead, rows, group = _sequences(case)
    lens = [a + n for a, n in zip(ahead, rows)]
    B, n = len(rows), sum(rows)
    used = [-(-L // P) for L in lens]
    mpp = max(1, max(used))
    # what a group shares lies in the same pages; everything else, scattered over the pool, is a sequence's own
    rng = np.random.RandomState(int(seed) % (1 << 31))
    common = [p // P for p in _ints(case["prefix"])] if op in ("prefixes", "shared") else [0] * B
    if op == "prefixes":   # where beams or prompts part is for the call to find
        common = [c - int(rng.randint(0, c // 2 + 1)) for c in common]
    pool = sum(u - common[group[b]] for b, u in enumerate(used)) + sum(common) + 5
    perm = rng.permutation(pool).astype(np.int32)
    table = np.full((B, mpp), -1, np.int32)
    at, prefix_pages = 0, {}
    for b in range(B):
        c = common[group[b]]
        if group[b] not in prefix_pages:
            prefix_pages[group[b]] = perm[at:at + c]
            at += c
        table[b, :c] = prefix_pages[group[b]]
        table[b, c:used[b]] = perm[at:at + used[b] - c]
        at += used[b] - c
    s = {"case": case, "op": op, "B": B, "pool": pool, "table": torch.from_numpy(table).cuda(), "lens": _int32(lens),
         "offsets": _int32(np.concatenate([[0], np.cumsum(rows)]).tolist())}
    if op == "prefixes":
        s["group_offsets"] = _int32(np.concatenate([[0], np.cumsum(_ints(case["groups"]))]).tolist())
        s["members"], s["prefix_lens"] = (torch.full((B,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        return s
    Hq, Hk = case["Hq"], case["Hk"]
    G = Hq // Hk
    # neighbouring rows look for the same things: a direction that drifts along a sequence, and a part of each row's own
    way = randn(B, Hk, D)[torch.tensor(group, device="cuda")]
    b_of = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(rows, device="cuda"), output_size=n)
    drift = randn(n // 64 + 1, Hk, D)[torch.arange(n, device="cuda") // 64]
    q = 0.7 * randn(n, Hk, G, D) + 0.5 * (way[b_of] + drift)[:, :, None]
    s["q"] = q.to(torch.bfloat16).view(n, Hq, D)
    if op == "select":
        s.update(_summaries(case, randn, way, lens, mpp))
        k = case["k"]
        s["sel_idx"] = torch.full((n, Hq, k), -1, dtype=torch.int32, device="cuda")
        s["sel_cnt"] = torch.full((n, Hq), -1, dtype=torch.int32, device="cuda")
        return s
    s["k_pool"], s["v_pool"] = (randn(pool, Hk, P, D).to(torch.bfloat16) for _ in range(2))
    first = s["table"][:, 0].long()   # the first token of a sequence draws attention
    s["k_pool"][first, :, 0] = (s["k_pool"][first, :, 0].float() + way).to(torch.bfloat16)
    s["out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(n, Hq, device="cuda")
    if op == "sparse":
        s["sel_idx"], s["sel_cnt"] = _selection(case, g)
        return s
    # what the prefixes call answers for these sequences: whole pages that two or more sequences share
    members, prefix_lens = [0] * B, [0] * B
    for b in range(B):
        m = group.count(group[b])
        if m > 1:
            prefix_lens[b] = common[group[b]] * P
            if prefix_lens[b] and group.index(group[b]) == b:
                members[b] = m
    s["members"], s["prefix_lens"] = _int32(members), _int32(prefix_lens)
    if case["tree"]:
        # every node hangs on a random earlier one (or on the last token of the cache): its word has its ancestors' bits and its own
        words = []
        for m in rows:
            up = []
            for i in range(m):
                parent = int(rng.randint(max(-1, i // 2 - 4), i)) if i else -1
                up.append((up[parent] if parent >= 0 else 0) | 1 << i)
            words += up
        s["mask"] = torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).cuda()
    return s


def _slots(case, mpp):
    return -(-mpp * P // min(_ints(case["bs"])))


def _summaries(case, randn, way, lens, mpp):
    """Block summaries of random keys, block by block as the cache has them; places without a block hold zeros."""
    bs, minmax = _ints(case["bs"]), case["mode"] == "minmax"
    out = torch.zeros(len(lens), case["Hk"], _slots(case, mpp), *((2, D) if minmax else (D,)), dtype=torch.bfloat16, device="cuda")
    for b, L in enumerate(lens):
        for kvh, size in enumerate(bs):
            nb = -(-L // size)
            k = randn(nb, size, D).to(torch.bfloat16)
            k[0, 0] = (k[0, 0].float() + way[b, kvh]).to(torch.bfloat16)
            # some blocks have what the sequence is about
            k += (0.5 * way[b, kvh] * (randn(nb, 1, 1) > 1.5)).to(torch.bfloat16)
            if minmax:
                out[b, kvh, :nb, 0], out[b, kvh, :nb, 1] = k.amin(1), k.amax(1)
            else:
                out[b, kvh, :nb] = k.float().mean(1).to(torch.bfloat16)
    return {"summaries": out}


def _candidates(case, size, p):
    """First and last + 1 candidate block of a row at position p (a tensor): those that meet the tokens between sink and window."""
    L = p + 1
    s_end = torch.clamp(L, max=case["sink"])
    w_beg = torch.maximum(L - case["window"], s_end)
    some = w_beg > s_end
    zero = torch.zeros_like(L)
    return torch.where(some, s_end // size, zero), torch.where(some, (w_beg + size - 1) // size, zero)


def _selection(case, g):
    """Lists of selected blocks as prompts and drafts have them: what a KV head looks for changes every 64 rows, its heads
    agree on most of it, and a row differs from its neighbours in some."""
    ahead, rows, _ = _sequences(case)
    Hq, Hk, k, bs = case["Hq"], case["Hk"], case["k"], _ints(case["bs"])
    G = Hq // Hk
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    idx, cnt = [], []
    for a, n in zip(ahead, rows):
        si = torch.full((n, Hk, G, k), -1, dtype=torch.int32, device="cuda")
        sc = torch.zeros(n, Hk, G, dtype=torch.int32, device="cuda")
        p = a + torch.arange(n, device="cuda")
        seg = (p - p[0]) // 64
        for kvh, size in enumerate(bs):
            j0, j1 = _candidates(case, size, p)
            nb = int(j1[-1])
            if nb == 0:
                continue
            topic = 1.5 * randn(int(seg[-1]) + 1, 1, nb) + 0.8 * randn(int(seg[-1]) + 1, G, nb)
            for i0 in range(0, n, 4096):
                i1 = min(n, i0 + 4096)
                score = topic[seg[i0:i1]] + 0.8 * randn(i1 - i0, G, nb)
                at = torch.arange(nb, device="cuda")
                score.masked_fill_(((at < j0[i0:i1, None]) | (at >= j1[i0:i1, None]))[:, None], -math.inf)
                val, ind = torch.topk(score, min(k, nb), dim=-1)
                ind = torch.where(torch.isinf(val), torch.full_like(ind, 1 << 30), ind).sort(-1).values
                si[i0:i1, kvh, :, :ind.shape[-1]] = torch.where(ind < 1 << 30, ind, torch.full_like(ind, -1)).int()
                sc[i0:i1, kvh] = (ind < 1 << 30).sum(-1).int()
        idx.append(si.view(n, Hq, k))
        cnt.append(sc.view(n, Hq))
    return torch.cat(idx), torch.cat(cnt)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from sparse_decode_attention_head_gb300 import sa
        Hk, Hq = case.get("Hk", 1), case.get("Hq", 1)
        B, mpp = s["table"].shape
        s["prob"] = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=mpp, num_pages=s["pool"], sink=case.get("sink", 4), window=case.get("window", 64),
                               block_sizes=_ints(case.get("bs", _text([P] * Hk))), k_per_head=[case.get("k", 1)] * Hq, kcap=case.get("k", 1),
                               mode=sa.SUMMARY_MEAN if case.get("mode") == "mean" else sa.SUMMARY_MINMAX,
                               selection=sa.SELECT_GROUP if case.get("group") else sa.SELECT_PER_HEAD)
        s["ws"] = sa.Workspace(s["prob"], rows=True, max_rows=int(s["offsets"][-1]))
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_prefixes(s):
    table, go = s["table"], s["group_offsets"].long()
    B, mpp = table.shape
    n_groups = go.numel() - 1
    b = torch.arange(B, device="cuda")
    g = torch.searchsorted(go, b, right=True) - 1
    first = go[g]
    ahead = (s["lens"] - (s["offsets"][1:] - s["offsets"][:-1])).long()
    at = torch.arange(mpp, device="cuda")
    same = (table == table[first]) & (table >= 0) & (table < s["pool"]) & ((at + 1) * P <= ahead[:, None])
    run_ = torch.where(same, torch.full_like(table, mpp), at.int()[None].expand_as(table)).amin(1).long()   # leading pages that are the first's
    least = torch.full((n_groups,), mpp, dtype=torch.int64, device="cuda").scatter_reduce_(0, g, run_, "amin")
    size = go[1:] - go[:-1]
    prefix = torch.where(size > 1, least * P, torch.zeros_like(least))[g]
    members = torch.where((b == first) & (prefix > 0), size[g], torch.zeros_like(b))
    return {"members": members.int(), "prefix_lens": prefix.int()}


def _plain_shared(s):
    """Every sequence over the whole of its own cache: that the prefix is shared changes nothing in the result."""
    c = s["case"]
    Hq, Hk = c["Hq"], c["Hk"]
    ahead, rows, _ = _sequences(c)
    G, N = Hq // Hk, max(rows)
    n = s["q"].shape[0]
    out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, Hq, device="cuda")
    step = max(1, (1 << 32) // (s["table"].shape[1] * P * Hk * D * 4))
    for b0 in range(0, len(rows), step):
        b1 = min(len(rows), b0 + step)
        B = b1 - b0
        o0, o1 = sum(rows[:b0]), sum(rows[:b1])
        off = s["offsets"][b0:b1 + 1].long() - o0
        at = torch.arange(o1 - o0, device="cuda")
        b = torch.searchsorted(off, at, right=True) - 1
        i = at - off[b]
        q = torch.zeros(B, N, Hq, D, device="cuda")
        q[b, i] = s["q"][o0:o1].float()
        q = q.view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
        L = -(-max(ahead[x] + rows[x] for x in range(b0, b1)) // P) * P
        table = s["table"][b0:b1, :L // P].long().clamp(min=0)
        k = s["k_pool"][table].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D).float()
        z = torch.matmul(q, k.transpose(-1, -2)).view(B, Hk, G, N, L)
        del k
        z *= 1.0 / math.sqrt(D)
        col = torch.arange(L, device="cuda")
        before = (s["lens"][b0:b1].long() - (off[1:] - off[:-1]))
        if not c["tree"]:
            seen = col[None, None] <= (before[:, None] + torch.arange(N, device="cuda"))[:, :, None]
        else:
            word = torch.zeros(B, N, dtype=torch.int64, device="cuda")
            word[b, i] = s["mask"][o0:o1]
            bit = col[None] - before[:, None]
            draft = (bit >= 0) & (col[None] < s["lens"][b0:b1, None])
            seen = (bit < 0)[:, None] | (draft[:, None] & ((word[:, :, None] >> bit.clamp(0, 63)[:, None]) & 1).bool())
        z.masked_fill_(~seen[:, None, None], -math.inf)
        m = z.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)   # places without a row
        z.sub_(m).exp_()
        total = z.sum(-1, keepdim=True)
        v = s["v_pool"][table].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D).float()
        o = torch.matmul(z.view(B, Hk, G * N, L), v).view(B, Hk, G, N, D) / total
        out[o0:o1] = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[b, i].to(torch.bfloat16)
        lse[o0:o1] = (m + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, N, Hq)[b, i]
    return {"out": out, "lse": lse}


def _row_scores(case, q, summ):
    """Scores [rows][heads][blocks] of one KV head's summaries in the order that the decode step's scores have: 8 lanes of 16
    neighbouring dims, each summed upwards (products of bf16 are exact in 32 bits), and the lanes joined 4, 2 and 1 apart."""
    q = q.float().view(q.shape[0], q.shape[1], 1, 8, 16)
    acc = None
    for d in range(16):
        x = q[..., d]
        if case["mode"] == "minmax":
            lo, hi = summ[:, 0].float().view(-1, 8, 16)[..., d], summ[:, 1].float().view(-1, 8, 16)[..., d]
            t = x * torch.where(x >= 0, hi, lo)
        else:
            t = x * summ.float().view(-1, 8, 16)[..., d]
        acc = t if acc is None else acc.add_(t)
    acc = acc[..., :4] + acc[..., 4:]
    acc = acc[..., :2] + acc[..., 2:]
    return acc[..., 0] + acc[..., 1] + 0.0


def _plain_select(s):
    c = s["case"]
    ahead, rows, _ = _sequences(c)
    Hq, Hk, k, bs = c["Hq"], c["Hk"], c["k"], _ints(c["bs"])
    G, at = Hq // Hk, 0
    for b, (a, n) in enumerate(zip(ahead, rows)):
        p = a + torch.arange(n, device="cuda")
        for kvh, size in enumerate(bs):
            j0, j1 = _candidates(c, size, p)
            nb = int(_candidates(c, size, torch.tensor(a + n - 1))[1])
            step = max(1, (1 << 28) // (G * max(nb, 1) * 8))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                r = slice(at + i0, at + i1)
                heads = slice(kvh * G, (kvh + 1) * G)
                ncand = (j1 - j0)[i0:i1]
                want = ncand.clamp(max=k)
                s["sel_cnt"][r, heads] = want[:, None].int()
                if nb == 0:
                    continue
                z = _row_scores(c, s["q"][r, heads], s["summaries"][b, kvh, :nb])
                if c["group"]:
                    total = z[:, 0]
                    for h in range(1, G):
                        total = total + z[:, h]
                    z = total[:, None].expand_as(z)
                col = torch.arange(nb, device="cuda")
                z = z.masked_fill(((col < j0[i0:i1, None]) | (col >= j1[i0:i1, None]))[:, None], -math.inf)
                order = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :k]   # ties go to the lowest index
                rank = torch.arange(order.shape[-1], device="cuda")
                ok = rank < want[:, None, None]
                got = torch.where(ok, order, torch.full_like(order, 1 << 30)).sort(-1).values
                old = s["sel_idx"][r, heads, :order.shape[-1]]
                s["sel_idx"][r, heads, :order.shape[-1]] = torch.where(ok.expand_as(got), got.int(), old)
        at += n
    return {"sel_idx": s["sel_idx"], "sel_cnt": s["sel_cnt"]}


def _plain_sparse(s):
    c = s["case"]
    ahead, rows, _ = _sequences(c)
    Hq, Hk, bs = c["Hq"], c["Hk"], _ints(c["bs"])
    G, at, n = Hq // Hk, 0, s["q"].shape[0]
    out = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, Hq, device="cuda")
    rank = torch.arange(s["sel_idx"].shape[-1], device="cuda")
    for b, (a, m) in enumerate(zip(ahead, rows)):
        for i0 in range(0, m, 2048):
            i1 = min(m, i0 + 2048)
            L = a + i1     # later positions are seen by none of these rows
            r = slice(at + i0, at + i1)
            p = a + torch.arange(i0, i1, device="cuda")
            page = s["table"][b, :-(-L // P)].long()
            t = torch.arange(L, device="cuda")
            upto = t <= p[:, None]
            dense = upto & ((t < c["sink"]) | (t > p[:, None] - c["window"]))
            for kvh, size in enumerate(bs):
                heads = slice(kvh * G, (kvh + 1) * G)
                nb = -(-L // size)
                sel = s["sel_idx"][r, heads].long()
                ok = rank < s["sel_cnt"][r, heads, None]
                block = torch.zeros(i1 - i0, G, nb + 1, dtype=torch.bool, device="cuda")
                block.scatter_(2, torch.where(ok & (sel < nb), sel, torch.full_like(sel, nb)), True)
                seen = block[..., :nb].repeat_interleave(size, -1)[..., :L]
                seen &= upto[:, None]
                seen |= dense[:, None]
                k = s["k_pool"][page, kvh].reshape(-1, D)[:L].float()
                v = s["v_pool"][page, kvh].reshape(-1, D)[:L].float()
                z = torch.matmul(s["q"][r, heads].float(), k.t())
                z *= 1.0 / math.sqrt(D)
                z.masked_fill_(~seen, -math.inf)
                top = z.amax(-1, keepdim=True)
                z.sub_(top).exp_()
                total = z.sum(-1, keepdim=True)
                out[r, heads] = (torch.matmul(z, v) / total).to(torch.bfloat16)
                lse[r, heads] = (top + torch.log(total))[..., 0]
        at += m
    return {"out": out, "lse": lse}


_PLAIN = {"prefixes": _plain_prefixes, "shared": _plain_shared, "select": _plain_select, "sparse": _plain_sparse}


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    from sparse_decode_attention_head_gb300 import sa
    p, ws, op = s["prob"], s["ws"], s["op"]
    if op == "prefixes":
        sa.shared_prefixes(p, s["table"], s["lens"], s["offsets"], s["group_offsets"], s["members"], s["prefix_lens"], ws)
        return {"members": s["members"], "prefix_lens": s["prefix_lens"]}
    if op == "select":
        sa.select_rows(p, s["q"], s["summaries"], s["lens"], s["offsets"], s["sel_idx"], s["sel_cnt"], ws)
        return {"sel_idx": s["sel_idx"], "sel_cnt": s["sel_cnt"]}
    if op == "shared":
        sa.shared_attention(p, s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["offsets"], s["members"], s["prefix_lens"], s["out"], ws,
                            lse=s["lse"], tree_mask=s.get("mask"))
    else:
        sa.sparse_row_attention(p, s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["offsets"], s["sel_idx"], s["sel_cnt"], s["out"], ws,
                                lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    ahead, rows, group = _sequences(case)
    n = sum(rows)
    if op in ("prefixes", "shared"):
        common = [p // P * P for p in _ints(case["prefix"])]   # at most, where the pages decide
        shared = [common[g] if group.count(g) > 1 else 0 for g in range(len(common))]
        if op == "prefixes":
            return {"bytes": 4 * sum(shared[g] // P for g in group) + 8 * len(rows), "flops": 0}
        Hq, Hk = case["Hq"], case["Hk"]
        cache = sum(shared) + sum(a + m - shared[g] for a, m, g in zip(ahead, rows, group))
        pairs = sum(m * a + m * (m + 1) // 2 for a, m in zip(ahead, rows))   # a tree's rows see at most the causal ones
        return {"bytes": cache * Hk * D * 4 + n * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}
    Hq, Hk, bs, k = case["Hq"], case["Hk"], _ints(case["bs"]), case["k"]
    S, W = case["sink"], case["window"]
    pairs, lists, least = 0, 0, 0
    for a, m in zip(ahead, rows):
        L = np.arange(a + 1, a + m + 1)
        s_end = np.minimum(L, S)
        w_beg = np.maximum(L - W, s_end)
        for size in bs:
            ncand = np.where(w_beg > s_end, -(-w_beg // size) - s_end // size, 0)
            lists += int(np.minimum(ncand, k).sum()) * Hq // Hk
            if op == "select":
                pairs += int(np.where(ncand > k, ncand, 0).sum()) * Hq // Hk
                least += int(ncand[-1]) if ncand[-1] > k else 0
            else:
                pairs += int((L - np.maximum(w_beg - s_end - k * size, 0)).sum()) * Hq // Hk
                least += int(min(a + m, (s_end + L - w_beg)[-1] + k * size + m))    # the rows of a sequence have at least the last one's tokens
    if op == "select":
        return {"bytes": n * Hq * (2 * D + 4) + 4 * lists + least * D * (4 if case["mode"] == "minmax" else 2), "flops": 2 * D * pairs}
    return {"bytes": n * Hq * (4 * D + 8) + 4 * lists + least * D * 4, "flops": 4 * D * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] in ("prefixes", "select"):
        return None   # whole numbers
    w = work(case)["flops"]
    if w > (6e12 if case["op"] == "shared" else 2e12):
        return None
    s = _inputs(case, seed)
    return _exact_shared(case, s) if case["op"] == "shared" else _exact_sparse(case, s)


def _exact_shared(case, s):
    """One sequence and KV head at a time, over the sequence's own row of the page table."""
    ahead, rows, _ = _sequences(case)
    Hq, Hk, at = case["Hq"], case["Hk"], 0
    G = Hq // Hk
    out = torch.zeros(sum(rows), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(rows), Hq, dtype=torch.float64, device="cuda")
    for b, (a, m) in enumerate(zip(ahead, rows)):
        t = torch.arange(a + m, device="cuda")
        page = s["table"][b].long()[t // P]
        k, v = s["k_pool"][page, :, t % P].double(), s["v_pool"][page, :, t % P].double()
        if case["tree"]:
            words = s["mask"][at:at + m].cpu().numpy().view(np.uint64)
            draft = np.array([[(int(w) >> j) & 1 for j in range(m)] for w in words], dtype=bool).reshape(m, m)
        else:
            draft = np.tril(np.ones((m, m), dtype=bool))
        seen = torch.cat([torch.ones(m, a, dtype=torch.bool, device="cuda"), torch.from_numpy(draft).cuda()], 1)
        for h in range(Hk):
            z = torch.einsum("mgd,td->mgt", s["q"][at:at + m, h * G:(h + 1) * G].double(), k[:, h]) / math.sqrt(D)
            z = torch.where(seen[:, None], z, torch.full_like(z, -math.inf))
            lse[at:at + m, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[at:at + m, h * G:(h + 1) * G] = torch.einsum("mgt,td->mgd", torch.softmax(z, -1), v[:, h])
        at += m
    return {"out": out, "lse": lse}


def _exact_sparse(case, s):
    """Some rows of one head at a time: the positions that each sees, listed, and their keys and values gathered."""
    ahead, rows, _ = _sequences(case)
    Hq, Hk, bs, S, W = case["Hq"], case["Hk"], _ints(case["bs"]), case["sink"], case["window"]
    out = torch.zeros(sum(rows), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(rows), Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (a, m) in enumerate(zip(ahead, rows)):
        for h in range(Hq):
            kvh = h * Hk // Hq
            size = bs[kvh]
            most = case["k"] * size + S + W
            step = max(1, (1 << 30) // (most * D * 8))
            for i0 in range(0, m, step):
                i1 = min(m, i0 + step)
                L = (a + 1 + torch.arange(i0, i1, device="cuda"))[:, None]
                s_end = torch.clamp(L, max=S)
                w_beg = torch.maximum(L - W, s_end)
                r = slice(at + i0, at + i1)
                listed_ = torch.arange(case["k"], device="cuda") < s["sel_cnt"][r, h, None]
                block = s["sel_idx"][r, h].long()
                tok = (block[..., None] * size + torch.arange(size, device="cuda")).flatten(1)
                ok = listed_.repeat_interleave(size, 1) & (tok >= s_end) & (tok < w_beg)
                sink = torch.arange(S, device="cuda").expand(i1 - i0, S)
                recent = w_beg + torch.arange(W, device="cuda")
                tok = torch.cat([tok, sink, recent], 1)
                ok = torch.cat([ok, sink < s_end, recent < L], 1)
                tok = torch.where(ok, tok, torch.zeros_like(tok))
                page = s["table"][b].long()[tok // P]
                k = s["k_pool"][page, kvh, tok % P].double()
                z = torch.einsum("id,itd->it", s["q"][r, h].double(), k) / math.sqrt(D)
                z = torch.where(ok, z, torch.full_like(z, -math.inf))
                lse[r, h] = torch.logsumexp(z, -1)
                out[r, h] = torch.einsum("it,itd->id", torch.softmax(z, -1), s["v_pool"][page, kvh, tok % P].double())
        at += m
    return {"out": out, "lse": lse}
