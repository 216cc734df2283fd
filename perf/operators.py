"""The operators around a decode step, as they are measured: rotation of packed rows into the cache, attention of a
prompt, attention of a tree of drafted tokens, and the bookkeeping of the cache's pages.

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
        # one decode step of a batch of eight at 32K: a row for each sequence, all latency
        {"name": "rotate_decode", "op": "rotate", "Hq": 32, "Hk": 8, "rows": "1,1,1,1,1,1,1,1",
         "prefix": "32767,32767,32767,32767,32767,32767,32767,32767", "norm": True, "axis_pairs": "64", "layout": "halves"},
        # prompts with images, positions of three axes (time, height, width), no norm, neighbouring pairs
        {"name": "rotate_axes", "op": "rotate", "Hq": 28, "Hk": 4, "rows": "4099,1,977,2048,517,63", "prefix": "0,65535,31,0,1024,7",
         "norm": False, "axis_pairs": "16,24,24", "layout": "pairs"},
        # a batch of eight prompts of 8K, norm and rotation
        {"name": "rotate_prompts", "op": "rotate", "Hq": 32, "Hk": 8, "rows": "8192,8192,8192,8192,8192,8192,8192,8192",
         "prefix": "0,0,0,0,0,0,0,0", "norm": True, "axis_pairs": "64", "layout": "halves"},
        # short questions of a small layer, ragged: latency
        {"name": "prompt_short", "op": "prompt", "Hq": 8, "Hk": 2, "rows": "200,1,33,97", "prefix": "0,0,0,0"},
        # packed prompts of different lengths, some behind a prefix that is in the cache already, seven heads to a group
        {"name": "prompt_packed", "op": "prompt", "Hq": 28, "Hk": 4, "rows": "4099,1,977,2048,517,63", "prefix": "0,4095,31,0,1024,7"},
        # one long prompt
        {"name": "prompt_16k", "op": "prompt", "Hq": 32, "Hk": 8, "rows": "16384", "prefix": "0"},
        # a tree of 16 drafted tokens of one sequence at 4K: latency
        {"name": "tree_4k", "op": "tree", "Hq": 8, "Hk": 2, "rows": "16", "prefix": "4080"},
        # 32 drafted tokens for each sequence of a batch of eight at 32K
        {"name": "tree_32k", "op": "tree", "Hq": 32, "Hk": 8, "rows": "32,32,32,32,32,32,32,32",
         "prefix": "32736,32736,32736,32736,32736,32736,32736,32736"},
        # a ragged batch of 16 up to 64K, drafts of 1 to 64 tokens, seven heads to a group
        {"name": "tree_ragged", "op": "tree", "Hq": 28, "Hk": 4, "rows": "1,5,64,33,8,8,1,17,12,25,3,64,7,1,16,40",
         "prefix": "65471,40001,65000,12345,33333,777,0,65519,50000,8191,60001,31999,64000,1,20011,47777"},
        # a step of beam search: 8 prompts of 8 beams, each beam goes on from one of its prompt's beams
        {"name": "pages_fork", "op": "fork", "Hk": 8, "prompts": 8, "beams": 8, "context": 8000, "generated": 77, "grow": 1, "spare": 2000},
        # a pool of 64K pages, half of them live and scattered, packed to its front
        {"name": "pages_compact", "op": "compact", "Hk": 8, "sequences": 32, "context": 16384, "pages": 65536},
        # 64 sequences take over the accepted rows of their trees
        {"name": "pages_accept", "op": "accept", "Hk": 8, "sequences": 64, "context": 4000, "nodes": 32, "most": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _text(v):
    return ",".join(str(int(x)) for x in v)


def draw(rng):
    op = rng.choice(("rotate", "rotate", "prompt", "prompt", "tree", "tree", "fork", "compact", "accept"))
    Hq, Hk = rng.choice(((8, 2), (32, 8), (28, 4), (8, 8), (16, 8), (20, 4), (24, 4), (8, 1)))
    if op == "rotate":
        n = rng.randint(1, 12)
        rows = [_log(rng, 1, 65536 // n) for _ in range(n)]
        pairs = rng.choice(((64,), (32,), (16,), (16, 24, 24), (8, 12, 12), (20, 30)))
        return {"op": op, "Hq": Hq, "Hk": Hk, "rows": _text(rows), "prefix": _text(rng.choice((0, _log(rng, 1, 100000))) for _ in rows),
                "norm": rng.random() < 0.6, "axis_pairs": _text(pairs), "layout": rng.choice(("halves", "pairs"))}
    if op == "prompt":
        n = rng.randint(1, 6)
        rows = [_log(rng, 1, 4096) for _ in range(n)]
        return {"op": op, "Hq": Hq, "Hk": Hk, "rows": _text(rows), "prefix": _text(rng.choice((0, _log(rng, 1, 2048))) for _ in rows)}
    if op == "tree":
        n = _log(rng, 1, 16)
        rows = [rng.randint(1, 64) for _ in range(n)]
        return {"op": op, "Hq": Hq, "Hk": Hk, "rows": _text(rows), "prefix": _text(_log(rng, 1, 32000) - 1 for _ in rows)}
    if op == "fork":
        return {"op": op, "Hk": Hk, "prompts": _log(rng, 1, 16), "beams": rng.randint(1, 8), "context": _log(rng, 1, 16000),
                "generated": _log(rng, 1, 300), "grow": _log(rng, 1, 64), "spare": _log(rng, 1, 2000)}
    if op == "compact":
        n = _log(rng, 1, 32)
        context = _log(rng, 16, 16000)
        return {"op": op, "Hk": Hk, "sequences": n, "context": context, "pages": int(n * (context // P + 1) * rng.uniform(1.05, 2.0)) + 1}
    nodes = rng.randint(2, 64)
    return {"op": op, "Hk": Hk, "sequences": _log(rng, 1, 128), "context": _log(rng, 1, 8000), "nodes": nodes, "most": rng.randint(1, max(1, nodes // 3))}


def _ints(text):
    return [int(x) for x in str(text).split(",")]


# ------------------------------------------------------------------ inputs

def _page_table(g, lens, extra, longest=None):
    """A table over a pool with `extra` more pages than the sequences need (or would, were each `longest`): a random permutation of the pool."""
    need = [max(1, -(-L // P)) for L in lens]
    room = [max(1, -(-(longest or L) // P)) for L in lens]
    mpp, pool = max(room), sum(room) + extra
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), mpp), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pool


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(rows):
    return _int32(np.concatenate([[0], np.cumsum(rows)]).tolist())


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, Hk = case["op"], case["Hk"]
    s = {"case": case, "op": op}
    if op in ("rotate", "prompt", "tree"):
        rows, prefix, Hq = _ints(case["rows"]), _ints(case["prefix"]), case["Hq"]
        lens = [p + n for p, n in zip(prefix, rows)]
        n = sum(rows)
        s["table"], pool = _page_table(g, lens, 5)
        s["offsets"], s["lens"] = _offsets(rows), _int32(lens)
        s["k_pool"] = torch.zeros(pool, Hk, P, D, dtype=torch.bfloat16, device="cuda")
        s["v_pool"] = torch.zeros(pool, Hk, P, D, dtype=torch.bfloat16, device="cuda")
        if op == "rotate":
            # the slices of one projection's output, as a layer has them
            qkv = randn(n, (Hq + 2 * Hk) * D).to(torch.bfloat16)
            s["q"] = qkv[:, :Hq * D].view(n, Hq, D)
            s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(n, Hk, D)
            s["v"] = qkv[:, (Hq + Hk) * D:].view(n, Hk, D)
            s["q_weight"] = (1 + 0.1 * randn(D)).to(torch.bfloat16) if case["norm"] else None
            s["k_weight"] = (1 + 0.1 * randn(D)).to(torch.bfloat16) if case["norm"] else None
            pairs = _ints(case["axis_pairs"])
            r = sum(pairs)
            s["inv_freq"] = torch.tensor([500000.0 ** (-j / r) for j in range(r)], dtype=torch.float32, device="cuda")
            own_pos = torch.cat([torch.arange(p, p + m, device="cuda") for p, m in zip(prefix, rows)])
            if len(pairs) == 1:
                s["positions"] = own_pos.to(torch.int32)[None].contiguous()
            else:  # pictures of 32 x 32 patches between the words
                grid = [own_pos // 1024 * 1024, own_pos // 1024 * 1024 + own_pos // 32 % 32, own_pos // 1024 * 1024 + own_pos % 32]
                s["positions"] = torch.stack(grid[:len(pairs)]).to(torch.int32).contiguous()
            s["q_out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
        else:
            G = Hq // Hk
            s["k_pool"].copy_(randn(pool, Hk, P, D))
            s["v_pool"].copy_(randn(pool, Hk, P, D))
            way = randn(Hk, D)
            way *= math.sqrt(D) / way.norm(dim=1, keepdim=True)
            q = 0.8 * randn(n, Hk, G, D) + 0.6 * way[None, :, None]
            s["q"] = q.to(torch.bfloat16).view(n, Hq, D)
            first = s["table"][:, 0].long()   # the first token of a sequence draws attention
            s["k_pool"][first, :, 0] = (s["k_pool"][first, :, 0].float() + way).to(torch.bfloat16)
            s["out"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros(n, Hq, device="cuda")
        if op == "tree":
            # every node hangs on a random earlier one (or on the last token of the cache): its word has its ancestors' bits and its own
            rng = np.random.RandomState(int(seed) % (1 << 31))
            words = []
            for m in rows:
                up = []
                for i in range(m):
                    parent = int(rng.randint(max(-1, i // 2 - 4), i)) if i else -1
                    up.append((up[parent] if parent >= 0 else 0) | 1 << i)
                words += up
            s["mask"] = torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64)).cuda()
        return s
    if op == "fork":
        prompts, beams, ctx, gen, grow = (case[k] for k in ("prompts", "beams", "context", "generated", "grow"))
        B = prompts * beams
        rng = np.random.RandomState(int(seed) % (1 << 31))
        full = [int(ctx * (0.5 + 0.5 * rng.rand())) // P for _ in range(prompts)]
        length = [f * P + int(rng.randint(1, P + 1)) + gen for f in full]   # a prompt's beams are as long as each other
        used = [-(-n // P) for n in length]
        mpp = (ctx + gen + grow) // P + 3
        pool = prompts * (ctx // P) + B * ((gen + grow) // P + 4) + case["spare"]
        perm = rng.permutation(pool).astype(np.int32)
        table = np.full((B, mpp), -1, np.int32)
        at = 0
        for p in range(prompts):
            shared = perm[at:at + full[p]]
            at += full[p]
            for k in range(beams):
                table[p * beams + k, :full[p]] = shared
                table[p * beams + k, full[p]:used[p]] = perm[at:at + used[p] - full[p]]
                at += used[p] - full[p]
        keep = np.repeat(length, beams)
        s["table"] = torch.from_numpy(table).cuda()
        s["parent"] = _int32((np.repeat(np.arange(prompts) * beams, beams) + rng.randint(0, beams, B)).tolist())
        s["keep"], s["lens"] = _int32(keep.tolist()), _int32((keep + grow).tolist())
        s["copy_src"], s["copy_dst"] = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    elif op == "compact":
        B, pool = case["sequences"], case["pages"]
        rng = np.random.RandomState(int(seed) % (1 << 31))
        lens = [max(1, int(case["context"] * (0.75 + 0.25 * rng.rand()))) for _ in range(B)]
        mpp = -(-case["context"] // P)
        perm = rng.permutation(pool).astype(np.int32)
        table = np.full((B, mpp), -1, np.int32)
        at = 0
        for b, L in enumerate(lens):
            u = -(-L // P)
            table[b, :u] = perm[at:at + u]
            at += u
            if b % 4 == 3:   # every fourth sequence shares half of a neighbour's prefix
                h = min(u, -(-lens[b - 1] // P)) // 2
                table[b, :h] = table[b - 1, :h]
        s["table"], s["lens"] = torch.from_numpy(table).cuda(), _int32(lens)
        s["copy_src"], s["copy_dst"] = (torch.zeros(pool, dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        B, nodes, most = case["sequences"], case["nodes"], case["most"]
        rng = np.random.RandomState(int(seed) % (1 << 31))
        base = [int(rng.randint(0, case["context"] + 1)) for _ in range(B)]
        s["table"], pool = _page_table(g, [n + nodes for n in base], 3, case["context"] + nodes)
        path, cnt = np.zeros((B, most), np.int32), []
        for b in range(B):   # the first branch is taken, then nodes of deeper levels
            c = int(rng.randint(1, most + 1))
            tail = np.sort(rng.choice(np.arange(c, nodes), min(c - 1, nodes - c), replace=False))
            c = 1 + len(tail)
            path[b, 1:c] = tail
            cnt.append(c)
        s["base"], s["path"], s["cnt"] = _int32(base), torch.from_numpy(path).cuda(), _int32(cnt)
    s["k_pool"] = randn(pool, Hk, P, D).to(torch.bfloat16)
    s["v_pool"] = randn(pool, Hk, P, D).to(torch.bfloat16)
    if op != "accept":
        s["table_out"] = torch.zeros_like(s["table"])
        s["counts"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from sparse_decode_attention_head_gb300 import sa
        Hk, Hq = case["Hk"], case.get("Hq", case["Hk"])
        B, mpp = s["table"].shape
        s["prob"] = sa.Problem(B=B, Hq=Hq, Hk=Hk, max_pages_per_seq=mpp, num_pages=s["k_pool"].shape[0], sink=4, window=64,
                               block_sizes=[P] * Hk, k_per_head=[1] * Hq, kcap=1)
        s["ws"] = sa.Workspace(s["prob"], rows=True)
        if s["op"] == "rotate":
            s["rope"] = sa.Rope(_ints(case["axis_pairs"]), sa.ROPE_HALVES if case["layout"] == "halves" else sa.ROPE_PAIRS)
    return s


# ------------------------------------------------------------------ the plain forms

def _where(s):
    """(sequence, row in it, position in the cache) of every packed row."""
    n = s["q"].shape[0]
    off = s["offsets"].long()
    at = torch.arange(n, device="cuda")
    b = torch.searchsorted(off, at, right=True) - 1
    i = at - off[b]
    return b, i, (s["lens"].long() - (off[1:] - off[:-1]))[b] + i


def _plain_rotate(s):
    c = s["case"]
    pairs = _ints(c["axis_pairs"])
    r = sum(pairs)
    axis = torch.repeat_interleave(torch.arange(len(pairs), device="cuda"), torch.tensor(pairs, device="cuda"), output_size=r)
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()      # [n][r], in 64 bits: a far position has many turns
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["layout"] == "halves":
            a, b, rest = x[..., :r], x[..., r:2 * r], x[..., 2 * r:]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1).to(torch.bfloat16)
        a, b, rest = x[..., 0:2 * r:2], x[..., 1:2 * r:2], x[..., 2 * r:]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1).to(torch.bfloat16)

    b, _, pos = _where(s)
    page, row = s["table"][b, pos // P].long(), pos % P
    s["k_pool"][page, :, row] = one(s["k"], s["k_weight"])
    s["v_pool"][page, :, row] = s["v"]
    return {"q": one(s["q"], s["q_weight"]), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_attention(s):
    c = s["case"]
    rows, Hq, Hk = _ints(c["rows"]), c["Hq"], c["Hk"]
    B, G, N = len(rows), Hq // Hk, max(rows)
    b, i, _ = _where(s)
    q = torch.zeros(B, N, Hq, D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, N, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    table = s["table"].long().clamp(min=0)
    L = table.shape[1] * P
    k = s["k_pool"][table].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D).float()
    z = torch.matmul(q, k.transpose(-1, -2)).view(B, Hk, G, N, L)
    del k
    z *= 1.0 / math.sqrt(D)
    col = torch.arange(L, device="cuda")
    before = (s["lens"] - (s["offsets"][1:] - s["offsets"][:-1])).long()    # tokens in the cache ahead of the rows
    if s["op"] == "prompt":
        seen = col[None, None] <= (before[:, None] + torch.arange(N, device="cuda"))[:, :, None]
    else:
        word = torch.zeros(B, N, dtype=torch.int64, device="cuda")
        word[b, i] = s["mask"]
        bit = col[None] - before[:, None]
        draft = (bit >= 0) & (col[None] < s["lens"][:, None])
        seen = (bit < 0)[:, None] | (draft[:, None] & ((word[:, :, None] >> bit.clamp(0, 63)[:, None]) & 1).bool())
    z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    v = s["v_pool"][table].permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D).float()
    o = torch.matmul(z.view(B, Hk, G * N, L), v).view(B, Hk, G, N, D) / total
    lse = (m + torch.log(total))[..., 0]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[b, i].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, N, Hq)[b, i]}


def _held(table, tokens):
    """How many rows hold each of `pool` pages: the first ceil(tokens / P) entries of a row are its own."""
    return torch.arange(table.shape[1], device="cuda")[None] < ((tokens + P - 1) // P)[:, None]


def _listed_pages(flag):
    """The indices at which flag is true, ascending, in a list of flag's length, and how many."""
    n = flag.numel()
    rank = torch.cumsum(flag.long(), 0) - 1
    got = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")
    got.scatter_(0, torch.where(flag, rank, torch.full_like(rank, n)), torch.arange(n, device="cuda"))
    got[n] = -1
    return got, flag.sum()


def _plain_copy(s, src, dst):
    src, dst = src[src >= 0].long(), dst[dst >= 0].long()
    s["k_pool"][dst] = s["k_pool"][src]
    s["v_pool"][dst] = s["v_pool"][src]


def _plain_fork(s):
    pool = s["k_pool"].shape[0]
    keep, room = s["keep"].long(), torch.maximum(s["lens"], s["keep"]).long()
    table = s["table"].long()[s["parent"].long()]
    B, mpp = table.shape
    held = _held(table, keep)
    refs = torch.zeros(pool, dtype=torch.int64, device="cuda").index_add_(0, table.clamp(min=0).flatten(), held.flatten().long())
    had, want = (keep + P - 1) // P, (room + P - 1) // P
    row = torch.arange(B, device="cuda")
    writes = (keep % P != 0) & (room > keep)
    tail = table[row, (had - 1).clamp(min=0)].clamp(min=0)
    writers = torch.zeros(pool, dtype=torch.int64, device="cuda").index_add_(0, tail, writes.long())
    lowest = torch.full((pool,), B, dtype=torch.int64, device="cuda").scatter_reduce_(0, tail, torch.where(writes, row, torch.full_like(row, B)), "amin")
    copy = writes & ~((writers[tail] == refs[tail]) & (lowest[tail] == row))
    need = copy.long() + want - had
    start = torch.cumsum(need, 0) - need
    free, n_free = _listed_pages(refs == 0)
    j = torch.arange(mpp, device="cuda")[None]
    take = torch.where(j == had[:, None] - 1, start[:, None], start[:, None] + copy[:, None] + j - had[:, None])
    new = free[take.clamp(0, pool)]
    fresh = (copy[:, None] & (j == had[:, None] - 1)) | ((j >= had[:, None]) & (j < want[:, None]))
    out = torch.where(fresh, new, torch.where(j < had[:, None], table, torch.full_like(table, -1)))
    which, n_copy = _listed_pages(copy)
    some = which[:B] >= 0
    src = torch.where(some, tail[which[:B].clamp(min=0)], torch.full_like(which[:B], -1))
    dst = torch.where(some, free[start[which[:B].clamp(min=0)].clamp(0, pool)], torch.full_like(which[:B], -1))
    _plain_copy(s, src, dst)
    return {"table": out.int(), "copy_src": src.int(), "copy_dst": dst.int(), "counts": torch.stack([n_copy, n_free - need.sum()]).int(),
            "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_compact(s):
    pool = s["k_pool"].shape[0]
    table = s["table"].long()
    held = _held(table, s["lens"].long())
    refs = torch.zeros(pool, dtype=torch.int64, device="cuda").index_add_(0, table.clamp(min=0).flatten(), held.flatten().long())
    at = torch.arange(pool, device="cuda")
    live = refs > 0
    n_live = live.sum()
    src, n_move = _listed_pages(live & (at >= n_live))
    dst, _ = _listed_pages(~live & (at < n_live))
    to = at.clone()
    to = torch.cat([to, to[:1]]).scatter_(0, torch.where(src[:pool] >= 0, src[:pool], torch.full_like(at, pool)), dst[:pool])[:pool]
    out = torch.where(held, to[table.clamp(min=0)], torch.full_like(table, -1))
    _plain_copy(s, src[:pool], dst[:pool])
    return {"table": out.int(), "copy_src": src[:pool].int(), "copy_dst": dst[:pool].int(), "counts": torch.stack([n_move, n_live]).int(),
            "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_accept(s):
    B, most = s["path"].shape
    step = torch.arange(most, device="cuda")[None]
    ok = (step < s["cnt"].long()[:, None]).flatten()
    b = torch.arange(B, device="cuda")[:, None].expand(B, most).flatten()[ok]
    base = s["base"].long()[:, None]
    src, dst = (base + s["path"].long()).flatten()[ok], (base + step).flatten()[ok]
    sp, dp = s["table"][b, src // P].long(), s["table"][b, dst // P].long()
    k, v = s["k_pool"][sp, :, src % P], s["v_pool"][sp, :, src % P]
    s["k_pool"][dp, :, dst % P] = k
    s["v_pool"][dp, :, dst % P] = v
    return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}


_PLAIN = {"rotate": _plain_rotate, "prompt": _plain_attention, "tree": _plain_attention, "fork": _plain_fork, "compact": _plain_compact, "accept": _plain_accept}


# ------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    from sparse_decode_attention_head_gb300 import sa
    p, ws, op = s["prob"], s["ws"], s["op"]
    if op == "rotate":
        sa.qk_norm_rope(p, s["q"], s["k"], s["v"], s["offsets"], s["lens"], s["table"],
                        s["q_out"], s["k_pool"], s["v_pool"], ws, rope=s["rope"], inv_freq=s["inv_freq"], positions=s["positions"],
                        q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "prompt":
        sa.prompt_attention(p, s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["offsets"], s["out"], ws, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "tree":
        sa.tree_attention(p, s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["offsets"], s["mask"], s["out"], ws, lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "accept":
        sa.accept_rows(p, s["k_pool"], s["v_pool"], s["table"], s["base"], s["path"], s["cnt"], ws)
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "fork":
        sa.plan_pages(p, s["table"], s["parent"], s["keep"], s["lens"], s["table_out"], s["copy_src"], s["copy_dst"], s["counts"], ws)
    else:
        sa.compact_pages(p, s["table"], s["lens"], s["table_out"], s["copy_src"], s["copy_dst"], s["counts"], ws)
    sa.copy_pages(p, s["k_pool"], s["v_pool"], s["copy_src"], s["copy_dst"], s["counts"], ws)
    return {"table": s["table_out"], "copy_src": s["copy_src"], "copy_dst": s["copy_dst"], "counts": s["counts"],
            "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, Hk = case["op"], case["Hk"]
    page = 2 * Hk * P * D * 2   # K and V of one page, all heads
    if op in ("rotate", "prompt", "tree"):
        rows, prefix, Hq = _ints(case["rows"]), _ints(case["prefix"]), case["Hq"]
        n = sum(rows)
        if op == "rotate":
            return {"bytes": 2 * n * (Hq + 2 * Hk) * D * 2 + 4 * n * len(_ints(case["axis_pairs"])), "flops": 10 * n * (Hq + Hk) * D}
        cache = sum(p + m for p, m in zip(prefix, rows)) * Hk * D * 2 * 2
        pairs = sum(m * p + m * (m + 1) // 2 for p, m in zip(prefix, rows))   # a tree's rows see at most the causal ones
        return {"bytes": cache + 2 * n * Hq * D * 2 + 4 * n * Hq, "flops": 4 * D * Hq * pairs}
    if op == "fork":
        B = case["prompts"] * case["beams"]
        table = 4 * B * -(-int(0.75 * case["context"] + case["generated"]) // P)
        return {"bytes": 2 * table + 2 * page * B // 2, "flops": 0}   # about half of the beams have to copy their last page
    if op == "compact":
        live = int(case["sequences"] * 0.875 * case["context"] / P * 0.875)
        moved = live * max(0, case["pages"] - live) // case["pages"]   # scattered evenly: what lies behind the live ones' count moves
        return {"bytes": 2 * 4 * live + 2 * page * moved, "flops": 0}
    return {"bytes": 2 * page // P * case["sequences"] * case["most"] // 2, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(case, s)
    if case["op"] in ("prompt", "tree"):
        return _exact_attention(case, s)
    return None   # whole numbers and copies


def _exact_rotate(case, s):
    """Each pair of dims as one complex number, turned by e^(i angle)."""
    pairs = _ints(case["axis_pairs"])
    r = sum(pairs)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    first = np.arange(r) if case["layout"] == "halves" else 2 * np.arange(r)
    second = first + (r if case["layout"] == "halves" else 1)
    first, second = (torch.from_numpy(x).cuda() for x in (first, second))
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    out, at = [], 0
    rows, prefix = _ints(case["rows"]), _ints(case["prefix"])
    for b, (n, p) in enumerate(zip(rows, prefix)):
        turn = torch.stack([s["positions"][a, at:at + n].double() for a in axis], 1) * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(turn), turn)
        both = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x[at:at + n].double()
            if w is not None:
                x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            y = torch.complex(x[..., first], x[..., second]) * turn[:, None]
            x = x.clone()
            x[..., first], x[..., second] = y.real, y.imag
            both.append(x)
        out.append(both[0])
        t = torch.arange(p, p + n, device="cuda")
        page = s["table"][b].long()[t // P]
        k_pool[page, :, t % P] = both[1]
        v_pool[page, :, t % P] = s["v"][at:at + n].double()
        at += n
    return {"q": torch.cat(out), "k_pool": k_pool, "v_pool": v_pool}


def _exact_attention(case, s):
    """One head's softmax over the positions it sees, a block of rows at a time."""
    rows, prefix, Hq, Hk = _ints(case["rows"]), _ints(case["prefix"]), case["Hq"], case["Hk"]
    if 4 * D * Hq * sum(m * (p + m) for p, m in zip(prefix, rows)) > 6e12:
        return None
    out = torch.zeros(sum(rows), Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(rows), Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, p) in enumerate(zip(rows, prefix)):
        t = torch.arange(p + n, device="cuda")
        page = s["table"][b].long()[t // P]
        k = s["k_pool"][page, :, t % P].double()   # [L][Hk][D]
        v = s["v_pool"][page, :, t % P].double()
        for i0 in range(0, n, 2048):
            i1 = min(n, i0 + 2048)
            L = p + i1 if case["op"] == "prompt" else p + n   # later positions are seen by none of these rows
            if case["op"] == "prompt":
                seen = t[None, :L] <= p + torch.arange(i0, i1, device="cuda")[:, None]
            else:
                words = s["mask"][at + i0:at + i1].cpu().numpy().view(np.uint64)
                bits = np.array([[(int(w) >> j) & 1 for j in range(n)] for w in words], dtype=bool)
                seen = torch.cat([torch.ones(i1 - i0, p, dtype=torch.bool, device="cuda"), torch.from_numpy(bits).cuda()], 1)
            for h in range(Hq):
                z = s["q"][at + i0:at + i1, h].double() @ k[:L, h * Hk // Hq].T / math.sqrt(D)
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                lse[at + i0:at + i1, h] = torch.logsumexp(z, -1)
                out[at + i0:at + i1, h] = torch.softmax(z, -1) @ v[:L, h * Hk // Hq]
        at += n
    return {"out": out, "lse": lse}
