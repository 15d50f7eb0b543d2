"""Cases of the operators that serve one step over a tree of drafted tokens: page tables and slot
maps from request lengths, head norms with the position rotation, attention of a draft tree over a
KV cache, and the greedy walk along the tree with the kept path's append.

``run`` computes an operator in plain torch (32 bits, rounded once at the end) or, with ``own``
true, calls the library's entry points.
"""
import math
import random

import torch

own = False

KINDS = ("pages", "rope", "attn", "commit")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a small batch: every request grows by a draft's width, few need a page
        dict(name="pages-step", op="pages", B=8, page=64, ctx=2183, new=8, release=0, spare=64),
        # a scheduler's step: prompt chunks, decodes and finished requests together
        dict(name="pages-mixed", op="pages", B=500, page=64, ctx=6000, new=96, release=9, spare=2048),
        # whole prompts of a large batch enter at once
        dict(name="pages-prompts", op="pages", B=1024, page=128, ctx=700, new=256, release=5, spare=8192),
        # the attention layer of one verify step: 8 rows of 24 q and 4 kv heads, rotated in place
        dict(name="rope-step", op="rope", M=8, Hq=24, Hkv=4, hd=256, rot=64, ctx=2183, base=1e7, inter=False, append=False),
        # a batch's chunk of prompt tokens far into their contexts, K and V straight into the pages
        dict(name="rope-chunk", op="rope", M=500, Hq=24, Hkv=4, hd=256, rot=64, ctx=131072, base=1e7, inter=False, append=True),
        # a long prompt through narrower heads, every dimension rotated in adjacent pairs
        dict(name="rope-prompt", op="rope", M=8192, Hq=32, Hkv=8, hd=128, rot=128, ctx=8192, base=1e4, inter=True, append=True),
        # the smallest attention layer, a short context
        dict(name="attn-tiny", op="attn", B=1, N=8, Hq=2, Hkv=1, hd=64, ctx=128, page=0, shape="mixed", gate=False),
        # one request at the usual context, a tree of 16 drafts, gated attention
        dict(name="attn-one", op="attn", B=1, N=16, Hq=24, Hkv=4, hd=256, ctx=2183, page=64, shape="mixed", gate=True),
        # a batch in flight, small trees, ragged lengths and node counts
        dict(name="attn-batch", op="attn", B=32, N=13, Hq=32, Hkv=8, hd=128, ctx=8000, page=128, shape="mixed", gate=False),
        # the widest tree over a long context
        dict(name="attn-long", op="attn", B=1, N=64, Hq=24, Hkv=4, hd=256, ctx=131072, page=0, shape="wide", gate=True),
        # one request's tree walked and its path kept
        dict(name="commit-one", op="commit", B=1, N=16, Hkv=4, hd=256, ctx=2183, page=64, shape="mixed"),
        # many requests with wide trees
        dict(name="commit-batch", op="commit", B=256, N=61, Hkv=4, hd=256, ctx=500, page=64, shape="mixed"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(KINDS)
    heads = rng.choice([(24, 4, 256), (32, 8, 128), (6, 2, 64), (16, 2, 256), (8, 8, 128), (5, 1, 64)])
    if op == "pages":
        B = _log_int(rng, 1, 1024)
        new = _log_int(rng, 1, 256)
        return dict(op=op, B=B, page=rng.choice([64, 128, 256]), ctx=_log_int(rng, 1, 4000), new=new,
                    release=rng.choice([0, 3, 7]), spare=rng.randint(0, 4096))
    if op == "rope":
        Hq, Hkv, hd = heads
        M = _log_int(rng, 1, 4096)
        return dict(op=op, M=M, Hq=Hq, Hkv=Hkv, hd=hd, rot=rng.choice([16, hd // 2, hd]), ctx=_log_int(rng, 16, 500000),
                    base=rng.choice([1e4, 1e6, 1e7]), inter=rng.random() < 0.5, append=rng.random() < 0.5)
    if op == "attn":
        Hq, Hkv, hd = heads
        N = _log_int(rng, 1, 64)
        B = _log_int(rng, 1, 32)
        most = max(64, min(131072, 40_000_000 // (B * N * Hq)))   # positions: bounds the score products
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=Hkv, hd=hd, ctx=_log_int(rng, 1, most), page=rng.choice([0, 64, 192, 256]),
                    shape=rng.choice(["mixed", "wide", "chain"]), gate=rng.random() < 0.5)
    return dict(op="commit", B=_log_int(rng, 1, 256), N=_log_int(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]),
                hd=rng.choice([64, 128, 256]), ctx=_log_int(rng, 1, 2000), page=rng.choice([0, 64, 128]),
                shape=rng.choice(["mixed", "wide", "chain"]))


# --------------------------------------------- what a case fixes by itself

def _lengths(case):
    """Ragged context lengths of a batch: the first the longest, the others down to about half."""
    ctx = case["ctx"]
    return [ctx - (b * 7919) % (ctx // 2 + 1) for b in range(case["B"])]


def _counts(case):
    """Nodes of each sequence's tree: the first full, the others down to about half."""
    N = case["N"]
    return [N - (b * 31) % (N // 2 + 1) for b in range(case["B"])]


def _new(case):
    """New rows of each request: mostly short, every fourth long; -1 for a finished one."""
    new, rel = case["new"], case["release"]
    out = []
    for b in range(case["B"]):
        n = new if b % 4 == 0 else max(0, new // 8 - b % 3)
        out.append(-1 if rel and b % rel == rel - 1 else n)
    return out


def _ceil(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "pages":
        lens, new, page = _lengths(case), _new(case), case["page"]
        rows = sum(max(n, 0) for n in new)
        moved = sum(_ceil(x, page) if n < 0 else max(0, _ceil(x + n, page) - _ceil(x, page)) for x, n in zip(lens, new))
        held = sum(_ceil(x + max(n, 0), page) - x // page for x, n in zip(lens, new) if n > 0)
        return {"bytes": 16 * case["B"] + 8 * moved + 4 * held + 12 * rows, "flops": 0}
    if op == "rope":
        q, kv = case["M"] * case["Hq"] * case["hd"], case["M"] * case["Hkv"] * case["hd"]
        n = q + (2 * kv if case["append"] else kv)
        return {"bytes": 4 * n + case["M"] * (12 if case["append"] else 4), "flops": 8 * (q + kv)}
    if op == "attn":
        lens, cnt = _lengths(case), _counts(case)
        Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
        rows = sum(cnt)
        nbytes = sum(4 * Hkv * hd * (x + n) for x, n in zip(lens, cnt)) + (6 if case["gate"] else 4) * rows * Hq * hd
        return {"bytes": nbytes, "flops": sum(4 * Hq * hd * n * (x + 1) for x, n in zip(lens, cnt))}
    B, N = case["B"], case["N"]
    # every node's token, parent and argmax is read; the root's row is always kept
    return {"bytes": 12 * B * N + B * 8 * case["Hkv"] * case["hd"], "flops": 0}


# ---------------------------------------------------------------- inputs

def _trees(case, seed):
    """parent [B, N] int32: parent[i] < i, -1 for the root (and for rows past a tree's nodes)."""
    B, N = case["B"], case["N"]
    rng = random.Random(seed * 1000003 + 17)
    rows = []
    for n in _counts(case):
        par = [-1]
        for i in range(1, n):
            if case["shape"] == "chain":
                par.append(i - 1)
            elif case["shape"] == "wide":
                par.append(rng.randrange(0, max(1, i // 3)))
            else:
                par.append(rng.randrange(max(0, i - 6), i))
        rows.append(par + [-1] * (N - n))
    return torch.tensor(rows, dtype=torch.int32).cuda()


def _normal(g, shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * sigma).to(torch.bfloat16)


def _pool_of(case, seed, rows_of):
    """Page table [B, max_pages], page size and page count of a cache that holds rows_of[b]
    positions for sequence b; page = 0 in the case means one page per sequence (a contiguous cache)."""
    B = case["B"]
    most = max(rows_of)
    page = case["page"] or _ceil(most, 64) * 64
    per = _ceil(most, page)
    n_pages = B * per + (0 if not case["page"] else 3)
    order = list(range(n_pages))
    if case["page"]:
        random.Random(seed * 7 + 3).shuffle(order)
    table = torch.tensor(order[: B * per], dtype=torch.int32).reshape(B, per).cuda()
    return table, page, n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 9176 + 5)
    s = dict(case=case)
    op = case["op"]
    if op == "pages":
        B, page = case["B"], case["page"]
        lens, new = _lengths(case), _new(case)
        held = [_ceil(x, page) for x in lens]
        need = [_ceil(x + max(n, 0), page) for x, n in zip(lens, new)]
        mp = max(need) + 2
        n_pages = sum(need) + case["spare"] + 1
        order = list(range(n_pages))
        random.Random(seed).shuffle(order)
        used = sum(held)
        grid = torch.full((B, mp), -1, dtype=torch.int32)
        h = torch.tensor(held)
        grid[torch.arange(mp)[None, :] < h[:, None]] = torch.tensor(order[:used], dtype=torch.int32)
        s["table"] = grid.cuda()
        free = torch.full((n_pages,), -1, dtype=torch.int32)
        free[: n_pages - used] = torch.tensor(order[used:], dtype=torch.int32)
        s["free"] = free.cuda()
        s["n_free"] = torch.tensor([n_pages - used], dtype=torch.int32).cuda()
        s["held"] = torch.tensor(held, dtype=torch.int32).cuda()
        s["ctx"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["new"] = torch.tensor(new, dtype=torch.int32).cuda()
        rows = sum(max(n, 0) for n in new) + 5         # five rows behind the last request
        s["n_free_out"] = torch.zeros_like(s["n_free"])
        s["held_out"] = torch.zeros_like(s["held"])
        s["row_start"] = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        s["pos"] = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        if own:
            from bit_exact_speculative_gb300 import xv
            s["pages"] = xv.kv_pages(s["table"], page, n_pages)
            s["ws"] = xv.workspace(xv.xv_kv_pages_workspace_size(B))
        return s
    if op == "rope":
        M, Hq, Hkv, hd = case["M"], case["Hq"], case["Hkv"], case["hd"]
        # rows of a projection [q | gate | k | v]
        s["proj"] = _normal(g, (M, (2 * Hq + 2 * Hkv) * hd), 1.3)
        s["qn"], s["kn"] = _normal(g, (hd,), 0.2), _normal(g, (hd,), 0.2)
        s["q_out"] = torch.zeros((M, Hq * hd), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros((M, Hkv * hd), dtype=torch.bfloat16, device="cuda")
        start = max(0, case["ctx"] - M)
        s["pos"] = (start + torch.arange(M, device="cuda")).to(torch.int32)
        if case["append"]:
            page = 64
            n_pages = _ceil(M, page) + 3
            perm = torch.randperm(n_pages, generator=g, device="cuda")
            r = torch.arange(M, device="cuda")
            s["slots"] = perm[r // page] * page + r % page
            s["page"], s["n_pages"] = page, n_pages
            s["kp"] = torch.zeros((n_pages, Hkv, page, hd), dtype=torch.bfloat16, device="cuda")
            s["vp"] = torch.zeros_like(s["kp"])
        if own:
            from bit_exact_speculative_gb300 import xv
            s["freqs"] = xv.rope_freqs(case["rot"], case["base"])
        else:
            s["freqs"] = case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        return s
    B, N, Hkv, hd = case["B"], case["N"], case["Hkv"], case["hd"]
    lens, cnt = _lengths(case), _counts(case)
    s["parent"] = _trees(case, seed)
    s["nodes"] = torch.tensor(cnt, dtype=torch.int32).cuda()
    s["ctx"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["table"], s["page"], s["n_pages"] = _pool_of(case, seed, [x + N for x in lens])
    s["kp"] = _normal(g, (s["n_pages"], Hkv, s["page"], hd))
    s["vp"] = _normal(g, (s["n_pages"], Hkv, s["page"], hd))
    if op == "attn":
        Hq = case["Hq"]
        # rows of a projection [q | gate | k | v]: the tree's own keys and values are read from them
        s["proj"] = _normal(g, (B * N, (2 * Hq + 2 * Hkv) * hd))
        s["out"] = torch.zeros((B * N, Hq * hd), dtype=torch.bfloat16, device="cuda")
        if own:
            from bit_exact_speculative_gb300 import xv
            s["pages"] = xv.kv_pages(s["table"], s["page"], s["n_pages"])
            s["ws"] = xv.workspace(xv.xv_attn_tree_workspace_size(B, N, Hq, hd, case["ctx"]))
        return s
    s["kv"] = _normal(g, (B * N, 2 * Hkv * hd))
    # the target's token after each node, and drafts that follow it about two times in three
    s["argmax"] = torch.randint(0, 50, (B, N), generator=g, device="cuda", dtype=torch.int32)
    follow = torch.gather(s["argmax"], 1, s["parent"].clamp_min(0).long())
    hit = torch.rand((B, N), generator=g, device="cuda") < 0.65
    s["tokens"] = torch.where(hit, follow, torch.randint(0, 50, (B, N), generator=g, device="cuda", dtype=torch.int32))
    s["path"] = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    s["n_keep"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    s["next"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if own:
        from bit_exact_speculative_gb300 import xv
        s["pages"] = xv.kv_pages(s["table"], s["page"], s["n_pages"])
    return s


# ------------------------------------------------------------- plain forms

def _ancestors(parent):
    """[B, N, N] bool: node j lies on the path from the root to node i (i itself included)."""
    B, N = parent.shape
    node = torch.arange(N, device=parent.device)
    step = (parent[:, :, None] == node) | (node[:, None] == node)
    return torch.linalg.matrix_power(step.float(), max(N - 1, 1)) > 0


def _plain_pages(s):
    page, ctx, new, held = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["held"].long()
    table, free, nf = s["table"], s["free"], s["n_free"].long()
    B, mp = table.shape
    j = torch.arange(mp, device="cuda")[None, :]
    gone = new < 0
    back = torch.where(gone, held, 0)
    back_at = back.cumsum(0) - back
    # released pages go on the stack, a request's last page first
    dest = nf + back_at[:, None] + held[:, None] - 1 - j
    dest = torch.where(gone[:, None] & (j < held[:, None]), dest, free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, dest.reshape(-1), table.reshape(-1))[:-1]
    need = torch.where(gone, 0, (ctx + new + page - 1) // page)
    add = (need - held).clamp_min(0).masked_fill(gone, 0)
    add_at = add.cumsum(0) - add
    src = (nf + back.sum() - 1 - add_at[:, None] - (j - held[:, None])).clamp(0, free.numel() - 1)
    fresh = ~gone[:, None] & (j >= held[:, None]) & (j < need[:, None])
    table = torch.where(fresh, stack[src], table)
    n = new.clamp_min(0)
    end = n.cumsum(0)
    t = torch.arange(s["pos"].numel(), device="cuda")
    b = torch.searchsorted(end, t, right=True).clamp_max(B - 1)
    live = t < end[-1]
    pos = ctx[b] + t - (end - n)[b]
    slot = table[b, (pos // page).clamp_max(mp - 1)].long() * page + pos % page
    start = torch.cat([end.new_zeros(1), end])
    return dict(table=table, free=stack, n_free=(nf + back.sum() - add.sum()).int(),
                held=torch.where(gone, 0, torch.maximum(held, need)).int(), row_start=start.int(),
                pos=torch.where(live, pos, -1).int(), slots=torch.where(live, slot, -1))


def _plain_norm_rope(x, w, cos, sin, rot, inter):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * (1 + w.float())
    r = y[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., : rot // 2], r[..., rot // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([c, d], -1).flatten(-2) if inter else torch.cat([c, d], -1)
    return torch.cat([r, y[..., rot:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    M, Hq, Hkv, hd = c["M"], c["Hq"], c["Hkv"], c["hd"]
    angle = s["pos"].double()[:, None] * s["freqs"]      # far positions need the angle in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = s["proj"][:, : Hq * hd].reshape(M, Hq, hd)
    kv = s["proj"][:, 2 * Hq * hd:].reshape(M, 2 * Hkv, hd)
    q = _plain_norm_rope(q, s["qn"], cos, sin, c["rot"], c["inter"])
    k = _plain_norm_rope(kv[:, :Hkv], s["kn"], cos, sin, c["rot"], c["inter"])
    if not c["append"]:
        return dict(q=q.reshape(M, -1), k=k.reshape(M, -1))
    pg, at = s["slots"] // s["page"], s["slots"] % s["page"]
    s["kp"][pg, :, at] = k
    s["vp"][pg, :, at] = kv[:, Hkv:]
    return dict(q=q.reshape(M, -1), kp=s["kp"], vp=s["vp"])


def _plain_attn(s):
    c = s["case"]
    B, N, Hq, Hkv, hd = c["B"], c["N"], c["Hq"], c["Hkv"], c["hd"]
    G = Hq // Hkv
    rows = s["proj"].reshape(B, N, -1, hd)
    q = rows[:, :, :Hq].reshape(B, N, Hkv, G, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * N, hd)
    tree = rows[:, :, 2 * Hq:].transpose(1, 2)
    # [B, Hkv, positions, hd]: the cache's pages in order, then the tree's own rows
    lk, lv = (x[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, : c["ctx"]] for x in (s["kp"], s["vp"]))
    seen = torch.arange(lk.shape[2], device="cuda")[None, :] < s["ctx"][:, None]
    real = torch.arange(N, device="cuda")[None, :] < s["nodes"][:, None]
    mask = torch.cat([seen[:, None, :].expand(-1, N, -1), _ancestors(s["parent"])], -1)
    k = torch.cat([lk, tree[:, :Hkv]], 2).float()
    p = q.float() @ k.transpose(-1, -2)
    del k
    p = p.reshape(B, Hkv, G, N, -1).mul_(hd ** -0.5).masked_fill_(~mask[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    ok = torch.cat([seen, real], -1)[:, None, :, None]
    v = torch.cat([lv, tree[:, Hkv:]], 2).float().masked_fill_(~ok, 0)
    o = (p.flatten(2, 3) @ v).reshape(B, Hkv, G, N, hd) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq * hd)
    if c["gate"]:
        o = o * torch.sigmoid(rows[:, :, Hq: 2 * Hq].reshape(B, N, -1).float())
    return o.masked_fill(~real[..., None], 0).reshape(B * N, -1).to(torch.bfloat16)


def _plain_commit(s):
    c = s["case"]
    B, N, Hkv, hd = c["B"], c["N"], c["Hkv"], c["hd"]
    parent, tokens, argmax = s["parent"].long(), s["tokens"], s["argmax"]
    node = torch.arange(N, device="cuda")
    real = node[None, :] < s["nodes"][:, None]
    same = (parent[:, :, None] == parent[:, None, :]) & (tokens[:, :, None] == tokens[:, None, :])
    first = ~(same & (node[None, :] < node[:, None])).any(-1)      # the lowest of equal siblings
    hit = (tokens == torch.gather(argmax, 1, parent.clamp_min(0))) & first & (parent >= 0) & real
    hit = hit | ((node == 0)[None, :] & real)
    anc = _ancestors(s["parent"])
    kept = ~(anc & ~hit[:, None, :]).any(-1)
    n_keep = kept.sum(-1)
    rank = torch.where(kept, kept.cumsum(-1) - 1, N)
    path = node.new_full((B, N + 1), -1).scatter(1, rank, node[None, :].expand(B, N))[:, :N]
    last = torch.gather(path, 1, (n_keep - 1).clamp_min(0)[:, None]).clamp_min(0)
    # kept node i goes to position ctx + its rank
    pos = s["ctx"].long()[:, None] + rank.clamp_max(N - 1)
    pg, at = torch.gather(s["table"].long(), 1, pos // s["page"]), pos % s["page"]
    rows = s["kv"].reshape(B, N, 2 * Hkv, hd)
    b, i = kept.nonzero(as_tuple=True)
    s["kp"][pg[b, i], :, at[b, i]] = rows[b, i, :Hkv]
    s["vp"][pg[b, i], :, at[b, i]] = rows[b, i, Hkv:]
    return dict(path=path.int(), n_keep=n_keep.int(), next=torch.gather(argmax, 1, last)[:, 0], kp=s["kp"], vp=s["vp"])


# --------------------------------------------------------------------- run

def _own(s):
    from bit_exact_speculative_gb300 import xv
    c = s["case"]
    op = c["op"]
    if op == "pages":
        xv.xv_kv_pages_update(s["pages"], s["free"], s["n_free"], s["held"], s["ctx"], s["new"], s["row_start"], s["pos"],
                              s["slots"], s["ws"], n_free_out=s["n_free_out"], held_out=s["held_out"])
        return dict(table=s["table"], free=s["free"], n_free=s["n_free_out"], held=s["held_out"],
                    row_start=s["row_start"], pos=s["pos"], slots=s["slots"])
    if op == "rope":
        Hq, Hkv, hd = c["Hq"], c["Hkv"], c["hd"]
        q, kv = s["proj"][:, : Hq * hd], s["proj"][:, 2 * Hq * hd:]
        if not c["append"]:
            xv.xv_qk_norm_rope(q, kv, s["pos"], Hq, Hkv, hd, s["q_out"], s["k_out"], q_norm=s["qn"], k_norm=s["kn"],
                               freqs=s["freqs"], interleaved=c["inter"])
            return dict(q=s["q_out"], k=s["k_out"])
        xv.xv_qk_norm_rope_append(q, kv, s["pos"], s["slots"], Hq, Hkv, hd, s["q_out"], s["kp"], s["vp"], s["page"],
                                  s["n_pages"], q_norm=s["qn"], k_norm=s["kn"], freqs=s["freqs"], interleaved=c["inter"])
        return dict(q=s["q_out"], kp=s["kp"], vp=s["vp"])
    B, N, Hkv, hd = c["B"], c["N"], c["Hkv"], c["hd"]
    if op == "attn":
        Hq = c["Hq"]
        q, gate, kv = s["proj"], s["proj"][:, Hq * hd:], s["proj"][:, 2 * Hq * hd:]
        gate = gate if c["gate"] else None
        if c["page"]:
            xv.xv_attn_tree_paged(q, s["kp"], s["vp"], s["pages"], s["ctx"], kv, s["parent"], s["nodes"], N, B, Hq, Hkv,
                                  hd, c["ctx"], hd ** -0.5, s["out"], s["ws"], gate=gate)
        else:
            xv.xv_attn_tree(q, s["kp"], s["vp"], s["ctx"], kv, s["parent"], s["nodes"], N, B, Hq, Hkv, hd, s["page"],
                            c["ctx"], hd ** -0.5, s["out"], s["ws"], gate=gate)
        return s["out"]
    xv.xv_tree_accept(s["tokens"], s["parent"], s["nodes"], s["argmax"], s["path"], s["n_keep"], s["next"])
    if c["page"]:
        xv.xv_kv_append_path_paged(s["kv"], s["path"], s["n_keep"], s["ctx"], N, B, Hkv, hd, s["pages"], s["kp"], s["vp"])
    else:
        xv.xv_kv_append_path(s["kv"], s["path"], s["n_keep"], s["ctx"], N, B, Hkv, hd, s["page"], s["kp"], s["vp"])
    return dict(path=s["path"], n_keep=s["n_keep"], next=s["next"], kp=s["kp"], vp=s["vp"])


def run(state):
    if own:
        return _own(state)
    return dict(pages=_plain_pages, rope=_plain_rope, attn=_plain_attn, commit=_plain_commit)[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_head(x, w, angle, inter):
    """One norm and rotation in 64 bits, as a product with each pair's complex number."""
    y = x.double()
    y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (w.double() + 1)
    n = angle.shape[-1]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = y.clone()
    if inter:
        z = torch.view_as_complex(y[..., : 2 * n].unflatten(-1, (n, 2)).contiguous()) * turn
        out[..., 0: 2 * n: 2], out[..., 1: 2 * n: 2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :n], y[..., n: 2 * n]) * turn
        out[..., :n], out[..., n: 2 * n] = z.real, z.imag
    return out


def _exact_commit(case, s):
    """The kept rows where a walk from each root puts them; the walk's whole numbers have no 64-bit value."""
    B, N, Hkv, page = case["B"], case["N"], case["Hkv"], s["page"]
    parent, tokens, target, table, cnt, lens = (x.tolist() if torch.is_tensor(x) else x for x in (
        s["parent"], s["tokens"], s["argmax"], s["table"], _counts(case), _lengths(case)))
    src, dst = [], []
    for b in range(B):
        at, depth = 0, 0
        while at is not None:
            p = lens[b] + depth
            src.append(b * N + at)
            dst.append(table[b][p // page] * page + p % page)
            at = next((i for i in range(at + 1, cnt[b]) if parent[b][i] == at and tokens[b][i] == target[b][at]), None)
            depth += 1
    rows = s["kv"].double().reshape(B * N, 2, Hkv, -1)[torch.tensor(src, device="cuda")]
    dst = torch.tensor(dst, device="cuda")
    out = dict(path=None, n_keep=None, next=None)
    for name, side in (("kp", 0), ("vp", 1)):
        flat = s[name].double().transpose(1, 2).reshape(-1, Hkv, case["hd"])
        flat[dst] = rows[:, side]
        out[name] = flat.reshape(s["n_pages"], page, Hkv, -1).transpose(1, 2).contiguous()
    return out


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "rope":
        M, Hq, Hkv, hd, rot = case["M"], case["Hq"], case["Hkv"], case["hd"], case["rot"]
        i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
        angle = torch.remainder(s["pos"].double()[:, None] * torch.exp(-2 * i / rot * math.log(case["base"])), 2 * math.pi)
        heads = s["proj"].reshape(M, -1, hd)
        q = _exact_head(heads[:, :Hq], s["qn"], angle, case["inter"])
        k = _exact_head(heads[:, 2 * Hq: 2 * Hq + Hkv], s["kn"], angle, case["inter"])
        if not case["append"]:
            return dict(q=q.flatten(1), k=k.flatten(1))
        kp, vp = torch.zeros_like(s["kp"], dtype=torch.float64), torch.zeros_like(s["vp"], dtype=torch.float64)
        kt, vt = kp.transpose(1, 2).reshape(-1, Hkv, hd), vp.transpose(1, 2).reshape(-1, Hkv, hd)
        kt[s["slots"]], vt[s["slots"]] = k, heads[:, 2 * Hq + Hkv:].double()
        back = lambda x: x.reshape(s["n_pages"], s["page"], Hkv, hd).transpose(1, 2).contiguous()  # noqa: E731
        return dict(q=q.flatten(1), kp=back(kt), vp=back(vt))
    if op == "pages":
        return None          # whole numbers
    if op == "commit":
        return _exact_commit(case, s)
    B, N, Hq, Hkv, hd = (case[k] for k in ("B", "N", "Hq", "Hkv", "hd"))
    G = Hq // Hkv
    parent, lens, cnt = s["parent"].tolist(), _lengths(case), _counts(case)
    rows = s["proj"].reshape(B, N, -1, hd)
    out = torch.zeros((B, N, Hq, hd), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, L = cnt[b], lens[b]
        path = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            a = i
            while a >= 0:
                path[i, a] = True
                a = parent[b][a]
        path = path.cuda()
        pages = s["table"][b].long()
        for h in range(Hkv):
            kc = s["kp"][pages, h].reshape(-1, hd)[:L].double()
            vc = s["vp"][pages, h].reshape(-1, hd)[:L].double()
            kt, vt = rows[b, :n, 2 * Hq + h].double(), rows[b, :n, 2 * Hq + Hkv + h].double()
            q = rows[b, :n, h * G: (h + 1) * G].double()
            sc = torch.einsum("ngd,ld->ngl", q, kc) / math.sqrt(hd)
            st = (torch.einsum("ngd,ld->ngl", q, kt) / math.sqrt(hd)).masked_fill(~path[:, None], -math.inf)
            lse = torch.logaddexp(torch.logsumexp(sc, -1), torch.logsumexp(st, -1))[..., None]
            out[b, :n, h * G: (h + 1) * G] = torch.einsum("ngl,ld->ngd", (sc - lse).exp(), vc) + \
                torch.einsum("ngl,ld->ngd", (st - lse).exp(), vt)
            del sc, st
    if case["gate"]:
        out = out / (1 + torch.exp(-rows[:, :, Hq: 2 * Hq].double()))
    return out.reshape(B * N, Hq * hd)
