"""Cases of the operators that decode and verify over an 8-bit KV cache: new K and V rows quantised
into the cache, attention of decode rows over it (whole contexts, or a sliding window with a few
first tokens kept), and the scores of a step's logits: log probabilities of given tokens, entropies
and top alternatives.

``run`` computes an operator in plain torch (32 bits, rounded once at the end) or, with ``own``
true, calls the library's entry points.

The cache: a head of a token is hd values of 8 bits (e4m3) and one fp32 scale, for K and for V:
den = min(max(largest |x|, 448 2^-40), 448 2^60), scale = den / 448, code = e4m3(448 x / den).
"""
import math
import random

import torch

own = False

KINDS = ("append", "attn", "score")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the attention layer of one verify step: 8 new rows into the pages
        dict(name="append-step", op="append", B=1, R=8, Hkv=4, hd=256, ctx=2183, page=64),
        # a batch in flight, 5 drafts or fewer per sequence
        dict(name="append-batch", op="append", B=64, R=5, Hkv=8, hd=128, ctx=500, page=128),
        # a long prompt enters a contiguous cache
        dict(name="append-prompt", op="append", B=1, R=8192, Hkv=8, hd=128, ctx=1, page=0),
        # the smallest attention layer decodes a token over a short context
        dict(name="attn-tiny", op="attn", B=1, R=1, Hq=2, Hkv=1, hd=64, ctx=128, page=0, window=0, sinks=0, gate=False),
        # one verify step at the usual context, gated attention
        dict(name="attn-verify", op="attn", B=1, R=8, Hq=24, Hkv=4, hd=256, ctx=2183, page=64, window=0, sinks=0, gate=True),
        # a batch decodes one token each, ragged lengths
        dict(name="attn-batch", op="attn", B=32, R=1, Hq=32, Hkv=8, hd=128, ctx=8000, page=128, window=0, sinks=0, gate=False),
        # a batch far into its contexts sees a window and the first tokens
        dict(name="attn-window", op="attn", B=8, R=4, Hq=24, Hkv=4, hd=256, ctx=32768, page=64, window=4096, sinks=4, gate=False),
        # one verify step over a long context
        dict(name="attn-long", op="attn", B=1, R=8, Hq=24, Hkv=4, hd=256, ctx=131072, page=64, window=0, sinks=0, gate=True),
        # one token of the smallest vocabulary scored, nothing else asked
        dict(name="score-one", op="score", M=1, V=2048, top=0, dtype="float32", masked=0.0),
        # the logits of one verify step with the alternatives that a client may ask for
        dict(name="score-verify", op="score", M=8, V=151936, top=20, dtype="float32", masked=0.0),
        # a batch under constrained decoding, logits of another engine's 16 bits, an odd vocabulary
        dict(name="score-batch", op="score", M=500, V=50257, top=5, dtype="bfloat16", masked=0.3),
        # a whole prompt's tokens scored
        dict(name="score-prompt", op="score", M=2048, V=151936, top=1, dtype="float32", masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(KINDS)
    if op == "append":
        Hkv, hd = rng.choice([(4, 256), (8, 128), (2, 64), (1, 64), (2, 256), (3, 128)])
        B = _log_int(rng, 1, 128)
        return dict(op=op, B=B, R=_log_int(rng, 1, 8192 // B), Hkv=Hkv, hd=hd, ctx=_log_int(rng, 1, 1000),
                    page=rng.choice([0, 64, 128, 192]))
    if op == "attn":
        Hq, Hkv, hd = rng.choice([(24, 4, 256), (32, 8, 128), (6, 2, 64), (16, 2, 256), (8, 8, 128), (5, 1, 64)])
        B, R = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        most = max(64, min(131072, 290_000_000 // (B * (2 * Hkv * hd + Hq * R))))   # positions: bounds the whole's work
        ctx = _log_int(rng, 1, most)
        window = 0 if rng.random() < 0.5 else _log_int(rng, 1, max(2, ctx))
        return dict(op=op, B=B, R=R, Hq=Hq, Hkv=Hkv, hd=hd, ctx=ctx, page=rng.choice([0, 64, 192, 256]), window=window,
                    sinks=rng.choice([0, 1, 4, 100]) if window else 0, gate=rng.random() < 0.5)
    V = _log_int(rng, 1000, 200000)
    return dict(op=op, M=_log_int(rng, 1, min(8192, 300_000_000 // V)), V=V, top=rng.choice([0, 1, 2, 5, 11, 20, 32]),
                dtype=rng.choice(["float32", "bfloat16"]), masked=rng.choice([0.0, 0.3, 0.9]))


# --------------------------------------------- what a case fixes by itself

def _lengths(case):
    """Visible positions of each sequence's first row, ragged: the first the longest, the others down to about half."""
    ctx = case["ctx"]
    return [ctx - (b * 7919) % (ctx // 2 + 1) for b in range(case["B"])]


def _counts(case):
    """Rows of each sequence: the first full, the others down to about half."""
    R = case["R"]
    return [R - (b * 31) % (R // 2 + 1) for b in range(case["B"])]


def _ceil(a, b):
    return -(-a // b)


def _seen(case, length):
    """Positions that a row of this visible length attends to."""
    w = case["window"]
    return length if not w or w >= length else w + min(case["sinks"], length - w)


def work(case):
    op = case["op"]
    if op == "append":
        n = sum(_counts(case)) * case["Hkv"]
        return {"bytes": 2 * n * (3 * case["hd"] + 4), "flops": 4 * n * case["hd"]}
    if op == "attn":
        Hq, Hkv, hd = case["Hq"], case["Hkv"], case["hd"]
        lens, cnt = _lengths(case), _counts(case)
        # a sequence's rows see the window of the first, and one position more each
        pos = sum(_seen(case, x) + n - 1 for x, n in zip(lens, cnt))
        rows = sum(cnt)
        return {"bytes": pos * Hkv * (2 * hd + 8) + (6 if case["gate"] else 4) * rows * Hq * hd,
                "flops": sum(4 * Hq * hd * _seen(case, x + r) for x, n in zip(lens, cnt) for r in range(n))}
    M, V, top = case["M"], case["V"], case["top"]
    return {"bytes": M * V * (4 if case["dtype"] == "float32" else 2) + M * (12 + 8 * top), "flops": 5 * M * V}


# ---------------------------------------------------------------- inputs

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


def _cache(g, n_pages, Hkv, page, hd):
    """Codes of normal values and scales that differ from token to token, page by page."""
    codes = torch.empty((n_pages, Hkv, page, hd), dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, 32_000_000 // (Hkv * page * hd))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i), Hkv, page, hd), generator=g, device="cuda")
        codes[i: i + step] = (x * 130).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.exp(torch.randn((n_pages, Hkv, page), generator=g, device="cuda") * 0.3) / 130
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 9176 + 5)
    s = dict(case=case)
    op = case["op"]
    if op == "score":
        M, V = case["M"], case["V"]
        x = torch.randn((M, V), generator=g, device="cuda").mul_(2.5)
        # a model is sure of a few tokens now and then
        peak = torch.randint(0, V, (M, 3), generator=g, device="cuda")
        x.scatter_add_(1, peak, torch.rand((M, 3), generator=g, device="cuda") * 12)
        token = torch.where(torch.rand(M, generator=g, device="cuda") < 0.7, peak[:, 0],
                            torch.randint(0, V, (M,), generator=g, device="cuda"))
        if case["masked"]:
            off = torch.rand(V, generator=g, device="cuda") < case["masked"]
            off[: V // 16] = False
            x.masked_fill_(off, -math.inf)
            token = torch.where(off[token], token % (V // 16), token)      # what was sampled was allowed
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        del x
        s["tokens"] = token.to(torch.int32)
        s["logprob"] = torch.zeros(M, device="cuda")
        s["entropy"] = torch.zeros(M, device="cuda")
        if case["top"]:
            s["ids"] = torch.zeros((M, case["top"]), dtype=torch.int32, device="cuda")
            s["top"] = torch.zeros((M, case["top"]), device="cuda")
        if own:
            from bit_exact_speculative_gb300 import xv
            s["ws"] = xv.workspace(xv.xv_logprobs_workspace_size(M, V, case["top"]))
        return s
    B, R, Hkv, hd = case["B"], case["R"], case["Hkv"], case["hd"]
    lens, cnt = _lengths(case), _counts(case)
    s["ctx"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["rows"] = torch.tensor(cnt, dtype=torch.int32).cuda()
    s["table"], s["page"], s["n_pages"] = _pool_of(case, seed, [x + R for x in lens])
    s["k"], s["ks"] = _cache(g, s["n_pages"], Hkv, s["page"], hd)
    s["v"], s["vs"] = _cache(g, s["n_pages"], Hkv, s["page"], hd)
    if op == "append":
        # rows of a projection [k | v], tokens of differing sizes
        size = torch.exp(torch.randn((B * R, 1), generator=g, device="cuda") * 0.5)
        s["kv"] = (torch.randn((B * R, 2 * Hkv * hd), generator=g, device="cuda") * size).to(torch.bfloat16)
    else:
        Hq = case["Hq"]
        # rows of a projection [q | gate]
        s["proj"] = _normal(g, (B * R, 2 * Hq * hd))
        s["out"] = torch.zeros((B * R, Hq * hd), dtype=torch.bfloat16, device="cuda")
    if own:
        from bit_exact_speculative_gb300 import xv
        s["cache"] = xv.kv_q8(s["k"], s["v"], s["ks"], s["vs"])
        s["pages"] = xv.kv_pages(s["table"], s["page"], s["n_pages"])
        if op == "attn":
            s["ws"] = xv.workspace(xv.xv_attn_q8_workspace_size(B, R, case["Hq"], hd, case["ctx"] + R - 1,
                                                                window=case["window"], sinks=case["sinks"]))
    return s


# ------------------------------------------------------------- plain forms

def _plain_append(s):
    c = s["case"]
    B, R, Hkv, hd = c["B"], c["R"], c["Hkv"], c["hd"]
    x = s["kv"].reshape(B, R, 2, Hkv, hd).float()
    den = x.abs().amax(-1, keepdim=True).clamp(448 * 2.0 ** -40, 448 * 2.0 ** 60)
    codes = (x * 448 / den).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = den[..., 0] / 448
    r = torch.arange(R, device="cuda")
    live = r[None, :] < s["rows"][:, None]
    pos = s["ctx"].long()[:, None] - 1 + r
    pg, at = torch.gather(s["table"].long(), 1, pos // s["page"]), pos % s["page"]
    b, i = live.nonzero(as_tuple=True)
    pg, at = pg[b, i], at[b, i]
    for side, (code, sc) in enumerate((("k", "ks"), ("v", "vs"))):
        s[code].view(torch.uint8)[pg, :, at] = codes[b, i, side].view(torch.uint8)
        s[sc][pg, :, at] = scale[b, i, side]
    return dict(k=s["k"], v=s["v"], ks=s["ks"], vs=s["vs"])


def _plain_attn(s):
    c = s["case"]
    B, R, Hq, Hkv, hd = c["B"], c["R"], c["Hq"], c["Hkv"], c["hd"]
    G = Hq // Hkv
    rows = s["proj"].reshape(B, R, 2, Hq, hd)
    q = rows[:, :, 0].reshape(B, R, Hkv, G, hd).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * R, hd)
    most = c["ctx"] + R - 1

    def whole(codes, scale):   # [B, Hkv, positions, hd]: the pages in order, as values
        t = s["table"].long()
        x = codes.view(torch.uint8)[t].transpose(1, 2).flatten(2, 3)[:, :, :most].view(torch.float8_e4m3fn).float()
        return x.mul_(scale[t].transpose(1, 2).flatten(2, 3)[:, :, :most, None])

    p = torch.arange(most, device="cuda")
    length = s["ctx"][:, None] + torch.arange(R, device="cuda")          # [B, R] visible positions of each row
    see = p < length[..., None]
    if c["window"]:
        see &= (p >= length[..., None] - c["window"]) | (p < c["sinks"])
    live = torch.arange(R, device="cuda")[None, :] < s["rows"][:, None]
    see |= ~live[..., None]
    a = q.float() @ whole(s["k"], s["ks"]).transpose(-1, -2)
    a = a.reshape(B, Hkv, G, R, -1).mul_(hd ** -0.5).masked_fill_(~see[:, None, None], -math.inf)
    a = a.sub_(a.amax(-1, keepdim=True)).exp_()
    total = a.sum(-1, keepdim=True)
    o = (a.flatten(2, 3) @ whole(s["v"], s["vs"])).reshape(B, Hkv, G, R, hd) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, R, Hq, hd)
    if c["gate"]:
        o = o * torch.sigmoid(rows[:, :, 1].float())
    return o.masked_fill(~live[..., None, None], 0).reshape(B * R, -1).to(torch.bfloat16)


def _plain_score(s):
    x = s["logits"].float()
    M, V = x.shape
    d = x - x.amax(-1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(-1)
    lse = torch.log(total)
    entropy = lse - (e.mul_(d.clamp(min=-1e30))).sum(-1) / total
    del e
    out = dict(logprob=torch.gather(d, 1, s["tokens"].long()[:, None])[:, 0] - lse, entropy=entropy)
    n = s["case"]["top"]
    if n:
        index = torch.arange(V, dtype=torch.int32, device="cuda")
        ids, top = [], []
        for _ in range(n):
            best = d.amax(-1, keepdim=True)
            at = torch.where(d == best, index, V).amin(-1, keepdim=True)      # the lowest of equals
            ids.append(at)
            top.append(best)
            d.scatter_(1, at.long(), -math.inf)
        out["ids"], out["top"] = torch.cat(ids, 1).int(), torch.cat(top, 1) - lse[:, None]
    return out


# --------------------------------------------------------------------- run

def _own(s):
    from bit_exact_speculative_gb300 import xv
    c = s["case"]
    if c["op"] == "score":
        if c["top"]:
            xv.xv_logprobs(s["logits"], s["tokens"], s["logprob"], s["ws"], entropy=s["entropy"], top_ids=s["ids"],
                           top_logprobs=s["top"])
            return dict(logprob=s["logprob"], entropy=s["entropy"], ids=s["ids"], top=s["top"])
        xv.xv_logprobs(s["logits"], s["tokens"], s["logprob"], s["ws"], entropy=s["entropy"])
        return dict(logprob=s["logprob"], entropy=s["entropy"])
    B, R, Hkv, hd = c["B"], c["R"], c["Hkv"], c["hd"]
    if c["op"] == "append":
        if c["page"]:
            xv.xv_kv_append_q8_paged(s["kv"], s["ctx"], R, B, Hkv, hd, s["pages"], s["cache"], n_rows=s["rows"])
        else:
            xv.xv_kv_append_q8(s["kv"], s["ctx"], R, B, Hkv, hd, s["page"], s["cache"], n_rows=s["rows"])
        return dict(k=s["k"], v=s["v"], ks=s["ks"], vs=s["vs"])
    Hq = c["Hq"]
    gate = s["proj"][:, Hq * hd:] if c["gate"] else None
    if c["page"]:
        xv.xv_attn_decode_rows_q8_paged(s["proj"], s["cache"], s["pages"], s["ctx"], R, B, Hq, Hkv, hd, c["ctx"] + R - 1,
                                        hd ** -0.5, s["out"], s["ws"], window=c["window"], sinks=c["sinks"], gate=gate,
                                        n_rows=s["rows"])
    else:
        xv.xv_attn_decode_rows_q8(s["proj"], s["cache"], s["ctx"], R, B, Hq, Hkv, hd, s["page"], c["ctx"] + R - 1,
                                  hd ** -0.5, s["out"], s["ws"], window=c["window"], sinks=c["sinks"], gate=gate,
                                  n_rows=s["rows"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return dict(append=_plain_append, attn=_plain_attn, score=_plain_score)[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_append(case, s):
    """The codes' values before their rounding, and the scales, where each sequence's rows go."""
    B, R, Hkv, hd, page = case["B"], case["R"], case["Hkv"], case["hd"], s["page"]
    table = s["table"].tolist()
    src, dst = [], []
    for b, (x, n) in enumerate(zip(_lengths(case), _counts(case))):
        for r in range(n):
            p = x - 1 + r
            src.append(b * R + r)
            dst.append(table[b][p // page] * page + p % page)
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    heads = s["kv"].double()[src].reshape(-1, 2, Hkv, hd)
    big = torch.maximum(heads.max(-1).values, -heads.min(-1).values)
    scale = torch.clamp(big, 448 / 2.0 ** 40, 448 * 2.0 ** 60) / 448
    value = torch.clamp(heads / scale[..., None], -448, 448)
    out = {}
    for side, name in enumerate(("k", "v")):
        flat = s[name].double().transpose(1, 2).reshape(-1, Hkv, hd)
        flat[dst] = value[:, side]
        out[name] = flat.reshape(s["n_pages"], page, Hkv, hd).transpose(1, 2).contiguous()
        flat = s[name + "s"].double().transpose(1, 2).reshape(-1, Hkv)
        flat[dst] = scale[:, side]
        out[name + "s"] = flat.reshape(s["n_pages"], page, Hkv).transpose(1, 2).contiguous()
    return out


def _exact_attn(case, s):
    B, R, Hq, Hkv, hd = (case[k] for k in ("B", "R", "Hq", "Hkv", "hd"))
    G = Hq // Hkv
    rows = s["proj"].reshape(B, R, 2 * Hq, hd)
    out = torch.zeros((B, R, Hq, hd), dtype=torch.float64, device="cuda")
    for b, (x, n) in enumerate(zip(_lengths(case), _counts(case))):
        far = x + n - 1
        first = max(0, x - case["window"]) if case["window"] else 0
        keep = sorted(set(range(min(case["sinks"], far))) | set(range(first, far))) if case["window"] else range(far)
        at = torch.tensor(list(keep), device="cuda")
        pg, row = s["table"][b].long()[at // s["page"]], at % s["page"]
        for h in range(Hkv):
            k = s["k"].view(torch.uint8)[pg, h, row].view(torch.float8_e4m3fn).double() * s["ks"][pg, h, row].double()[:, None]
            v = s["v"].view(torch.uint8)[pg, h, row].view(torch.float8_e4m3fn).double() * s["vs"][pg, h, row].double()[:, None]
            q = rows[b, :n, h * G: (h + 1) * G].double()
            sc = torch.einsum("rgd,ld->rgl", q, k) / math.sqrt(hd)
            for r in range(n):
                hide = at >= x + r
                if case["window"]:
                    hide |= (at < x + r - case["window"]) & (at >= case["sinks"])
                sc[r, :, hide] = -math.inf
            out[b, :n, h * G: (h + 1) * G] = torch.einsum("rgl,ld->rgd", (sc - torch.logsumexp(sc, -1, keepdim=True)).exp(), v)
    if case["gate"]:
        out = out / (1 + torch.exp(-rows[:, :, Hq:].double()))
    return out.reshape(B * R, Hq * hd)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    M, n = case["M"], case["top"]
    out = dict(logprob=torch.empty(M, dtype=torch.float64, device="cuda"), entropy=torch.empty(M, dtype=torch.float64, device="cuda"))
    if n:
        out.update(ids=None, top=torch.empty((M, n), dtype=torch.float64, device="cuda"))
    step = max(1, 100_000_000 // case["V"])
    for i in range(0, M, step):
        x = s["logits"][i: i + step].double()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        out["logprob"][i: i + step] = lp.gather(1, s["tokens"][i: i + step].long()[:, None])[:, 0]
        out["entropy"][i: i + step] = -torch.where(lp == -math.inf, 0.0, lp.exp() * lp).sum(-1)
        if n:
            out["top"][i: i + step] = lp.sort(-1, descending=True).values[:, :n]
    return out
