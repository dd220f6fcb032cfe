"""The paged-cache operators: what they compute, and the calls that reach them.

A server holds its full KV cache in pages and feeds batches in which every
sequence brings its own number of new tokens ("chunk"): one while decoding, a
drafted block while verifying, hundreds while a prompt is read in.  Four
operators carry such a batch:

  append  per-head RMS norm of queries and keys, position rotation, and the
          write of the new keys and values into the pages
  attn    causal attention of the chunks over the pages
  mass    the same, adding each cached token's attention weight to its score
  evict   the best tokens of every (sequence, kv head) by score, and the newest
          ones, moved to other pages

`run` computes them with elementary torch operations, or with `own` by the
framework's entry points.
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases --
def listed():
    dec = dict(Hq=32, Hkv=8, d=128, page=64, dtype="bf16")
    return [
        # one decode step of 16 sequences: a few hundred kB, launch latency counts
        dict(name="append decode", op="append", B=16, n=1, ragged=0, ctx=500, pos0=30000, rotary=128, norm=True, **dec),
        # prompts read in chunks: 5 sequences, 4670 tokens in one batch
        dict(name="append prompts", op="append", B=5, n=3000, ragged=1, ctx=100, pos0=100000, rotary=128, norm=True,
             **dec),
        # the shortest call: one sequence, one token, a short context
        dict(name="attn one token", op="attn", B=1, n=1, ragged=0, ctx=200, Hq=8, Hkv=8, d=64, page=16, dtype="bf16"),
        # a decode step of 16 sequences with 32k tokens each
        dict(name="attn decode", op="attn", B=16, n=1, ragged=0, ctx=32768, **dec),
        # verification of 32 drafts and the pending token over the same cache
        dict(name="attn verify", op="attn", B=16, n=33, ragged=0, ctx=32768, **dec),
        # a chunk of a long prompt
        dict(name="attn prompt chunk", op="attn", B=1, n=2048, ragged=0, ctx=30000, **dec),
        # a mixed batch: chunks and contexts of every length, 7 query heads per kv head
        dict(name="attn mixed", op="attn", B=9, n=700, ragged=2, ctx=20000, Hq=28, Hkv=4, d=128, page=16,
             dtype="bf16"),
        # the fp32 model of the losslessness checks: drafted blocks over short contexts
        dict(name="attn fp32", op="attn", B=4, n=17, ragged=3, ctx=2000, Hq=4, Hkv=2, d=64, page=32, dtype="fp32"),
        # a decode step that keeps scores
        dict(name="mass decode", op="mass", B=16, n=1, ragged=0, ctx=32768, **dec),
        # prompt chunks whose attention ranks the cached tokens
        dict(name="mass prompt chunks", op="mass", B=2, n=512, ragged=0, ctx=16000, **dec),
        # four long sequences cut to a quarter plus the newest 256 tokens
        dict(name="evict long", op="evict", B=4, ctx=131072, ragged=0, top=32768, recent=256, Hkv=8, d=128, page=64,
             dtype="bf16"),
        # short ragged sequences, some below the budget
        dict(name="evict short", op="evict", B=7, ctx=3500, ragged=5, top=600, recent=65, Hkv=2, d=64, page=16,
             dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "mass", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
    c = dict(op=op, dtype=dtype, d=d, page=page, Hkv=Hkv, ragged=rng.randrange(1, 1 << 20))
    if op == "append":
        n = _log(rng, 1, 4000)
        c.update(Hq=Hq, n=n, B=_log(rng, 1, max(1, min(64, 4000 // n))), ctx=rng.randrange(0, 300),
                 pos0=_log(rng, 1, 1000000), rotary=rng.choice([d, d, d // 2]), norm=rng.random() < 0.7)
    elif op == "evict":
        L = _log(rng, 40, 131072)
        c.update(B=_log(rng, 1, max(1, min(32, 131072 * 4 // L))), ctx=L, top=max(1, int(L * rng.uniform(0.05, 0.6))),
                 recent=rng.randrange(0, 300))
    else:
        n = _log(rng, 1, 1500)
        ctx = _log(rng, 1, 30000)
        most = 3e4 * 2048 * 32 * 128 / (8 if dtype == "fp32" else 1)       # rows x keys x channels of the largest
        B = _log(rng, 1, 24)
        while B > 1 and (B * n * (n + ctx) * Hq * d > most or B * (ctx + n) * Hkv > 16 * 32768 * 4):
            B -= 1
        while n > 1 and n * (n + ctx) * Hq * d > most:
            n = n * 2 // 3
        c.update(Hq=Hq, n=n, ctx=ctx, B=B)
    return c


def _lengths(case):
    """(chunk lengths, context lengths) of the case's sequences."""
    B, n, ctx = case["B"], case.get("n", 0), case["ctx"]
    if not case["ragged"]:
        return [n] * B, [ctx] * B
    r = random.Random(case["ragged"])
    ns = [r.randint(1, n) if n else 0 for _ in range(B)]
    cs = [r.randint(0, ctx) for _ in range(B)]
    if case["op"] not in ("append", "evict") and B > 2:
        ns[0], cs[1] = 1, 0                       # a decode step and a fresh prompt among the chunks
    cs[-1] = ctx
    return ns, cs


def _kept(L, case):
    return min(case["top"], max(L - case["recent"], 0)) + min(case["recent"], L)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    ns, cs = _lengths(case)
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "append":
        T, Hq = sum(ns), case["Hq"]
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * d * e + 4 * T, "flops": 10 * T * (Hq + Hkv) * d}
    if case["op"] == "evict":
        k = sum(_kept(L, case) for L in cs) * Hkv
        return {"bytes": 4 * Hkv * sum(cs) + k * (4 * d * e + 12), "flops": Hkv * sum(cs)}
    Hq, L = case["Hq"], sum(ns) + sum(cs)
    rows = sum(n * c + n * (n + 1) // 2 for n, c in zip(ns, cs))
    b = 2 * sum(ns) * Hq * d * e + 2 * L * Hkv * d * e
    if case["op"] == "mass":
        b += 8 * L * Hkv
    return {"bytes": b, "flops": 4 * rows * Hq * d}


# ------------------------------------------------------------------ inputs --
def _pool(case, lens, gen, dtype, spare=3):
    """A page pool holding sequences of `lens` tokens on pages in random order;
    table entries past a sequence's last page are -1."""
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    blocks = [-(-L // page) for L in lens]
    n_pages, width = sum(blocks) + spare, max(max(blocks), 1)
    order = torch.randperm(n_pages, generator=gen, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(blocks):
        table[b, :m] = order[at:at + m]
        at += m
    return n_pages, table, (n_pages, Hkv, page, d)


def prepare(case, seed):
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ns, cs = _lengths(case)
    B, d, Hkv = case["B"], case["d"], case["Hkv"]
    i32 = dict(dtype=torch.int32, device="cuda")

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype) * scale

    lens = [n + c for n, c in zip(ns, cs)]
    n_pages, table, shape = _pool(case, lens, gen, dtype)
    s = dict(case=case, dtype=dtype, ns=ns, cs=cs, lens=lens, table=table, n_pages=n_pages, scale=d ** -0.5)
    s["ctx"] = torch.tensor(cs, **i32)
    s["max_len"] = max(lens)
    if case["op"] == "evict":
        s["k"], s["v"] = normal(*shape), normal(*shape)
        S = table.shape[1] * case["page"]
        # accumulated weight falls off as 1 / rank^1.1 over shuffled positions; the tail was never looked at
        rank = torch.rand(B, Hkv, S, generator=gen, device="cuda").argsort(-1).argsort(-1).float() + 1
        s["scores"] = torch.where(rank <= 0.3 * s["max_len"], rank.pow(-1.1), torch.zeros_like(rank))
        kept = [_kept(L, case) for L in lens]
        n2, table2, shape2 = _pool(case, kept, gen, dtype, spare=1)
        s["k2"], s["v2"] = torch.zeros(*shape2, dtype=dtype, device="cuda"), torch.zeros(*shape2, dtype=dtype,
                                                                                         device="cuda")
        s["table2"], s["n_pages2"], s["most"] = table2, n2, max(max(kept), 1)
        s["len2"] = torch.zeros(B, **i32)
        s["kept"] = torch.full((B, Hkv, s["most"]), -1, **i32)
        s["scores2"] = torch.zeros(B, Hkv, s["most"], device="cuda")
        # a page of the second pool that no table names takes what is not kept
        used = set(table2.flatten().tolist())
        s["spare"] = next(p for p in range(n2) if p not in used)
    else:
        Hq = case["Hq"]
        T = sum(ns)
        start = [0]
        for n in ns:
            start.append(start[-1] + n)
        s["start"] = torch.tensor(start, **i32)
        s["T"], s["max_n"] = T, max(ns)
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(ns, device="cuda"))
        s["seq"] = seq                                        # sequence of each new token
        s["at"] = torch.arange(T, device="cuda") - s["start"][seq].long()   # its place in the chunk
        if case["op"] == "append":
            s["qkv"] = normal(T, (Hq + 2 * Hkv) * d)
            s["qg"], s["kg"] = normal(d, scale=0.1) + 1, normal(d, scale=0.1) + 1
            s["pos"] = (s["at"] + case["pos0"] + 17 * seq).int()
            s["q"] = torch.zeros(T, Hq, d, dtype=dtype, device="cuda")
            s["k"], s["v"] = torch.zeros(*shape, dtype=dtype, device="cuda"), torch.zeros(*shape, dtype=dtype,
                                                                                          device="cuda")
        else:
            s["q"] = normal(T, Hq, d, scale=1.5)
            s["k"], s["v"] = normal(*shape), normal(*shape)
            s["out"] = torch.zeros(T, Hq, d, dtype=dtype, device="cuda")
            if case["op"] == "mass":
                s["scores"] = torch.rand(B, Hkv, table.shape[1] * case["page"], generator=gen, device="cuda")
    if own:
        from lossless_draft_verify_gb300 import vc
        s["cache"] = vc.PagedCache(s["k"], s["v"], table)
        if case["op"] == "append":
            s["rope"] = vc.vc_rope_init(case["rotary"], 500000.0)
        elif case["op"] == "evict":
            s["cache2"] = vc.PagedCache(s["k2"], s["v2"], s["table2"])
        elif case["op"] == "mass":
            s["ws"] = vc.Workspace(vc.vc_paged_attn_h2o_workspace_bytes(s["cache"], s["T"], case["Hq"]))
        else:
            s["ws"] = vc.Workspace(vc.vc_paged_attn_workspace_bytes(s["cache"], s["T"], case["Hq"]))
    return s


# --------------------------------------------------------------------- run --
def run(s):
    return _RUN[s["case"]["op"]](s)


def _append(s):
    c = s["case"]
    Hq, Hkv, d, r = c["Hq"], c["Hkv"], c["d"], c["rotary"]
    if own:
        from lossless_draft_verify_gb300 import vc
        vc.vc_paged_append(s["qkv"], s["cache"], s["start"], s["ctx"], s["q"], s["rope"], positions=s["pos"],
                           q_gain=s["qg"] if c["norm"] else None, k_gain=s["kg"] if c["norm"] else None, eps=EPS)
        return s["q"], s["k"], s["v"]
    x = s["qkv"].view(s["T"], Hq + 2 * Hkv, d)
    qk = x[:, :Hq + Hkv].float()
    if c["norm"]:
        gain = torch.cat([s["qg"].float().expand(Hq, d), s["kg"].float().expand(Hkv, d)])
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * gain
    w = 500000.0 ** (-2.0 * torch.arange(r // 2, device="cuda", dtype=torch.float64) / r)
    angle = s["pos"].double()[:, None, None] * w
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = qk[..., :r // 2], qk[..., r // 2:r]
    qk = torch.cat([a * cos - b * sin, b * cos + a * sin, qk[..., r:]], -1).to(s["dtype"])
    slot = s["ctx"].long()[s["seq"]] + s["at"]
    where = s["table"].long()[s["seq"], slot // c["page"]]
    s["q"].copy_(qk[:, :Hq])
    s["k"][where, :, slot % c["page"]] = qk[:, Hq:]
    s["v"][where, :, slot % c["page"]] = x[:, Hq + Hkv:]
    return s["q"], s["k"], s["v"]


def _rows(pages, table, n):
    """[B][Hkv][tokens][d] in fp32 of the first n tokens (whole pages)."""
    blocks = -(-n // pages.shape[2])
    x = pages[table[:, :blocks].long().clamp(min=0)].float()
    return x.transpose(1, 2).reshape(table.shape[0], pages.shape[1], -1, pages.shape[3])


def _attn(s):
    c = s["case"]
    if own:
        from lossless_draft_verify_gb300 import vc
        if c["op"] == "mass":
            vc.vc_paged_attn_h2o(s["q"], s["cache"], s["start"], s["ctx"], s["scale"], s["out"], s["scores"], s["ws"])
            return s["out"], s["scores"]
        vc.vc_paged_attn(s["q"], s["cache"], s["start"], s["ctx"], s["scale"], s["out"], s["ws"])
        return s["out"]
    B, Hkv, G, d, N = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["d"], s["max_n"]
    k, v = _rows(s["k"], s["table"], s["max_len"]), _rows(s["v"], s["table"], s["max_len"])
    S = k.shape[2]
    q = torch.zeros(B, N, Hkv, G, d, device="cuda")
    q[s["seq"], s["at"]] = s["q"].view(-1, Hkv, G, d).float()
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, d)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, N, G, S)
    last = s["ctx"].long()[:, None] + torch.arange(N, device="cuda")
    hidden = torch.arange(S, device="cuda") > last[:, :, None]
    p.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p.view(B, Hkv, N * G, S), v).view(B, Hkv, N, G, d).permute(0, 2, 1, 3, 4)
    s["out"].copy_(o[s["seq"], s["at"]].reshape(-1, c["Hq"], d))
    if c["op"] != "mass":
        return s["out"]
    real = torch.arange(N, device="cuda") < (s["start"][1:] - s["start"][:-1])[:, None]
    s["scores"][..., :S] += p.mul_(real[:, None, :, None, None]).sum((2, 3))
    return s["out"], s["scores"]


def _evict(s):
    c = s["case"]
    if own:
        from lossless_draft_verify_gb300 import vc
        # no more than the longest sequence has: what the outputs have room for
        recent = min(c["recent"], s["max_len"])
        top = min(c["top"], s["max_len"] - recent)
        vc.vc_paged_evict(s["scores"], s["cache"], s["ctx"], top, recent, s["cache2"], s["len2"], s["kept"],
                          scores_out=s["scores2"])
        return s["kept"], s["len2"], s["k2"], s["v2"], s["scores2"]
    B, Hkv, page, most = c["B"], c["Hkv"], c["page"], s["most"]
    L = s["ctx"].long()[:, None, None]
    x = s["scores"][..., :s["max_len"]]
    slot = torch.arange(x.shape[-1], device="cuda")
    x = torch.where(slot >= L, -math.inf, torch.where(slot >= L - c["recent"], math.inf, x))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    n = torch.clamp(L - c["recent"], min=0).clamp(max=c["top"]) + torch.clamp(L, max=c["recent"])
    best = torch.where(slot[:most] < n, order[..., :most], x.shape[-1])
    kept = torch.sort(best, dim=-1).values
    ok = slot[:most] < n
    kept = torch.where(ok, kept, 0)
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    src = s["table"].long()[b, kept // page].clamp(min=0)
    j = slot[:most].expand(B, Hkv, most)
    dst = torch.where(ok, s["table2"].long()[b, j // page], s["spare"])
    for pages, pages2 in ((s["k"], s["k2"]), (s["v"], s["v2"])):
        pages2[dst, h, j % page] = pages[src, h, kept % page]
        pages2[s["spare"]] = 0
    s["kept"].copy_(torch.where(ok, kept, -1))
    s["scores2"].copy_(torch.where(ok, s["scores"][b, h, kept], 0))
    s["len2"].copy_(n.view(-1))
    return s["kept"], s["len2"], s["k2"], s["v2"], s["scores2"]


_RUN = {"append": _append, "attn": _attn, "mass": _attn, "evict": _evict}


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    ns, cs, page, Hkv = s["ns"], s["cs"], case["page"], case["Hkv"]
    table = s["table"].tolist()

    def tokens(pages, b, h, n):
        used = table[b][:-(-n // page)]
        return torch.cat([pages[p, h] for p in used])[:n].double() if n else pages[0, h, :0].double()

    if case["op"] == "append":
        Hq, d, r = case["Hq"], case["d"], case["rotary"]
        x = s["qkv"].double().reshape(s["T"], -1, d)
        y = x.clone()
        pos = s["pos"].double()
        for h in range(Hq + Hkv):
            u = x[:, h]
            if case["norm"]:
                g = (s["qg"] if h < Hq else s["kg"]).double()
                u = u / ((u * u).sum(1) / d + EPS).sqrt()[:, None] * g
            y[:, h] = u
            for j in range(r // 2):
                t = pos * math.pow(500000.0, -2.0 * j / r)
                y[:, h, j] = u[:, j] * torch.cos(t) - u[:, j + r // 2] * torch.sin(t)
                y[:, h, j + r // 2] = u[:, j] * torch.sin(t) + u[:, j + r // 2] * torch.cos(t)
        k, v = s["k"].double(), s["v"].double()
        row = 0
        for b, (n, c) in enumerate(zip(ns, cs)):
            i = 0
            while i < n:                                # runs of tokens that share a page
                o = (c + i) % page
                m = min(n - i, page - o)
                p = table[b][(c + i) // page]
                k[p, :, o:o + m] = y[row + i:row + i + m, Hq:Hq + Hkv].transpose(0, 1)
                v[p, :, o:o + m] = y[row + i:row + i + m, Hq + Hkv:].transpose(0, 1)
                i += m
            row += n
        return y[:, :Hq], k, v
    if case["op"] == "evict":
        kept, len2 = s["kept"].clone(), s["len2"].clone()
        k2, v2, scores2 = s["k2"].double(), s["v2"].double(), s["scores2"].double()
        to = s["table2"].tolist()
        for b, L in enumerate(cs):
            n, old = _kept(L, case), max(L - case["recent"], 0)
            len2[b] = n
            for h in range(Hkv):
                best = torch.sort(s["scores"][b, h, :old].double(), descending=True, stable=True).indices
                keep = torch.cat([best[:n - (L - old)].sort().values, torch.arange(old, L, device="cuda")])
                kept[b, h, :n] = keep.int()
                scores2[b, h, :n] = s["scores"][b, h, keep].double()
                for pages, new in ((s["k"], k2), (s["v"], v2)):
                    rows = tokens(pages, b, h, L)[keep]
                    for i in range(0, n, page):
                        new[to[b][i // page], h, :min(page, n - i)] = rows[i:i + page]
        return kept, len2, k2, v2, scores2
    Hq, d = case["Hq"], case["d"]
    out = torch.empty(s["T"], Hq, d, dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if case["op"] == "mass" else None
    row = 0
    for b, (n, c) in enumerate(zip(ns, cs)):
        sees = torch.arange(n + c, device="cuda")[None] <= c + torch.arange(n, device="cuda")[:, None]
        for h in range(Hkv):
            k, v = tokens(s["k"], b, h, n + c), tokens(s["v"], b, h, n + c)
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                x = (s["q"][row:row + n, g].double() @ k.T) / math.sqrt(d)
                e = torch.where(sees, (x - torch.where(sees, x, -math.inf).max(1, keepdim=True).values).exp(), 0.0)
                e = e / e.sum(1, keepdim=True)
                out[row:row + n, g] = e @ v
                if scores is not None:
                    scores[b, h, :n + c] += e.sum(0)
        row += n
    return out if scores is None else (out, scores)
