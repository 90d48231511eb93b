"""A bounded paged cache and the norm in front of the MoE layer: what is measured, in plain torch and through the library.

Four operators: `window` (attention over the paged cache with a sliding window and a few first tokens that stay visible),
`usage` (the attention weight that every cached token has received, added up over a call's tokens and heads), `evict` (each
kv head keeps the cached tokens of the largest usage, beside the first and the last ones, and moves them to new pages) and
`norm` (the residual's addition, root-mean-square norm, and the result in bf16 and in e4m3 with scales).

The cache is [pages, 2, kv heads, page size, head dim] (keys, values), bf16 or e4m3 with a float32 scale per kv head;
its pages are handed out in random order. Sizes: one GPU's share of GLM4-MoE attention under TP8 (12 query heads on 1
kv head, head dim 128), the unsharded heads (96 on 8), the layer's hidden size 5120, and generic ones.
"""
import math
import random

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one token of one sequence a little past its window: launch latency
        window("window decode one", 1, 1, 777, 512, 4, "bf16", ragged=False),
        # a serving batch deep in long generations; of each sequence the cache holds the window and the sinks alone
        window("window decode 64", 64, 1, 131072, 4096, 4, "bf16"),
        # a 16384-token chunk behind 16384 cached tokens, 8-bit cache
        window("window prefill 16k e4m3", 1, 16384, 32768, 4096, 4, "e4m3", page=64, ragged=False),
        # ragged prompts on the unsharded heads, a short window, capped scores, sinks that end inside a page
        window("window prefill ragged", 7, 2500, 9000, 1024, 37, "bf16", q_heads=96, kv_heads=8, cap=30.0),
        # a decoding step's weights: keys are read once
        usage("usage decode 64", 64, 1, 8192, "bf16"),
        # the last 64 tokens of a long prompt look at all of it, 8-bit cache, nothing known of the tokens before
        usage("usage last 64 of 131072", 1, 64, 131072, "e4m3", prev=False, ragged=False),
        # every token of a prompt, beside a cached part
        usage("usage prefill 4096", 2, 4096, 6000, "bf16", decay=0.9, ragged=False),
        # one sequence that has outgrown its budget by a few pages: launch latency
        evict("evict one", 1, 2112, 2048, 2048, 4, 256, "bf16", ragged=False),
        # prompts of many lengths cut to a budget, 8-bit cache; some are short enough to stay
        evict("evict 64 e4m3", 64, 16384, 4096, 4096, 4, 512, "e4m3", page=32),
        # long contexts on the unsharded heads
        evict("evict unsharded 24", 24, 16384, 4096, 4096, 64, 1024, "bf16", q_heads=96, kv_heads=8, page=64, ragged=False),
        # a decoding step, bf16 for the router and e4m3 for the experts
        norm("norm decode 64", 64, 5120, "row"),
        # a 16384-token chunk, one scale per 128 columns
        norm("norm 16384", 16384, 5120, "block"),
    ]


def heads(q_heads=12, kv_heads=1, dim=128, page=16):
    return {"q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page}


def window(name, seqs, nodes, kv, size, sinks, kind, cap=0.0, ragged=True, lens=1, **more):
    return {"name": name, "op": "window", "seqs": seqs, "nodes": nodes, "kv": kv, "window": size, "sinks": sinks, "kind": kind,
            "cap": cap, "ragged": ragged, "lens": lens, **heads(**more)}


def usage(name, seqs, nodes, kv, kind, cap=0.0, decay=1.0, prev=True, ragged=True, lens=1, **more):
    return {"name": name, "op": "usage", "seqs": seqs, "nodes": nodes, "kv": kv, "kind": kind, "cap": cap, "decay": decay,
            "prev": prev, "ragged": ragged, "lens": lens, **heads(**more)}


def evict(name, seqs, kv, limit, budget, sinks, recent, kind, ragged=True, lens=1, **more):
    return {"name": name, "op": "evict", "seqs": seqs, "nodes": 1, "kv": kv, "limit": limit, "budget": budget, "sinks": sinks,
            "recent": recent, "kind": kind, "ragged": ragged, "lens": lens, **heads(**more)}


def norm(name, tokens, hidden, scales, residual=True, bf16=True):
    return {"name": name, "op": "norm", "tokens": tokens, "hidden": hidden, "scales": scales, "residual": residual, "bf16": bf16}


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["window", "window", "usage", "evict", "norm"])
    if op == "norm":
        scales = rng.choice(["none", "row", "block"])
        hidden = rng.choice([128, 1024, 2048, 4096, 5120, 5120, 8192]) if scales == "block" else 8 * size(16, 1024)
        c = norm("", size(1, max(64, min(16384, 16384 * 5120 // hidden))), hidden, scales, residual=rng.random() < 0.8,
                 bf16=scales == "none" or rng.random() < 0.8)
        del c["name"]
        return c
    q_heads, kv_heads, dim = rng.choice([(12, 1, 128), (12, 1, 128), (96, 8, 128), (8, 2, 64), (16, 4, 128), (7, 1, 64),
                                         (8, 1, 256)])
    more = {"q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]),
            "kind": rng.choice(["bf16", "e4m3"]), "lens": rng.randrange(1 << 30), "ragged": rng.random() < 0.6}
    if op == "evict":
        budget = size(16, 8192)
        kv = budget + size(65, 122000)
        seqs = max(1, min(size(1, 96), (3 << 20) // (kv * kv_heads)))
        sinks = min(rng.choice([0, 4, size(1, 128)]), budget // 4)
        c = evict("", seqs, kv, budget + rng.choice([0, 0, 64]), budget, sinks, rng.choice([0, 1, budget // 4]), **more)
    else:
        nodes = rng.choice([1, 1, size(2, 64), size(65, 8192)])
        context = size(1, 131072) if nodes < 100 else rng.choice([0, size(16, 16384)])
        kv = nodes + context
        reach = size(16, 8192) if op == "window" else kv
        pairs = nodes * min(kv, reach + nodes) * q_heads * max(1, dim // 128)  # scores of the plain form
        while pairs > int(1.6e9):
            nodes, context = nodes // 2 + 1, context // 2
            kv = nodes + context
            pairs = nodes * min(kv, reach + nodes) * q_heads * max(1, dim // 128)
        seqs = max(1, min(size(1, 96), int(1.6e9) // pairs, (1 << 20) // (min(kv, reach + nodes) * kv_heads)))
        cap = rng.choice([0.0, 0.0, 30.0])
        if op == "window":
            c = window("", seqs, nodes, kv, reach, rng.choice([0, 4, size(1, 300)]), cap=cap, **more)
        else:
            c = usage("", seqs, nodes, kv, cap=cap, decay=rng.choice([1.0, 0.9]), prev=rng.random() < 0.7, **more)
    del c["name"]
    return c


def lengths(case):
    """Tokens of each sequence in this call, and its cached tokens after them."""
    r = random.Random(case["lens"])
    n, kv = [], []
    for _ in range(case["seqs"]):
        t = r.randint(max(1, case["nodes"] // 4), case["nodes"]) if case["ragged"] else case["nodes"]
        c = case["kv"] - case["nodes"]
        c = r.randint(c // 8, c) if case["ragged"] else c
        n.append(t)
        kv.append(c + t)
    return n, kv


def first_seen(case, n, kv):
    """The first cached token in the window of a sequence's first token."""
    return max(0, kv - n + 1 - case["window"])


def work(case):
    if case["op"] == "norm":
        t, h = case["tokens"], case["hidden"]
        groups = {"none": 0, "row": 1, "block": h // 128}[case["scales"]]
        each = 2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0) + (1 if groups else 0)
        return {"bytes": t * (h * each + 4 * groups) + 4 * h, "flops": t * h * 8}
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    es = 2 if case["kind"] == "bf16" else 1
    n, kv = lengths(case)
    if case["op"] == "evict":
        out = [k for k in kv if k > case["limit"]]
        return {"bytes": 8 * len(kv) + hk * (4 * sum(out) + len(out) * case["budget"] * (4 * d * es + 8)), "flops": hk * sum(out)}
    if case["op"] == "usage":
        pairs = sum(a * (k - a) + a * (a + 1) // 2 for a, k in zip(n, kv))
        known = sum(k - a for a, k in zip(n, kv)) if case["prev"] else 0
        return {"bytes": sum(n) * hq * (d * 2 + 4) + hk * (sum(kv) * (d * es + 4) + known * 4), "flops": pairs * hq * d * 2}
    tokens = pairs = 0
    for a, k in zip(n, kv):
        low = first_seen(case, a, k)
        tokens += k - low + min(low, case["sinks"])
        for i in range(k - a, k):  # the token at position i
            inside = min(i + 1, case["window"])
            pairs += inside + min(i + 1 - inside, case["sinks"])
    return {"bytes": sum(n) * hq * (d * 4 + 4) + tokens * hk * d * 2 * es, "flops": pairs * hq * d * 4}


def cache(case, pages, g):
    """Keys and values [pages, 2, kv heads, page, dim], and the scales of an 8-bit cache."""
    shape = (pages, 2, case["kv_heads"], case["page"], case["dim"])
    kv = torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=g)
    if case["kind"] == "bf16":
        return kv, None, None
    scales = [torch.empty(case["kv_heads"], device="cuda").uniform_(0.01, 0.03, generator=g) for _ in range(2)]
    kv = (kv.float() / torch.stack(scales)[None, :, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return kv, scales[0], scales[1]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "norm":
        shape = (case["tokens"], case["hidden"])
        # hidden channels of very different sizes, as a residual stream has them
        spread = torch.randn(case["hidden"], device="cuda", generator=g).exp()
        return {"case": case, "x": torch.randn(shape, device="cuda", generator=g).bfloat16(),
                "residual": torch.randn(shape, device="cuda", generator=g).mul_(spread).bfloat16() if case["residual"] else None,
                "weight": torch.empty(case["hidden"], device="cuda").uniform_(0.5, 1.5, generator=g)}
    page, seqs = case["page"], case["seqs"]
    n, kvl = lengths(case)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    used = []  # the pages that each sequence has: all, or those of its sinks and its window
    for a, k in zip(n, kvl):
        every = list(range(-(-k // page)))
        if case["op"] == "window":
            low = first_seen(case, a, k)
            every = [p for p in every if p * page < case["sinks"] or (p + 1) * page > low]
        used.append(every)
    new = -(-case["budget"] // page) if case["op"] == "evict" else 0
    pages = sum(len(u) for u in used) + seqs * new + 5
    kv, ks, vs = cache(case, pages, g)
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((seqs, -(-max(kvl) // page)), -1, dtype=torch.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, u] = torch.arange(at, at + len(u), dtype=torch.int32)
        at += len(u)
    table = torch.where(table.cuda() >= 0, order[table.clamp(min=0).cuda().long()], -1).contiguous()
    total = sum(n)
    s = {"case": case, "kv": kv, "ks": ks, "vs": vs, "table": table, "kv_lens": torch.tensor(kvl, **i32),
         "total": total, "max_q": max(n), "scale": case["dim"] ** -0.5}
    tokens = table.shape[1] * page

    def weights():  # what attention leaves behind: a few tokens with most of it, some with nothing at all
        w = torch.randn((seqs, case["kv_heads"], tokens), device="cuda", generator=g).mul_(2).exp_()
        return w * (torch.rand(w.shape, device="cuda", generator=g) > 0.05)

    if case["op"] == "evict":
        s |= {"usage": weights(), "new_usage": torch.zeros((seqs, case["kv_heads"], tokens), device="cuda"),
              "new_table": order[at:at + seqs * new].view(seqs, new).contiguous(), "new_lens": torch.zeros(seqs, **i32),
              "kept": torch.zeros((seqs, case["kv_heads"], case["budget"]), **i32)}
        return s
    s |= {"q": torch.randn((total, case["q_heads"], case["dim"]), device="cuda", dtype=torch.bfloat16, generator=g),
          "cu_q": torch.tensor([0] + n).cumsum(0).to(**i32)}
    if case["op"] == "usage":
        # the attention's own statistics, about what random queries and keys give
        seen = torch.cat([torch.arange(k - a, k, device="cuda") + 1.0 for a, k in zip(n, kvl)])
        noise = torch.randn((total, case["q_heads"]), device="cuda", generator=g)
        s |= {"lse": (seen.log()[:, None] + 0.5 + 0.1 * noise).contiguous(), "prev": weights() if case["prev"] else None,
              "usage": torch.zeros((seqs, case["kv_heads"], tokens), device="cuda")}
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"window": window_own, "usage": usage_own, "evict": evict_own, "norm": norm_own}[op](state)
    return {"window": window_plain, "usage": usage_plain, "evict": evict_plain, "norm": norm_plain}[op](state)


# ------------------------------------------------------------------------------------------- the library's calls
def window_own(s):
    import shared_routed_expert_amd as srmoe
    c, kv, q = s["case"], s["kv"], s["q"]
    if "out" not in s:
        s["out"] = torch.empty_like(q)
        s["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        s["ws_bytes"] = srmoe.moe_attention_workspace_bytes(c["seqs"], s["total"], s["max_q"], c["q_heads"], c["kv_heads"],
                                                            c["dim"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    srmoe.moe_window_attention(q, q.stride(0), kv[:, 0], kv[:, 1], srmoe.KV_BF16 if c["kind"] == "bf16" else srmoe.KV_E4M3,
                               s["ks"], s["vs"], kv.shape[0], c["page"], kv.stride(0), s["table"], s["table"].shape[1],
                               s["cu_q"], s["kv_lens"], c["window"], c["sinks"], c["seqs"], s["total"], s["max_q"],
                               c["q_heads"], c["kv_heads"], c["dim"], s["scale"], c["cap"], s["out"], s["lse"], s["ws"],
                               s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def usage_own(s):
    import shared_routed_expert_amd as srmoe
    c, kv, q = s["case"], s["kv"], s["q"]
    if "ws" not in s:
        s["ws_bytes"] = srmoe.moe_kv_usage_workspace_bytes(c["seqs"], s["total"], s["max_q"], c["q_heads"], c["kv_heads"],
                                                           c["dim"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    srmoe.moe_kv_usage(q, q.stride(0), kv[:, 0], srmoe.KV_BF16 if c["kind"] == "bf16" else srmoe.KV_E4M3, s["ks"],
                       kv.shape[0], c["page"], kv.stride(0), s["table"], s["table"].shape[1], s["cu_q"], s["kv_lens"], None,
                       s["lse"], c["seqs"], s["total"], s["max_q"], c["q_heads"], c["kv_heads"], c["dim"], s["scale"],
                       c["cap"], s["prev"], c["decay"], s["usage"], None, c["seqs"], s["ws"], s["ws_bytes"])
    return s["usage"]


def evict_own(s):
    import shared_routed_expert_amd as srmoe
    c, kv = s["case"], s["kv"]
    srmoe.moe_kv_evict(kv[:, 0], kv[:, 1], srmoe.KV_BF16 if c["kind"] == "bf16" else srmoe.KV_E4M3, kv.shape[0], c["page"],
                       kv.stride(0), s["table"], s["table"].shape[1], s["kv_lens"], s["usage"], s["new_usage"], None,
                       c["seqs"], c["seqs"], c["kv_heads"], c["dim"], c["limit"], c["budget"], c["sinks"], c["recent"],
                       s["new_table"], s["new_table"].shape[1], s["new_lens"], s["kept"])
    return {"kv": kv, "usage": s["new_usage"], "lens": s["new_lens"], "kept": s["kept"]}


def norm_own(s):
    import shared_routed_expert_amd as srmoe
    c, x = s["case"], s["x"]
    t, h = x.shape
    if "made" not in s:
        s["made"] = True
        s["h"] = torch.empty_like(x) if c["residual"] else None
        s["y"] = torch.empty_like(x) if c["bf16"] else None
        groups = {"none": 0, "row": 1, "block": h // 128}[c["scales"]]
        s["xq"] = torch.empty((t, h), dtype=torch.float8_e4m3fn, device="cuda") if groups else None
        s["sx"] = torch.empty((t, groups), device="cuda") if groups else None
    srmoe.moe_add_rms_norm(x, x.stride(0), s["residual"], s["h"], s["weight"], EPS, t, h,
                           srmoe.SCALE_BLOCK128 if c["scales"] == "block" else srmoe.SCALE_PER_CHANNEL, s["y"], s["xq"],
                           s["sx"])
    return {k: s[k] for k in ("h", "y", "xq", "sx") if s[k] is not None}


# ------------------------------------------------------------------------------------------------- the plain forms
def cached(s, which, index, inside):
    """Float32 keys (which = 0) or values (1) of the tokens `index` [seqs, m] of each sequence, [seqs, kv heads, m, dim]; zeros
    where `inside` is false."""
    c, kv = s["case"], s["kv"]
    index = torch.where(inside, index, 0)
    page = torch.where(inside, s["table"].long().gather(1, index // c["page"]), 0)
    raw = kv if c["kind"] == "bf16" else kv.view(torch.uint8)
    x = raw[page, which, :, index % c["page"]]  # [seqs, m, kv heads, dim]
    x = x.float() if c["kind"] == "bf16" else x.view(torch.float8_e4m3fn).float()
    scale = s["ks"] if which == 0 else s["vs"]
    if scale is not None:
        x = x * scale[:, None]
    return torch.where(inside[:, :, None, None], x, 0.0).transpose(1, 2).contiguous()


def padded(s):
    """Each sequence's tokens side by side: rows [seqs, most] of q, which are real, and the heads
    [seqs, kv heads, most * group, dim] in float32."""
    c = s["case"]
    hk, group, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["dim"]
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device="cuda")
    real = i < n[:, None]
    row = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"].float()[row].view(c["seqs"], s["max_q"], hk, group, d).permute(0, 2, 1, 3, 4)
    return n, i, real, row, q.reshape(c["seqs"], hk, s["max_q"] * group, d)


def scores(s, q, k):
    c = s["case"]
    z = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    if c["cap"]:
        z = z.div_(c["cap"]).tanh_().mul_(c["cap"])
    return z


def window_plain(s):
    c = s["case"]
    seqs, most, hk = c["seqs"], s["max_q"], c["kv_heads"]
    group, d = c["q_heads"] // hk, c["dim"]
    n, i, real, row, q = padded(s)
    lens = s["kv_lens"].long()
    ctx = lens - n
    # the sinks, then everything from the first token's window on
    low = (ctx + 1 - c["window"]).clamp(min=0)
    reach = s["total"] if seqs == 1 else most
    span = min(s["table"].shape[1] * c["page"], c["window"] - 1 + reach)
    j = torch.cat([torch.arange(c["sinks"], device="cuda").expand(seqs, -1), low[:, None] + torch.arange(span, device="cuda")], 1)
    first = torch.arange(j.shape[1], device="cuda") < c["sinks"]
    inside = (j < lens[:, None]) & torch.where(first, True, j >= c["sinks"])
    pos = ctx[:, None] + i
    see = (j[:, None] <= pos[:, :, None]) & ((j[:, None] > pos[:, :, None] - c["window"]) | (j < c["sinks"])[:, None])
    see = see & inside[:, None] & real[:, :, None]
    needed = inside & ((j < c["sinks"]) | (j >= low[:, None]))
    z = scores(s, q, cached(s, 0, j, needed)).view(seqs, hk, most, group, -1).masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(seqs, hk, most * group, -1) @ cached(s, 1, j, needed)).view(seqs, hk, most, group, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 2, 1, 3, 4).reshape(seqs, most, c["q_heads"], d)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(seqs, most, c["q_heads"])[real]
    return {"out": out.bfloat16(), "lse": lse}


def usage_plain(s):
    c = s["case"]
    seqs, most, hk = c["seqs"], s["max_q"], c["kv_heads"]
    group = c["q_heads"] // hk
    n, i, real, row, q = padded(s)
    lens = s["kv_lens"].long()
    tokens = s["table"].shape[1] * c["page"]
    j = torch.arange(tokens, device="cuda").expand(seqs, -1)
    inside = j < lens[:, None]
    z = scores(s, q, cached(s, 0, j, inside)).view(seqs, hk, most, group, tokens)
    lse = s["lse"][row].view(seqs, most, hk, group).permute(0, 2, 1, 3)
    see = (j[:, None] <= (lens - n)[:, None, None] + i[:, None]) & inside[:, None] & real[:, :, None]
    new = z.sub_(lse[..., None]).exp_().masked_fill_(~see[:, None, :, None, :], 0.0).sum((2, 3))
    if s["prev"] is not None:
        new = new + torch.where((j < (lens - n)[:, None])[:, None], c["decay"] * s["prev"], 0.0)
    return torch.where(inside[:, None], new, s["usage"])


def evict_plain(s):
    c, kv = s["case"], s["kv"]
    seqs, hk, page, budget = c["seqs"], c["kv_heads"], c["page"], c["budget"]
    lens = s["kv_lens"].long()
    out = lens > c["limit"]
    w = s["usage"]
    j = torch.arange(w.shape[2], device="cuda")
    always = (j < c["sinks"]) | ((j >= lens[:, None] - c["recent"]) & (j < lens[:, None]))
    w = torch.where(always[:, None], math.inf, w)
    w = torch.where((j < lens[:, None])[:, None], w, -math.inf)
    w, order = w.sort(dim=-1, descending=True, stable=True)
    # (a table that holds no sequence over the limit may be narrower than the budget)
    keep = order[..., :budget].sort(dim=-1).values
    which = out.nonzero()[:, 0]
    keep = keep[which]
    if which.numel():
        h = torch.arange(hk, device="cuda")[None, :, None]
        to = torch.arange(budget, device="cuda")
        source = s["table"].long()[which[:, None, None], keep // page]
        target = s["new_table"].long()[which][:, to // page][:, None]
        raw = kv if c["kind"] == "bf16" else kv.view(torch.uint8)
        moved = raw[source, :, h, keep % page]
        raw[target.expand(-1, hk, -1), :, h, (to % page).expand(len(which), hk, -1)] = moved
        s["kept"][which] = keep.int()
        s["new_usage"][which, :, :budget] = s["usage"][which].gather(-1, keep)
    s["new_lens"].copy_(torch.where(out, budget, lens))
    return {"kv": kv, "usage": s["new_usage"], "lens": s["new_lens"], "kept": s["kept"]}


def norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    r = {"h": h.bfloat16()} if c["residual"] else {}
    if c["bf16"]:
        r["y"] = y.bfloat16()
    if c["scales"] != "none":
        parts = y.view(y.shape[0], -1, 128 if c["scales"] == "block" else y.shape[1])
        most = parts.abs().amax(-1)
        sx = torch.where(most > 0, most / 448, 1.0)
        r |= {"xq": (parts / sx[..., None]).clamp(-448, 448).view_as(y).to(torch.float8_e4m3fn), "sx": sx}
    return r


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"window": window_exact, "usage": usage_exact, "evict": evict_exact, "norm": norm_exact}[case["op"]](s)


def tokens_of(s, which, b, h, index):
    """The keys or values of tokens `index` of sequence b and kv head h, in float64."""
    page = s["case"]["page"]
    x = s["kv"][s["table"][b].long()[index // page], which, h, index % page].double()
    scale = s["ks"] if which == 0 else s["vs"]
    return x if scale is None else x * scale[h].double()


def logits(s, b, qh, at, n, keys):
    c = s["case"]
    z = s["q"][at:at + n, qh].double() @ keys.T * s["scale"]
    return c["cap"] * torch.tanh(z / c["cap"]) if c["cap"] else z


def window_exact(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros((s["total"], c["q_heads"], c["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], c["q_heads"]), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(*lengths(c))):
        low = first_seen(c, n, kv)
        index = torch.arange(kv, device="cuda")
        index = index[(index >= low) | (index < c["sinks"])]
        p = kv - n + torch.arange(n, device="cuda")[:, None]
        hidden = (index > p) | ((p - index >= c["window"]) & (index >= c["sinks"]))
        for h in range(c["kv_heads"]):
            k, v = (tokens_of(s, w, b, h, index) for w in (0, 1))
            for qh in range(h * group, (h + 1) * group):
                z = logits(s, b, qh, at, n, k)
                z[hidden] = -math.inf
                total = torch.logsumexp(z, 1)
                lse[at:at + n, qh] = total
                out[at:at + n, qh] = torch.exp(z - total[:, None]) @ v
        at += n
    return {"out": out, "lse": lse}


def usage_exact(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    result = s["usage"].double()
    at = 0
    for b, (n, kv) in enumerate(zip(*lengths(c))):
        index = torch.arange(kv, device="cuda")
        for h in range(c["kv_heads"]):
            k = tokens_of(s, 0, b, h, index)
            got = torch.zeros(kv, dtype=torch.float64, device="cuda")
            if s["prev"] is not None:
                got[:kv - n] = s["prev"][b, h, :kv - n].double() * c["decay"]
            for qh in range(h * group, (h + 1) * group):
                p = torch.exp(logits(s, b, qh, at, n, k) - s["lse"][at:at + n, qh, None].double())
                got += torch.tril(p, kv - n).sum(0)
            result[b, h, :kv] = got
        at += n
    return result


def evict_exact(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    kv, used = s["kv"].double(), s["new_usage"].double()
    lens, kept = s["kv_lens"].clone(), s["kept"].clone()
    for b, n in enumerate(lengths(c)[1]):
        if n <= c["limit"]:
            continue
        lens[b] = budget
        start, end = min(c["sinks"], n), max(c["sinks"], n - c["recent"])
        for h in range(c["kv_heads"]):
            middle = s["usage"][b, h, start:end].double()
            best = torch.argsort(-middle, stable=True)[:budget - start - (n - end)] + start
            chosen = torch.zeros(n, dtype=torch.bool, device="cuda")
            chosen[:start] = True
            chosen[end:] = True
            chosen[best] = True
            index = chosen.nonzero()[:, 0]
            kept[b, h] = index.int()
            used[b, h, :budget] = s["usage"][b, h, index].double()
            to = torch.arange(budget, device="cuda")
            for w in (0, 1):
                kv[s["new_table"][b].long()[to // page], w, h, to % page] = \
                    s["kv"][s["table"][b].long()[index // page], w, h, index % page].double()
    return {"kv": kv, "usage": used, "lens": lens, "kept": kept}


def norm_exact(s):
    c = s["case"]
    h = s["x"].double()
    if c["residual"]:
        h = h + s["residual"].double()
    y = h / ((h * h).sum(1, keepdim=True) / c["hidden"] + EPS).sqrt() * s["weight"].double()
    r = {"h": h} if c["residual"] else {}
    if c["bf16"]:
        r["y"] = y
    if c["scales"] != "none":
        wide = 128 if c["scales"] == "block" else c["hidden"]
        groups = c["hidden"] // wide
        sx = torch.stack([y[:, g * wide:(g + 1) * wide].abs().max(1).values for g in range(groups)], 1) / 448
        r |= {"xq": y / sx.repeat_interleave(wide, 1), "sx": sx}
    return r
