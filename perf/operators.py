"""The paged key/value cache and the attention that reads it: what is measured, in plain torch and through the library.

Three operators: `append` (per-head norm and rotation of q and k, keys and values into the paged cache), `tree`
(attention of a few drafted tokens per sequence over the cache; one token per sequence is ordinary decoding) and
`prefill` (a chunk's tokens over the cache, causal, with an optional prefix seen by every token).

The cache is [pages, 2, kv heads, page size, head dim] (keys, values), bf16 or e4m3 with a float32 scale per kv head;
its pages are handed out in random order. Sizes: one GPU's share of GLM4-MoE attention under TP8 (12 query heads on 1
kv head, head dim 128, half of it rotated), the unsharded heads (96 on 8), and generic ones.
"""
import math
import random

import torch

own = False

THETA, EPS, MAX_POS = 1e6, 1e-5, 131072


def listed():
    return [
        # one token of one short sequence: launch latency
        tree("decode one short sequence", 1, 1, 777, "bf16", ragged=False),
        # a serving batch, one token per sequence, ordinary lengths
        tree("decode batch 64", 64, 1, 8192, "bf16"),
        # few long sequences in an 8-bit cache: one sequence's keys spread over the whole card
        tree("decode 3 long e4m3", 3, 1, 131072, "e4m3", ragged=False),
        # a large batch of long sequences on the unsharded heads
        tree("decode unsharded 24", 24, 1, 16384, "bf16", q_heads=96, kv_heads=8, page=64),
        # drafted trees of up to 16 tokens
        tree("trees of 16 e4m3", 48, 16, 6000, "e4m3", page=32),
        # large trees of up to 64 tokens, capped scores
        tree("trees of 64", 8, 64, 4099, "bf16", cap=30.0),
        # one prompt in one chunk
        prefill("prefill 4096", 1, 4096, 0, "bf16", ragged=False),
        # a 16384-token chunk made of ragged parts of long prompts, 8-bit cache
        prefill("prefill 16k e4m3", 4, 4096, 16384, "e4m3", page=64, ragged=False),
        # many short ragged prompts with a prefix that every token sees, small heads
        prefill("prefill ragged prefix", 23, 700, 300, "bf16", q_heads=8, kv_heads=2, dim=64, prefix=True, page=16),
        # the cache writes of the same steps: a decode batch, a 16384-token chunk, the unsharded heads
        append("append decode 64", 64, "bf16"),
        append("append 16k e4m3", 16384, "e4m3", page=64),
        append("append unsharded 5000", 5000, "bf16", q_heads=96, kv_heads=8),
    ]


def tree(name, seqs, nodes, kv, kind, q_heads=12, kv_heads=1, dim=128, page=16, cap=0.0, ragged=True, lens=1):
    return {"name": name, "op": "tree", "seqs": seqs, "nodes": nodes, "kv": kv, "kind": kind, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cap": cap, "ragged": ragged, "lens": lens}


def prefill(name, seqs, chunk, context, kind, q_heads=12, kv_heads=1, dim=128, page=16, cap=0.0, prefix=False,
            ragged=True, lens=1):
    return {"name": name, "op": "prefill", "seqs": seqs, "nodes": chunk, "kv": context + chunk, "kind": kind,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "cap": cap, "prefix": prefix,
            "ragged": ragged, "lens": lens}


def append(name, tokens, kind, q_heads=12, kv_heads=1, dim=128, page=16, neox=True, lens=1):
    return {"name": name, "op": "append", "tokens": tokens, "kind": kind, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "rotary": dim // 2, "page": page, "neox": neox, "lens": lens}


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "tree", "tree", "prefill"])
    q_heads, kv_heads, dim = rng.choice([(12, 1, 128), (12, 1, 128), (96, 8, 128), (8, 2, 64), (16, 4, 128), (7, 1, 64),
                                         (8, 1, 256)])
    more = {"q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128]),
            "kind": rng.choice(["bf16", "e4m3"]), "lens": rng.randrange(1 << 30)}
    if op == "append":
        c = append("", size(1, max(64, 16384 * 14 // (q_heads + 2 * kv_heads))), neox=rng.random() < 0.7, **more)
    elif op == "tree":
        nodes = rng.choice([1, 1, size(2, 64)])
        seqs = size(1, 96)
        kv = size(64, 131072)
        seqs = max(1, min(seqs, (1 << 20) // (kv * kv_heads), (1 << 25) // (kv * nodes * q_heads) or 1))
        c = tree("", seqs, nodes, kv, cap=rng.choice([0.0, 0.0, 30.0]), ragged=rng.random() < 0.7, **more)
    else:
        chunk = size(65, 8192)
        context = rng.choice([0, size(16, 16384)])
        seqs = max(1, min(size(1, 16), int(1.6e9) // ((context + chunk) * chunk * q_heads * max(1, dim // 128))))
        while seqs == 1 and (context + chunk) * chunk * q_heads * max(1, dim // 128) > 1.6e9:
            chunk, context = chunk // 2 + 1, context // 2
        c = prefill("", seqs, chunk, context, cap=rng.choice([0.0, 0.0, 30.0]), prefix=rng.random() < 0.3,
                    ragged=rng.random() < 0.6, **more)
    del c["name"]
    return c


def lengths(case):
    """Tokens of each sequence in this call, its cached tokens after them, and its prefix."""
    r = random.Random(case["lens"])
    n, kv, prefix = [], [], []
    for _ in range(case["seqs"]):
        t = r.randint(max(1, case["nodes"] // 4), case["nodes"]) if case["ragged"] else case["nodes"]
        c = case["kv"] - case["nodes"]
        c = r.randint(c // 8, c) if case["ragged"] else c
        n.append(t)
        kv.append(c + t)
        prefix.append(r.randint(0, c + t) if case.get("prefix") else 0)
    return n, kv, prefix


def visible(case):
    """Query/key pairs of one query head that the masks leave, about (a drafted tree: half of its own square)."""
    total = 0
    for n, kv, pre in zip(*lengths(case)):
        first = kv - n + 1  # keys that the first token sees
        full = max(0, min(n, pre - first))  # tokens that see the prefix and nothing more
        total += full * pre + (n - full) * (first + full + kv) // 2
    return total


def work(case):
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    size = 2 if case["kind"] == "bf16" else 1
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": t * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * d * size + case["rotary"] * 4 + 8),
                "flops": t * (hq + hk) * d * 8}
    n, kv, _ = lengths(case)
    return {"bytes": sum(n) * hq * (d * 4 + 4) + sum(kv) * hk * d * 2 * size, "flops": visible(case) * hq * d * 4}


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
    d, hq, hk, page = case["dim"], case["q_heads"], case["kv_heads"], case["page"]
    if case["op"] == "append":
        t = case["tokens"]
        pages = 2 * (-(-t // page)) + 3
        kv, ks, vs = cache(case, pages, g)
        row = (hq + 2 * hk) * d
        qkv = torch.randn((t, row), device="cuda", generator=g) * torch.randn(row, device="cuda", generator=g).mul(0.5).exp()
        order = torch.randperm(pages, device="cuda", generator=g)
        token = torch.arange(t, device="cuda")
        slots = (order[token // page] * page + token % page).int()
        if t > 8:
            slots[-3:] = -1  # a padded batch: these tokens are not cached
        pos = torch.randint(0, MAX_POS, (t,), device="cuda", generator=g) if t <= 256 else token % MAX_POS
        freq = THETA ** (-torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"])
        angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * freq
        return {"case": case, "qkv": qkv.bfloat16(), "kv": kv, "ks": ks, "vs": vs, "slots": slots, "pos": pos.int(),
                "qw": torch.empty(d, device="cuda").uniform_(0.5, 1.5, generator=g),
                "kw": torch.empty(d, device="cuda").uniform_(0.5, 1.5, generator=g),
                "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float()}
    n, kvl, prefix = lengths(case)
    need = [-(-k // page) for k in kvl]
    pages = sum(need) + 5
    kv, ks, vs = cache(case, pages, g)
    order = torch.randperm(pages, device="cuda", generator=g).int()
    width = -(-max(kvl) // page)
    start = torch.tensor([0] + need[:-1]).cumsum(0)[:, None]
    at = torch.arange(width)[None]
    inside = at < torch.tensor(need)[:, None]
    table = torch.where(inside.cuda(), order[torch.where(inside, start + at, 0).cuda()], 0).int().contiguous()
    total = sum(n)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"case": case, "q": torch.randn((total, hq, d), device="cuda", dtype=torch.bfloat16, generator=g), "kv": kv,
         "ks": ks, "vs": vs, "table": table, "cu_q": torch.tensor([0] + n).cumsum(0).to(**i32),
         "kv_lens": torch.tensor(kvl, **i32), "prefix": torch.tensor(prefix, **i32) if case.get("prefix") else None,
         "max_q": max(n), "total": total, "scale": d ** -0.5, "mask": None}
    if case["op"] == "tree" and case["nodes"] > 1:
        r = random.Random(seed)
        masks = []
        for k in n:
            own_path = []
            for i in range(k):  # a token's parent is one of those before it, or the context
                parent = r.randrange(-1, i)
                own_path.append((own_path[parent] if parent >= 0 else 0) | 1 << i)
            masks += [m - (1 << 64) if m >> 63 else m for m in own_path]
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return s


def run(state):
    return (append_own if own else append_plain)(state) if state["case"]["op"] == "append" else \
        (attention_own if own else attention_plain)(state)


# ------------------------------------------------------------------------------------------- the library's calls
def append_own(s):
    import shared_routed_expert_amd as srmoe
    c, kv = s["case"], s["kv"]
    if "q_out" not in s:
        s["q_out"] = torch.empty((c["tokens"], c["q_heads"], c["dim"]), dtype=torch.bfloat16, device="cuda")
    k, v = kv[:, 0], kv[:, 1]
    srmoe.moe_kv_append(s["qkv"], s["qkv"].stride(0), c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rotary"],
                        c["neox"], s["qw"], s["kw"], EPS, s["pos"], s["cos_sin"], MAX_POS, s["slots"], s["q_out"], k, v,
                        srmoe.KV_BF16 if c["kind"] == "bf16" else srmoe.KV_E4M3, s["ks"], s["vs"], kv.shape[0], c["page"],
                        kv.stride(0))
    return {"q": s["q_out"], "kv": kv}


def attention_own(s):
    import shared_routed_expert_amd as srmoe
    c, kv, q = s["case"], s["kv"], s["q"]
    if "out" not in s:
        s["out"] = torch.empty_like(q)
        s["lse"] = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        s["ws_bytes"] = srmoe.moe_attention_workspace_bytes(c["seqs"], s["total"], s["max_q"], c["q_heads"], c["kv_heads"],
                                                            c["dim"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    call = srmoe.moe_tree_attention if c["op"] == "tree" else srmoe.moe_prefill_attention
    call(q, q.stride(0), kv[:, 0], kv[:, 1], srmoe.KV_BF16 if c["kind"] == "bf16" else srmoe.KV_E4M3, s["ks"], s["vs"],
         kv.shape[0], c["page"], kv.stride(0), s["table"], s["table"].shape[1], s["cu_q"], s["kv_lens"],
         s["mask"] if c["op"] == "tree" else s["prefix"], c["seqs"], s["total"], s["max_q"], c["q_heads"], c["kv_heads"],
         c["dim"], s["scale"], c["cap"], s["out"], s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------- the plain forms
def append_plain(s):
    c, kv = s["case"], s["kv"]
    d, hq, hk, rd = c["dim"], c["q_heads"], c["kv_heads"], c["rotary"]
    x = s["qkv"].float().view(-1, hq + 2 * hk, d)
    qk, v = x[:, :hq + hk], x[:, hq + hk:]
    w = torch.cat([s["qw"].expand(hq, d), s["kw"].expand(hk, d)])
    y = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS) * w
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, None, :rd // 2], cs[:, None, rd // 2:]
    if c["neox"]:
        a, b = y[..., :rd // 2], y[..., rd // 2:rd]
        rotated = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rd:2], y[..., 1:rd:2]
        rotated = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    y = torch.cat([rotated, y[..., rd:]], -1)
    k = y[:, hq:]
    slots = s["slots"].long()
    kept = (slots >= 0).nonzero()[:, 0]
    page, at = slots[kept] // c["page"], slots[kept] % c["page"]
    new = torch.stack([k, v], 1)[kept]  # [tokens, 2, kv heads, dim]
    if c["kind"] == "bf16":
        kv[page, :, :, at] = new.bfloat16()
    else:
        scales = torch.stack([s["ks"], s["vs"]])[None, :, :, None]
        kv.view(torch.uint8)[page, :, :, at] = (new / scales).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"q": y[:, :hq].bfloat16(), "kv": kv}


def attention_plain(s):
    c, kv = s["case"], s["kv"]
    d, hq, hk = c["dim"], c["q_heads"], c["kv_heads"]
    seqs, most, group = c["seqs"], s["max_q"], hq // hk
    table = s["table"].long()
    keys = table.shape[1] * c["page"]
    cu = s["cu_q"].long()
    n, lens = cu[1:] - cu[:-1], s["kv_lens"].long()
    # the sequences' keys and values side by side: [2, seqs, kv heads, keys, dim]
    if c["kind"] == "bf16":
        kv = kv[table].float()
    else:
        kv = kv.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, seqs, hk, keys, d)
    if s["ks"] is not None:
        kv = kv * torch.stack([s["ks"], s["vs"]])[:, None, :, None, None]
    j = torch.arange(keys, device="cuda")
    kv = torch.where((j < lens[:, None])[None, :, None, :, None], kv, 0.0)
    # the tokens of each sequence, padded: [seqs, most]
    i = torch.arange(most, device="cuda")
    real = i < n[:, None]
    row = torch.where(real, cu[:-1, None] + i, 0)
    q = s["q"].float()[row].view(seqs, most, hk, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, most * group, d)
    score = (q @ kv[0].transpose(-1, -2)).mul_(s["scale"])
    if c["cap"]:
        score = score.div_(c["cap"]).tanh_().mul_(c["cap"])
    first = lens - n  # position of a sequence's first token
    pos = first[:, None] + i
    if s["mask"] is not None:
        bit = (j - first[:, None])[:, None, :]
        seen = (s["mask"][row][:, :, None] >> bit.clamp(0, 63)) & 1
        see = torch.where(bit < 0, True, (bit < most) & (seen == 1))
    else:
        see = j <= pos[:, :, None]
        if s["prefix"] is not None:
            see = see | (j < s["prefix"][:, None, None])
    see = see & (j < lens[:, None])[:, None, :] & real[:, :, None]
    score = score.view(seqs, hk, most, group, keys).masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(seqs, hk, most * group, keys) @ kv[1]).view(seqs, hk, most, group, d)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 2, 1, 3, 4).reshape(seqs, most, hq, d)[real]
    lse = lse.permute(0, 2, 1, 3).reshape(seqs, most, hq)[real]
    return {"out": out.bfloat16(), "lse": lse}


# ------------------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return append_exact(s) if case["op"] == "append" else attention_exact(s)


def append_exact(s):
    c = s["case"]
    d, hq, hk, rd = c["dim"], c["q_heads"], c["kv_heads"], c["rotary"]
    half = rd // 2
    heads = s["qkv"].double().view(c["tokens"], hq + 2 * hk, d)
    turn = torch.zeros((c["tokens"], half), dtype=torch.complex128, device="cuda")
    for i in range(half):
        angle = s["pos"].double() * THETA ** (-2.0 * i / rd)
        turn[:, i] = torch.polar(torch.ones_like(angle), angle)

    def normed(x, w):
        return x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()

    def rotated(x):
        x = x.clone()
        even, odd = (slice(0, half), slice(half, rd)) if c["neox"] else (slice(0, rd, 2), slice(1, rd, 2))
        z = torch.complex(x[..., even], x[..., odd]) * turn[:, None]
        x[..., even], x[..., odd] = z.real, z.imag
        return x

    q = rotated(normed(heads[:, :hq], s["qw"]))
    k = rotated(normed(heads[:, hq:hq + hk], s["kw"]))
    kv = s["kv"].double()
    for which, x, scale in ((0, k, s["ks"]), (1, heads[:, hq + hk:], s["vs"])):
        if scale is not None:
            x = (x / scale.double()[None, :, None]).clamp(-448, 448)
        flat = kv[:, which].transpose(1, 2).reshape(-1, hk, d)  # [slots, kv heads, dim]
        put = s["slots"] >= 0
        flat[s["slots"][put].long()] = x[put]
        kv[:, which] = flat.view(-1, c["page"], hk, d).transpose(1, 2)
    return {"q": q, "kv": kv}


def attention_exact(s):
    c = s["case"]
    d, hq, hk, page = c["dim"], c["q_heads"], c["kv_heads"], c["page"]
    group = hq // hk
    ns, lens, prefix = lengths(c)
    out = torch.zeros((s["total"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], hq), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, kv, pre) in enumerate(zip(ns, lens, prefix)):
        pages = s["table"][b, :-(-kv // page)].long()
        token = torch.arange(kv, device="cuda")
        node = torch.arange(n, device="cuda")
        if s["mask"] is not None:
            path = s["mask"][at:at + n]
            hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
            for t in range(n):
                hidden[:, kv - n + t] = path.bitwise_right_shift(t).bitwise_and(1) == 0
        else:
            hidden = (token[None] > (kv - n + node)[:, None]) & (token[None] >= pre)
        for h in range(hk):
            kh, vh = (s["kv"][pages, w, h].double().reshape(-1, d)[:kv] for w in (0, 1))
            if s["ks"] is not None:
                kh, vh = kh * s["ks"][h].double(), vh * s["vs"][h].double()
            for qh in range(h * group, (h + 1) * group):
                z = s["q"][at:at + n, qh].double() @ kh.T * s["scale"]
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                z[hidden] = -math.inf
                norm = torch.logsumexp(z, 1)
                lse[at:at + n, qh] = norm
                out[at:at + n, qh] = torch.exp(z - norm[:, None]) @ vh
        at += n
    return {"out": out, "lse": lse}
