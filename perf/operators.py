"""The serving step's operators, as they are measured: cases, inputs, the plain
form and the 64-bit result of each.

  append   the new tokens' rows into a paged cache: latent or key norm, rotation
           by position, and the queries' norm and rotation in the same pass
  attend   attention of the new tokens (one or a chunk per sequence) over the
           paged cache, MLA (latent rows) and GQA (K and V planes)
"""

import math

import torch

own = False

LATENT, ROPE = 512, 64          # an MLA row: latent values, then the rotated band
NOPE = 128                      # the unrotated part of a projected MLA query head
EPS = 1e-6


def _mla(name, op, heads, n, q, kv, page):
    return dict(name=name, op=op, kind="mla", heads=heads, n=n, q=q, kv=kv, page=page)


def _gqa(name, op, kv_heads, group, dim, rot, pairing, n, q, kv, page, norm=True, window=0):
    return dict(name=name, op=op, kind="gqa", kv_heads=kv_heads, group=group, dim=dim, rot=rot, pairing=pairing,
                n=n, q=q, kv=kv, page=page, norm=norm, window=window)


def listed():
    return [
        # one user's next token: a single row of a 16-head MLA model, all latency
        _mla("mla_append_token", "append", 16, 1, 1, 4097, 16),
        # a decoding batch of a model with 8 KV heads of 128 and per-head norms
        _gqa("gqa_append_batch", "append", 8, 4, 128, 128, "half", 96, 1, 2048, 16),
        # three prompts of a 128-head MLA model prefilled together
        _mla("mla_append_prompts", "append", 128, 3, 8192, 8192, 64),
        # prompts of a model with odd head counts, a partial band, tiny pages and no norms
        _gqa("gqa_append_prompts_odd", "append", 3, 5, 96, 32, "interleaved", 5, 5003, 6007, 4, norm=False),
        # one user's next token over a short context: the smallest attention
        _mla("mla_attend_token", "attend", 16, 1, 1, 1531, 16),
        # a decoding batch with long contexts: bound by reading the cache
        _mla("mla_attend_batch", "attend", 16, 64, 1, 32768, 16),
        # two speculated tokens each on 128 heads: reading and arithmetic in balance
        _mla("mla_attend_draft", "attend", 128, 32, 2, 8192, 64),
        # prompt chunks over what is cached already: bound by arithmetic
        _mla("mla_attend_chunk", "attend", 16, 2, 2048, 16384, 16),
        # one user's next token over a very long context: one sequence has to fill the chip
        _gqa("gqa_attend_token", "attend", 8, 4, 128, 128, "half", 1, 1, 131072, 16),
        # a decoding batch of ordinary, ragged contexts
        _gqa("gqa_attend_batch", "attend", 8, 4, 128, 128, "half", 128, 1, 8192, 16),
        # a prompt chunk deep in a long prompt
        _gqa("gqa_attend_chunk", "attend", 8, 4, 128, 128, "half", 1, 4096, 32768, 16),
        # a sliding window over small ragged chunks, odd heads, a head size between the powers of two
        _gqa("gqa_attend_window_odd", "attend", 3, 5, 96, 32, "interleaved", 7, 333, 5501, 4, window=1000),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend"])
    shape = rng.choice(["token", "batch", "chunk"])
    n = {"token": 1, "batch": log(2, 128), "chunk": log(1, 6)}[shape]
    q = {"token": 1, "batch": rng.choice([1, 1, 1, 2, 3]), "chunk": log(16, 6000 if op == "append" else 3000)}[shape]
    kv = max(q, log(1, 131072 if shape == "token" else 16384))
    page = rng.choice([1, 4, 16, 64, 256])
    if rng.random() < 0.5:
        c = _mla("", op, rng.choice([8, 16, 32, 64, 128, 20]), n, q, kv, page)
        heads = c["heads"]
    else:
        dim, rot = rng.choice([(64, 64), (128, 128), (128, 64), (96, 32), (80, 16), (256, 64), (32, 32)])
        c = _gqa("", op, rng.choice([1, 2, 4, 8, 3]), rng.choice([1, 4, 5, 8]), dim, rot,
                 rng.choice(["half", "interleaved"]), n, q, kv, page, norm=rng.random() < 0.5,
                 window=rng.choice([0, 0, log(1, 4096)]) if op == "attend" else 0)
        heads = c["kv_heads"] * c["group"]
    del c["name"]
    # no pass costs more than the largest listed one, nor has more scores or rows
    while (c["n"] * c["q"] * heads * c["kv"] > 1 << 31 if op == "attend" else c["n"] * c["kv"] > 1 << 18) \
            or work(c)["flops"] > 2e12 or work(c)["bytes"] > 2.7e9:
        if c["n"] > 1:
            c["n"] = (c["n"] + 1) // 2
        else:
            c["kv"] = max(c["q"], c["kv"] * 2 // 3)
            c["q"] = c["q"] if c["kv"] > c["q"] else c["q"] * 2 // 3
    return c


def _lengths(c):
    """(new tokens, cached tokens with them) of each sequence: the first is the
    longest, the others are spread over the lower part of the range."""
    counts, kvs = [], []
    for i in range(c["n"]):
        q = c["q"] - (i * 131) % (c["q"] // 2 + 1) if c["q"] > 3 else c["q"]
        low = max(q, c["kv"] // 4)
        counts.append(q)
        kvs.append(c["kv"] - (i * 7919) % (c["kv"] - low + 1))
    return counts, kvs


def _shape(c):
    """(query heads, rotated width, frequency base, scale)."""
    if c["kind"] == "mla":
        return c["heads"], ROPE, 10000.0, (NOPE + ROPE) ** -0.5
    return c["kv_heads"] * c["group"], c["rot"], 500000.0, c["dim"] ** -0.5


def _angles(c, positions):
    _, rot, base, _ = _shape(c)
    theta = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=positions.device) / rot)
    return positions.double()[:, None] * theta


def prepare(case, seed):
    c, dev = case, torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    counts, kvs = _lengths(c)
    heads, rot, base, scale = _shape(c)
    P, n, T = c["page"], c["n"], sum(counts)
    per = [-(-k // P) for k in kvs]
    total, width = sum(per) + 3, max(per)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    # every sequence's pages lie anywhere in the pool
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    host = order.cpu().numpy()
    table = torch.full((n, width), -1, dtype=torch.int32)
    pages, at = [], 0
    for i, k in enumerate(per):
        pages.append(host[at:at + k])
        table[i, :k] = torch.from_numpy(pages[i])
        at += k
    table = table.to(dev)

    count = torch.tensor(counts, device=dev)
    length = torch.tensor(kvs, device=dev)
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count)
    off = torch.arange(T, device=dev) - torch.repeat_interleave(count.cumsum(0) - count, count)
    row = (length - count)[seq] + off                     # a token's row in its sequence, and its position
    slot = table[seq, row // P].long() * P + row % P      # where it lies in the pool
    s = dict(case=c, scale=scale, table=table, count=count, length=length, seq=seq, off=off, row=row, slot=slot,
             max_q=max(counts), max_kv=max(kvs))
    if c["kind"] == "mla":
        s["cache"] = randn(1, total, P, LATENT + ROPE)
    else:
        s["k_cache"] = randn(1, total, P, c["kv_heads"], c["dim"])
        s["v_cache"] = randn(1, total, P, c["kv_heads"], c["dim"])
    if c["op"] == "append":
        ang = _angles(c, row)
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()   # a model keeps these for all its layers
        if c["kind"] == "mla":
            s["kv"] = randn(T, LATENT + ROPE) * 2.0                 # the rows of one projection
            s["norm"] = 1 + 0.25 * randn(LATENT)
            s["q"] = randn(T, heads, NOPE + ROPE)
            s["q_out"] = torch.zeros(T, heads, LATENT + ROPE, device=dev, dtype=torch.bfloat16)
        else:
            s["qkv"] = randn(T, heads + 2 * c["kv_heads"], c["dim"]) * 2.0
            s["q_out"] = torch.zeros(T, heads, c["dim"], device=dev, dtype=torch.bfloat16)
            s["norm"] = 1 + 0.25 * randn(c["dim"]) if c["norm"] else None
            s["q_norm"] = 1 + 0.25 * randn(c["dim"]) if c["norm"] else None
    else:
        width = LATENT + ROPE if c["kind"] == "mla" else c["dim"]
        s["q"] = randn(T, heads, width)
        s["out"] = torch.zeros(T, heads, LATENT if c["kind"] == "mla" else width, device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.zeros(T, heads, device=dev)
    if own:
        # what a serving loop holds: the pool, its sequences, and the plan of this
        # step, which every layer of the model uses
        from mla_paged_cache_amd import leyline as L
        if c["kind"] == "mla":
            s["pool"] = L.Pool(s["cache"], table, rope_base=base)
        else:
            s["pool"] = L.GqaPool(s["k_cache"], s["v_cache"], table, rotary_dim=rot, rope_base=base,
                                  pairing=L.ROPE_HALF if c["pairing"] == "half" else L.ROPE_INTERLEAVED)
        for i in range(n):
            s["pool"].seq_set_pages(i, pages[i], kvs[i])
        s["step"] = s["pool"].step(heads, max_seqs=n, max_tokens=T)
        s["step"].begin(list(range(n)), counts, grow=False)
    return s


def _turn(x, cos, sin, pairing):
    """Each pair of the last axis turned by its token's angle."""
    h = x.shape[-1] // 2
    if pairing == "half":
        a, b = x[..., :h], x[..., h:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain_append(s):
    c = s["case"]
    if c["kind"] == "mla":
        kv, cos, sin = s["kv"].float(), s["cos"], s["sin"]
        new = torch.cat([_normed(kv[:, :LATENT], s["norm"]), _turn(kv[:, LATENT:], cos, sin, "interleaved")], -1)
        s["cache"].view(-1, LATENT + ROPE).index_copy_(0, s["slot"], new.bfloat16())
        q = _turn(s["q"][..., NOPE:].float(), cos[:, None], sin[:, None], "interleaved")
        s["q_out"][..., LATENT:] = q.bfloat16()
        return s["cache"], s["q_out"][..., LATENT:]
    heads, H, D, rot = c["kv_heads"] * c["group"], c["kv_heads"], c["dim"], c["rot"]
    cos, sin = s["cos"][:, None], s["sin"][:, None]
    q, k = _normed(s["qkv"][:, :heads].float(), s["q_norm"]), _normed(s["qkv"][:, heads:heads + H].float(), s["norm"])
    q = torch.cat([_turn(q[..., :rot], cos, sin, c["pairing"]), q[..., rot:]], -1)
    k = torch.cat([_turn(k[..., :rot], cos, sin, c["pairing"]), k[..., rot:]], -1)
    s["k_cache"].view(-1, H, D).index_copy_(0, s["slot"], k.bfloat16())
    s["v_cache"].view(-1, H, D).index_copy_(0, s["slot"], s["qkv"][:, heads + H:])
    s["q_out"].copy_(q)
    return s["k_cache"], s["v_cache"], s["q_out"]


def _plain_attend(s):
    """Sequences side by side, padded to the longest; masked scores weigh nothing."""
    c, P, dev = s["case"], s["case"]["page"], s["q"].device
    T, heads, width = s["q"].shape
    j = torch.arange(s["max_kv"], device=dev)
    rows = s["table"][:, j // P].clamp(min=0).long() * P + j % P                    # [n][kv]
    i = torch.arange(s["max_q"], device=dev)
    start = s["count"].cumsum(0) - s["count"]
    token = (start[:, None] + i).clamp(max=T - 1)                                   # [n][q]
    at = (s["length"] - s["count"])[:, None] + i                                    # a query's own row
    seen = j <= at[..., None]
    if c.get("window"):
        seen &= j > at[..., None] - c["window"]
    n, nq, nk = seen.shape
    if c["kind"] == "mla":
        k = s["cache"].view(-1, LATENT + ROPE)[rows].float()[:, None]               # [n][1][kv][576]
        v, H = k[..., :LATENT], 1
    else:
        H = c["kv_heads"]
        k = s["k_cache"].view(-1, H, width)[rows].float().transpose(1, 2)
        v = s["v_cache"].view(-1, H, width)[rows].float().transpose(1, 2)
    G = heads // H
    q = s["q"][token].float().view(n, nq, H, G, width).permute(0, 2, 1, 3, 4).reshape(n, H, nq * G, width)
    x = torch.matmul(q, k.transpose(-1, -2)).view(n, H, nq, G, nk).mul_(s["scale"])
    x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, H, nq * G, nk), v).view(n, H, nq, G, -1) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(n, nq, heads, -1)[s["seq"], s["off"]]
    lse = (top + total.log()).permute(0, 2, 1, 3, 4).reshape(n, nq, heads)[s["seq"], s["off"]]
    return o.bfloat16(), lse


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_append(s) if c["op"] == "append" else _plain_attend(s)
    if c["op"] == "attend":
        return s["step"].attend(0, s["q"], scale=s["scale"], window=c.get("window", 0), out=s["out"], lse=s["lse"])
    if c["kind"] == "mla":
        q = s["step"].append(0, s["kv"][:, :LATENT], s["kv"][:, LATENT:], norm=s["norm"], eps=EPS,
                             q=s["q"][..., NOPE:], q_out=s["q_out"][..., LATENT:])
        return s["cache"], q
    heads, H = c["kv_heads"] * c["group"], c["kv_heads"]
    q = s["step"].append(0, s["qkv"][:, heads:heads + H], s["qkv"][:, heads + H:], norm=s["norm"], eps=EPS,
                         q=s["qkv"][:, :heads], q_norm=s["q_norm"], q_out=s["q_out"])
    return s["k_cache"], s["v_cache"], q


def work(case):
    c = case
    counts, kvs = _lengths(c)
    heads, rot, _, _ = _shape(c)
    T = sum(counts)
    mla = c["kind"] == "mla"
    row = 2 * (LATENT + ROPE) if mla else 4 * c["kv_heads"] * c["dim"]      # bytes a token has in the cache
    if c["op"] == "append":
        q = 2 * heads * (ROPE if mla else c["dim"])
        flops = T * (3 * rot * (heads + (1 if mla else c["kv_heads"])) + (4 * LATENT if mla else 0))
        if not mla and c["norm"]:
            flops += 4 * T * (heads + c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * T * (row + q), "flops": flops}
    w = c.get("window", 0)
    read = pairs = 0
    for q, k in zip(counts, kvs):
        first = k - q                                                       # the first query's own row
        low = max(0, first - w + 1) if w else 0
        read += k - low
        if w:
            full = max(0, min(q, w - 1 - first))                            # queries that see all before them
            pairs += full * (first + 1) + full * (full - 1) // 2 + (q - full) * w
        else:
            pairs += q * (first + 1) + q * (q - 1) // 2
    dq, dv = (LATENT + ROPE, LATENT) if mla else (c["dim"], c["dim"])
    return {"bytes": read * row + T * heads * (2 * (dq + dv) + 4), "flops": 2 * pairs * heads * (dq + dv)}


def _exact_append(s):
    c, z = s["case"], torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), _angles(s["case"], s["row"]))

    def turned(x, pairing):     # [T][heads][rot], each pair a complex number
        h = x.shape[-1] // 2
        re, im = (x[..., :h], x[..., h:]) if pairing == "half" else x.unflatten(-1, (h, 2)).unbind(-1)
        y = torch.complex(re, im) * z[:, None]
        return torch.cat([y.real, y.imag], -1) if pairing == "half" else torch.view_as_real(y).flatten(-2)

    def normed(x, w):
        return x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()

    if c["kind"] == "mla":
        cache = s["cache"].double()
        flat = cache.view(-1, LATENT + ROPE)
        flat[s["slot"], :LATENT] = normed(s["kv"][:, :LATENT].double(), s["norm"])
        flat[s["slot"], LATENT:] = turned(s["kv"][:, None, LATENT:].double(), "interleaved")[:, 0]
        return cache, turned(s["q"][..., NOPE:].double(), "interleaved")
    heads, H, rot = c["kv_heads"] * c["group"], c["kv_heads"], c["rot"]
    x = s["qkv"].double()
    q, k = normed(x[:, :heads], s["q_norm"]), normed(x[:, heads:heads + H], s["norm"])
    q[..., :rot], k[..., :rot] = turned(q[..., :rot], c["pairing"]), turned(k[..., :rot], c["pairing"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.view(-1, H, c["dim"])[s["slot"]] = k
    vc.view(-1, H, c["dim"])[s["slot"]] = x[:, heads + H:]
    return kc, vc, q


def _exact_attend(s):
    """One sequence and one head after another, queries in blocks."""
    c, P = s["case"], s["case"]["page"]
    heads = s["q"].shape[1]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for i, (nq, nk) in enumerate(zip(*_lengths(c))):
        j = torch.arange(nk, device="cuda")
        slot = s["table"][i, j // P].long() * P + j % P
        for h in range(heads):
            if c["kind"] == "mla":
                if h == 0:
                    k = s["cache"].view(-1, LATENT + ROPE)[slot].double()
                    v = k[:, :LATENT]
            elif h % c["group"] == 0:
                k = s["k_cache"].view(-1, c["kv_heads"], c["dim"])[slot, h // c["group"]].double()
                v = s["v_cache"].view(-1, c["kv_heads"], c["dim"])[slot, h // c["group"]].double()
            for b in range(0, nq, 4096):
                e = min(nq, b + 4096)
                r = torch.arange(nk - nq + b, nk - nq + e, device="cuda")[:, None]
                gone = j > r
                if c.get("window"):
                    gone |= j <= r - c["window"]
                x = (s["q"][at + b:at + e, h].double() @ k.t() * s["scale"]).masked_fill_(gone, -math.inf)
                lse[at + b:at + e, h] = torch.logsumexp(x, -1)
                out[at + b:at + e, h] = x.sub_(lse[at + b:at + e, h, None]).exp_() @ v
        at += nq
    return out, lse


def exact(case, seed):
    if work(case)["flops"] > 3e13 or case["n"] * (case.get("heads") or case["kv_heads"] * case["group"]) > 20000:
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
