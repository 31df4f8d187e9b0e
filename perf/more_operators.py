"""Operators around eviction by attention weight, as they are measured: cases,
inputs, the plain form and the 64-bit result of each.

  attend  attention of the new tokens over the paged cache, its scores capped by a
          tanh (one token or a chunk per sequence)
  weigh   the attention weight that each cached row gets from the step's tokens,
          summed over tokens and heads (what an eviction goes by)
  keep    the heaviest rows of each sequence as an eviction's keep mask, and their
          weights moved together as that eviction moves the rows
  train   the trainer's attention under the evictions' death times (query q sees
          key k iff k <= q < death[k]; packed documents are such death times too)
  back    its backward pass
"""

import math

import torch

own = False

LATENT, ROPE = 512, 64          # an MLA row: latent values, then the rotated band
NOPE = 128                      # the unrotated part of a projected MLA query head


def _mla(name, op, heads, n, q, kv, page, cap=0.0):
    return dict(name=name, op=op, kind="mla", heads=heads, n=n, q=q, kv=kv, page=page, cap=cap, window=0)


def _gqa(name, op, kv_heads, group, dim, n, q, kv, page, cap=0.0, window=0):
    return dict(name=name, op=op, kind="gqa", kv_heads=kv_heads, group=group, dim=dim, n=n, q=q, kv=kv, page=page,
                cap=cap, window=window)


def _keep(name, n, kv, budget, sinks, recent):
    return dict(name=name, op="keep", n=n, kv=kv, budget=budget, sinks=sinks, recent=recent)


def _train(name, op, n, tokens, kv_heads, group, dk, dv, cap=0.0, every=0, budget=0, doc=0):
    return dict(name=name, op=op, n=n, tokens=tokens, kv_heads=kv_heads, group=group, dk=dk, dv=dv, cap=cap,
                every=every, budget=budget, doc=doc)


def listed():
    return [
        # one user's next token under capped scores: latency
        _gqa("capped_attend_token", "attend", 8, 4, 128, 1, 1, 4097, 16, cap=50.0),
        # prompt chunks of a model of wide heads and capped scores: bound by arithmetic
        _gqa("capped_attend_chunk", "attend", 4, 2, 256, 2, 1024, 8192, 16, cap=50.0),
        # what one user's next token attends to: the smallest weighing
        _mla("weigh_token", "weigh", 16, 1, 1, 1531, 16),
        # a decoding batch of ragged contexts: bound by reading the keys
        _gqa("weigh_batch", "weigh", 8, 4, 128, 64, 1, 16384, 16),
        # prompts weighed in chunks, odd sizes, capped: bound by arithmetic
        _gqa("weigh_chunk", "weigh", 8, 4, 128, 3, 1501, 8191, 16, cap=30.0),
        # one user's cache cut to half
        _keep("keep_one", 1, 4097, 2048, 4, 64),
        # a serving batch cut to a quarter at once
        _keep("keep_batch", 96, 32768, 8192, 4, 256),
        # one short rollout of an MLA model (projected heads), cut every 128 tokens
        _train("train_short", "train", 1, 511, 16, 1, 192, 128, every=128, budget=200),
        # long rollouts of a GQA model with capped scores, cut every 2048 tokens
        _train("train_long", "train", 2, 8192, 8, 4, 128, 128, cap=50.0, every=2048, budget=2048),
        # short documents packed together, odd heads, a head size between the powers of two
        _train("back_documents", "back", 3, 389, 3, 5, 96, 96, doc=100),
        # rollouts of a GQA model, cut every 1024 tokens
        _train("back_rollouts", "back", 2, 4096, 8, 4, 128, 128, every=1024, budget=1024),
        # an MLA model's long rollout without evictions, capped, of odd length
        _train("back_mla", "back", 1, 4001, 16, 1, 192, 128, cap=30.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attend", "weigh", "weigh", "keep", "train", "back"])
    if op == "keep":
        kv = log(1, 131072)
        budget = max(1, int(kv * rng.choice([rng.random(), rng.random(), 1.5])))
        sinks = min(budget, rng.choice([0, 1, 4, 64]))
        c = _keep("", max(1, min(log(1, 128), (1 << 21) // kv)), kv, budget, sinks, min(budget - sinks, log(1, 2000) - 1))
    elif op in ("attend", "weigh"):
        shape = rng.choice(["token", "batch", "chunk"])
        n = {"token": 1, "batch": log(2, 64), "chunk": log(1, 6)}[shape]
        q = {"token": 1, "batch": rng.choice([1, 1, 2, 3]), "chunk": log(16, 2000)}[shape]
        kv = max(q, log(1, 131072 if shape == "token" else 16384))
        page, cap = rng.choice([1, 4, 16, 64, 256]), rng.choice([0.0, 15.0, 30.0, 50.0])
        if op == "attend":
            cap = cap or 50.0
        if rng.random() < 0.4:
            c = _mla("", op, rng.choice([8, 16, 32, 64, 128, 20]), n, q, kv, page, cap)
            heads, width = c["heads"], LATENT + ROPE
        else:
            c = _gqa("", op, rng.choice([1, 2, 4, 8, 3]), rng.choice([1, 4, 5, 8]),
                     rng.choice([32, 64, 80, 96, 128, 256]), n, q, kv, page, cap, rng.choice([0, 0, log(1, 4096)]))
            heads, width = c["kv_heads"] * c["group"], c["kv_heads"] * c["dim"]
        # no pass has more scores or rows than the listed ones
        while c["n"] * c["q"] * heads * c["kv"] > 1 << 30 or c["n"] * c["kv"] * width > 1 << 30 \
                or work(c)["flops"] > 1.2e11 or work(c)["bytes"] > 1.0e9:
            if c["n"] > 1:
                c["n"] = (c["n"] + 1) // 2
            else:
                c["kv"] = max(c["q"], c["kv"] * 2 // 3)
                c["q"] = c["q"] if c["kv"] > c["q"] else c["q"] * 2 // 3
    else:
        n, tokens = log(1, 4), log(1, 8192)
        dk, dv = rng.choice([(64, 64), (128, 128), (192, 128), (96, 96), (32, 32), (80, 80), (256, 256), (128, 64)])
        mask = rng.choice(["all", "cut", "cut", "doc"])
        c = _train("", op, n, tokens, rng.choice([1, 2, 4, 8, 3]), rng.choice([1, 2, 4, 5]), dk, dv,
                   cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                   every=log(16, max(17, tokens)) if mask == "cut" else 0, budget=log(1, max(2, tokens // 2)),
                   doc=log(1, tokens + 1) if mask == "doc" else 0)
        while c["n"] * c["kv_heads"] * c["group"] * c["tokens"] ** 2 > 1 << 30 or work(c)["flops"] > 6e11:
            if c["n"] > 1:
                c["n"] = (c["n"] + 1) // 2
            else:
                c["tokens"] = c["tokens"] * 2 // 3
    del c["name"]
    return c


# ---- the plan of a case

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


def _keep_lengths(c):
    """(rows, rows kept) of each sequence."""
    rows = [c["kv"] - (i * 7919) % (c["kv"] - c["kv"] // 2 + 1) for i in range(c["n"])]
    return rows, [min(c["budget"], r) for r in rows]


def _rollouts(c):
    """Length of each rollout of the batch."""
    t = c["tokens"]
    return [t - (i * 37) % (t // 4 + 1) for i in range(c["n"])]


def _cuts(c, length):
    return range(c["every"], length, c["every"]) if c["every"] else range(0)


def _shape(c):
    """(query heads, scale)."""
    if c["kind"] == "mla":
        return c["heads"], (NOPE + ROPE) ** -0.5
    return c["kv_heads"] * c["group"], c["dim"] ** -0.5


# ---- inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    return {"attend": _prepare_step, "weigh": _prepare_step, "keep": _prepare_keep, "train": _prepare_train,
            "back": _prepare_train}[case["op"]](case, dev, g)


def _prepare_step(c, dev, g):
    counts, kvs = _lengths(c)
    heads, scale = _shape(c)
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
    seq = torch.repeat_interleave(torch.arange(n, device=dev), count)
    off = torch.arange(T, device=dev) - torch.repeat_interleave(count.cumsum(0) - count, count)
    s = dict(case=c, scale=scale, table=table, count=count, length=torch.tensor(kvs, device=dev), seq=seq, off=off,
             max_q=max(counts), max_kv=max(kvs))
    if c["kind"] == "mla":
        s["cache"] = randn(1, total, P, LATENT + ROPE)
        s["q"] = randn(T, heads, LATENT + ROPE)
    else:
        s["k_cache"] = randn(1, total, P, c["kv_heads"], c["dim"])
        s["v_cache"] = randn(1, total, P, c["kv_heads"], c["dim"])
        s["q"] = randn(T, heads, c["dim"]) * 2.0
    if c["op"] == "attend":
        s["out"] = torch.zeros(T, heads, LATENT if c["kind"] == "mla" else c["dim"], device=dev, dtype=torch.bfloat16)
        s["lse"] = torch.zeros(T, heads, device=dev)
    else:
        x, _ = _scores(s)
        s["lse"] = _by_token(s, torch.logsumexp(x, -1)).contiguous()      # the attention before gave these
        s["weights"] = torch.zeros(n, width * P, device=dev)              # room for every row a sequence may hold
    if own:
        # what a serving loop holds: the pool, its sequences, and the plan of this
        # step, which every layer of the model uses
        from mla_paged_cache_amd import leyline as L
        if c["kind"] == "mla":
            s["pool"] = L.Pool(s["cache"], table)
        else:
            rot = 16
            while rot < 128 and c["dim"] % (2 * rot) == 0:
                rot *= 2
            s["pool"] = L.GqaPool(s["k_cache"], s["v_cache"], table, rotary_dim=rot)
        for i in range(n):
            s["pool"].seq_set_pages(i, pages[i], kvs[i])
        s["step"] = s["pool"].step(heads, max_seqs=n, max_tokens=T)
        s["step"].begin(list(range(n)), counts, grow=False)
    return s


def _prepare_keep(c, dev, g):
    rows, kept = _keep_lengths(c)
    n, room = c["n"], -(-max(rows) // 16) * 16
    length, budget = torch.tensor(rows, device=dev), torch.tensor(kept, device=dev)
    j = torch.arange(room, device=dev)
    live = j < length[:, None]
    # a few rows get most of the weight, many the same little, some none at all
    w = torch.exp(2.5 * torch.randn(n, room, generator=g, device=dev))
    coarse = torch.rand(n, room, generator=g, device=dev) < 0.4
    w = torch.where(coarse, w.bfloat16().float(), w)
    w = torch.where(torch.rand(n, room, generator=g, device=dev) < 0.1, torch.zeros_like(w), w)
    s = dict(case=c, weights=torch.where(live, w, torch.zeros_like(w)), length=length, budget=budget, room=room,
             place=torch.nonzero(live.flatten()).flatten(), kept=torch.zeros(n, room, device=dev),
             keep=torch.zeros(sum(rows), dtype=torch.uint8, device=dev))
    if own:
        from mla_paged_cache_amd import leyline as L
        per = [-(-r // 16) for r in rows]
        s["cache"] = torch.zeros(1, sum(per), 16, LATENT + ROPE, dtype=torch.bfloat16, device=dev)
        s["table"] = torch.full((n, room // 16), -1, dtype=torch.int32, device=dev)
        s["pool"] = L.Pool(s["cache"], s["table"])
        for r in rows:
            s["pool"].seq_alloc(r)
        s["seqs"], s["budgets"] = list(range(n)), [c["budget"]] * n
    return s


def _prepare_train(c, dev, g):
    n, T = c["n"], c["tokens"]
    H, heads, lens = c["kv_heads"], c["kv_heads"] * c["group"], _rollouts(c)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    death = torch.empty(n, T, dtype=torch.int32, device=dev)
    for i, length in enumerate(lens):
        j = torch.arange(T, device=dev)
        if c["doc"]:
            d = ((j // c["doc"] + 1) * c["doc"]).clamp(max=T)
        else:
            # the engine's evictions: each keeps `budget` of the tokens held then
            d = torch.full((T,), T, device=dev)
            held = torch.zeros(0, dtype=torch.int64, device=dev)
            before = 0
            for t in _cuts(c, length):
                held = torch.cat([held, torch.arange(before, t, device=dev)])
                before = t
                if held.numel() > c["budget"]:
                    p = torch.randperm(held.numel(), generator=g, device=dev)
                    d[held[p[c["budget"]:]]] = t
                    held = held[p[:c["budget"]]]
        death[i] = torch.where(j < length, d, j).to(torch.int32)
    real = torch.arange(T, device=dev) < torch.tensor(lens, device=dev)[:, None]
    s = dict(case=c, scale=c["dk"] ** -0.5, death=death, q=randn(n, T, heads, c["dk"]) * 2.0, k=randn(n, T, H, c["dk"]),
             v=randn(n, T, H, c["dv"]))
    if c["op"] == "back":
        s["dout"] = randn(n, T, heads, c["dv"]) * real[..., None, None].bfloat16()     # padding has no loss
        p, lse, _ = _probabilities(s)
        out = torch.matmul(p, s["v"].float().transpose(1, 2)).view(n, H, c["group"], T, c["dv"])
        s["out"] = out.permute(0, 3, 1, 2, 4).reshape(n, T, heads, c["dv"]).bfloat16()    # the forward pass gave
        s["lse"] = lse.permute(0, 3, 1, 2).reshape(n, T, heads).contiguous()              # these two
    if own:
        from mla_paged_cache_amd import leyline as L
        s["kvs"] = L.KvsMask(dev.index)
    return s


# ---- the plain forms

def _capped(x, cap):
    return cap * torch.tanh(x / cap) if cap else x


def _scores(s):
    """(scores [n][KV heads][queries][group][rows], values) of the step's tokens over
    their sequences, side by side and padded to the longest; unseen scores -inf."""
    c, P, dev = s["case"], s["case"]["page"], s["q"].device
    T, heads, width = s["q"].shape
    j = torch.arange(s["max_kv"], device=dev)
    rows = s["table"][:, j // P].clamp(min=0).long() * P + j % P                    # [n][kv]
    i = torch.arange(s["max_q"], device=dev)
    start = s["count"].cumsum(0) - s["count"]
    token = (start[:, None] + i).clamp(max=T - 1)                                   # [n][q]
    at = (s["length"] - s["count"])[:, None] + i                                    # a query's own row
    seen = (j <= at[..., None]) & (j < s["length"][:, None, None])
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    n, nq, nk = seen.shape
    if c["kind"] == "mla":
        k = s["cache"].view(-1, LATENT + ROPE)[rows].float()[:, None]               # [n][1][kv][576]
        v, H = k[..., :LATENT], 1
    else:
        H = c["kv_heads"]
        k = s["k_cache"].view(-1, H, width)[rows].float().transpose(1, 2)
        v = s["v_cache"].view(-1, H, width)[rows].float().transpose(1, 2) if c["op"] == "attend" else None
    G = heads // H
    q = s["q"][token].float().view(n, nq, H, G, width).permute(0, 2, 1, 3, 4).reshape(n, H, nq * G, width)
    x = torch.matmul(q, k.transpose(-1, -2)).view(n, H, nq, G, nk).mul_(s["scale"])
    return _capped(x, c["cap"]).masked_fill_(~seen[:, None, :, None, :], -math.inf), v


def _by_token(s, x):
    """[n][KV heads][queries][group] as [tokens][heads]."""
    return x.permute(0, 2, 1, 3).reshape(x.shape[0], x.shape[2], -1)[s["seq"], s["off"]]


def _plain_attend(s):
    x, v = _scores(s)
    n, H, nq, G, nk = x.shape
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, H, nq * G, nk), v).view(n, H, nq, G, -1) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(n, nq, H * G, -1)[s["seq"], s["off"]]
    return o.bfloat16(), _by_token(s, (top + total.log())[..., 0])


def _plain_weigh(s):
    x, _ = _scores(s)
    n, H, nq, G, nk = x.shape
    lse = torch.full((n, nq, H * G), math.inf, device=x.device)
    lse[s["seq"], s["off"]] = s["lse"]
    lse = lse.view(n, nq, H, G).permute(0, 2, 1, 3)[..., None]
    w = s["weights"]
    j = torch.arange(nk, device=x.device)
    w[:, :nk] = torch.where(j < s["length"][:, None], x.sub_(lse).exp_().sum((1, 2, 3)), w[:, :nk])
    return w


def _plain_keep(s):
    c, w = s["case"], s["weights"]
    n, room = w.shape
    j = torch.arange(room, device=w.device)
    length, budget = s["length"][:, None], s["budget"][:, None]
    safe = (j < c["sinks"]) | (j >= length - c["recent"])
    order = torch.where(j >= length, -math.inf, torch.where(safe, math.inf, w)).argsort(dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, j.expand(n, room))
    keep = rank < budget
    to = torch.where(keep, keep.cumsum(1) - 1, room)
    kept = torch.zeros(n, room + 1, device=w.device).scatter_(1, to, w)[:, :room]
    return keep.flatten()[s["place"]].to(torch.uint8), kept


def _probabilities(s):
    """(softmax weights [n][KV heads][group * T][T], lse [n][KV heads][group][T], the
    scores' tanh or None) under the death times."""
    c = s["case"]
    n, T, H, G = c["n"], c["tokens"], c["kv_heads"], c["group"]
    j = torch.arange(T, device=s["q"].device)
    seen = (j <= j[:, None]) & (j[:, None] < s["death"][:, None, :])                    # [n][q][k]
    q = s["q"].float().view(n, T, H, G, c["dk"]).permute(0, 2, 3, 1, 4).reshape(n, H, G * T, c["dk"])
    k = s["k"].float().transpose(1, 2)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(n, H, G, T, T)
    t = None
    if c["cap"]:
        t = x.div_(c["cap"]).tanh_()
        x = t * c["cap"]
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + total.log(), -math.inf)[..., 0]
    p /= torch.where(total > 0, total, 1.0)
    return p.view(n, H, G * T, T), lse, t


def _plain_train(s):
    c = s["case"]
    n, T, H, G = c["n"], c["tokens"], c["kv_heads"], c["group"]
    p, lse, _ = _probabilities(s)
    o = torch.matmul(p, s["v"].float().transpose(1, 2)).view(n, H, G, T, c["dv"])
    return o.permute(0, 3, 1, 2, 4).reshape(n, T, H * G, c["dv"]).bfloat16(), \
        lse.permute(0, 3, 1, 2).reshape(n, T, H * G).contiguous()


def _plain_back(s):
    c = s["case"]
    n, T, H, G, dk, dv = c["n"], c["tokens"], c["kv_heads"], c["group"], c["dk"], c["dv"]
    p, _, t = _probabilities(s)
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    q = s["q"].float().view(n, T, H, G, dk).permute(0, 2, 3, 1, 4).reshape(n, H, G * T, dk)
    do = s["dout"].float().view(n, T, H, G, dv).permute(0, 2, 3, 1, 4).reshape(n, H, G * T, dv)
    gv = torch.matmul(p.transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2))
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    if t is not None:
        ds *= 1 - t.view(ds.shape).square()
    gq = torch.matmul(ds, k).view(n, H, G, T, dk).permute(0, 3, 1, 2, 4).reshape(n, T, H * G, dk)
    gk = torch.matmul(ds.transpose(-1, -2), q)
    return gq.bfloat16(), gk.transpose(1, 2).bfloat16(), gv.transpose(1, 2).bfloat16()


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attend": _plain_attend, "weigh": _plain_weigh, "keep": _plain_keep, "train": _plain_train,
                "back": _plain_back}[c["op"]](s)
    if c["op"] == "attend":
        return s["step"].attend(0, s["q"], scale=s["scale"], window=c["window"], cap=c["cap"], out=s["out"], lse=s["lse"])
    if c["op"] == "weigh":
        # the weights of this step alone: what was there counts nothing
        return s["step"].weigh(0, s["q"], s["lse"], s["weights"], scale=s["scale"], window=c["window"], cap=c["cap"],
                               decay=0.0)
    if c["op"] == "keep":
        s["pool"].keep_heaviest(s["seqs"], s["budgets"], s["weights"], sinks=c["sinks"], recent=c["recent"],
                                keep=s["keep"], kept_weights=s["kept"])
        return s["keep"], s["kept"]
    if c["op"] == "train":
        return s["kvs"].attend(s["q"], s["k"], s["v"], s["death"], scale=s["scale"], cap=c["cap"])
    return s["kvs"].attend_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["death"], scale=s["scale"],
                                    cap=c["cap"])


# ---- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "keep":
        rows, kept = _keep_lengths(c)
        return {"bytes": sum(rows) * 9, "flops": sum(rows)}
    if c["op"] in ("train", "back"):
        pairs = 0
        for length in _rollouts(c):
            T, held, cuts = c["tokens"], 0, set(_cuts(c, length)) if not c["doc"] else ()
            for q in range(T):
                if c["doc"] and q % c["doc"] == 0:
                    held = 0
                if q in cuts:
                    held = min(held, c["budget"])
                held += q < length
                pairs += held
        heads, rows = c["kv_heads"] * c["group"], c["n"] * c["tokens"]
        q, kv, o = rows * heads * c["dk"] * 2, rows * c["kv_heads"] * (c["dk"] + c["dv"]) * 2, rows * heads * c["dv"] * 2
        if c["op"] == "train":
            return {"bytes": q + kv + o + rows * (4 * heads + 4), "flops": 2 * pairs * heads * (c["dk"] + c["dv"])}
        return {"bytes": 2 * q + 2 * kv + 2 * o + rows * (4 * heads + 4),
                "flops": 2 * pairs * heads * (3 * c["dk"] + 2 * c["dv"])}
    counts, kvs = _lengths(c)
    heads, _ = _shape(c)
    T, mla, w = sum(counts), c["kind"] == "mla", c["window"]
    read = pairs = 0
    for q, k in zip(counts, kvs):
        first = k - q                                                       # the first query's own row
        read += k - max(0, first - w + 1) if w else k
        if w:
            full = max(0, min(q, w - 1 - first))                            # queries that see all before them
            pairs += full * (first + 1) + full * (full - 1) // 2 + (q - full) * w
        else:
            pairs += q * (first + 1) + q * (q - 1) // 2
    dq, dv = (LATENT + ROPE, LATENT) if mla else (c["dim"], c["dim"])
    row = 2 * dq * (1 if mla else c["kv_heads"])                            # a token's keys
    if c["op"] == "weigh":
        return {"bytes": read * row + T * heads * (2 * dq + 4) + 4 * sum(kvs), "flops": 2 * pairs * heads * dq}
    return {"bytes": read * row * (1 if mla else 2) + T * heads * (2 * (dq + dv) + 4), "flops": 2 * pairs * heads * (dq + dv)}


# ---- in 64 bits

def _exact_step(s):
    """One sequence and one head after another, queries in blocks."""
    c, P = s["case"], s["case"]["page"]
    heads = s["q"].shape[1]
    attend = c["op"] == "attend"
    if attend:
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    else:
        weights = s["weights"].double()
    at = 0
    for i, (nq, nk) in enumerate(zip(*_lengths(c))):
        j = torch.arange(nk, device="cuda")
        slot = s["table"][i, j // P].long() * P + j % P
        total = torch.zeros(nk, dtype=torch.float64, device="cuda")
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
                if c["window"]:
                    gone |= j <= r - c["window"]
                x = s["q"][at + b:at + e, h].double() @ k.t() * s["scale"]
                if c["cap"]:
                    x = (x / c["cap"]).tanh() * c["cap"]
                x.masked_fill_(gone, -math.inf)
                if attend:
                    lse[at + b:at + e, h] = torch.logsumexp(x, -1)
                    out[at + b:at + e, h] = (x - lse[at + b:at + e, h, None]).exp() @ v
                else:
                    total += (x - s["lse"][at + b:at + e, h, None].double()).exp().sum(0)
        if not attend:
            weights[i, :nk] = total
        at += nq
    return (out, lse) if attend else weights


def _exact_keep(s):
    """Row after row of the sorted weights; ties by their place."""
    c = s["case"]
    rows, kept = _keep_lengths(c)
    keep, moved = [], torch.zeros(s["kept"].shape, dtype=torch.float64)
    for i, (r, b) in enumerate(zip(rows, kept)):
        w = s["weights"][i, :r].double().cpu().tolist()
        safe = set(range(min(c["sinks"], r))) | set(range(max(0, r - c["recent"]), r))
        rest = sorted((x for x in range(r) if x not in safe), key=lambda x: -w[x])
        mine = sorted(safe | set(rest[:max(0, b - len(safe))]))
        k = torch.zeros(r, dtype=torch.uint8)
        k[mine] = 1
        keep.append(k)
        moved[i, :len(mine)] = torch.tensor([w[x] for x in mine], dtype=torch.float64)
    return torch.cat(keep), moved


def _exact_train(s):
    """One rollout and one head after another."""
    c = s["case"]
    n, T, heads, back = c["n"], c["tokens"], c["kv_heads"] * c["group"], c["op"] == "back"
    kw = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(n, T, heads, c["dv"], **kw), torch.zeros(n, T, heads, **kw)
    gq, gk, gv = (torch.zeros(s[x].shape, **kw) for x in "qkv")
    at = torch.arange(T, device="cuda")
    for i in range(n):
        gone = (at[None, :] > at[:, None]) | (at[:, None] >= s["death"][i][None, :])
        blind = gone.all(1)
        for h in range(heads):
            q, k, v = s["q"][i, :, h].double(), s["k"][i, :, h // c["group"]].double(), s["v"][i, :, h // c["group"]].double()
            x = q @ k.t() * s["scale"]
            slope = None
            if c["cap"]:
                x = (x / c["cap"]).tanh_()
                slope = 1 - x * x if back else None
                x *= c["cap"]
            x.masked_fill_(gone, -math.inf)
            lse[i, :, h] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            p[blind] = 0
            if not back:
                out[i, :, h] = p @ v
                continue
            do = s["dout"][i, :, h].double()
            gv[i, :, h // c["group"]] += p.t() @ do
            o = p @ v
            ds = p * (do @ v.t() - (do * o).sum(-1, keepdim=True)) * s["scale"]
            if slope is not None:
                ds *= slope
            gq[i, :, h] = ds @ k
            gk[i, :, h // c["group"]] += ds.t() @ q
    return (gq, gk, gv) if back else (out, lse)


def exact(case, seed):
    c = case
    if c["op"] in ("attend", "weigh") and c["n"] * (c.get("heads") or c["kv_heads"] * c["group"]) > 10000:
        return None
    s = prepare(case, seed)
    return {"attend": _exact_step, "weigh": _exact_step, "keep": _exact_keep, "train": _exact_train,
            "back": _exact_train}[c["op"]](s)
