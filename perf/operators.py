"""What is measured of the shared-prefix cache: attention of a batch whose
sequences share prompts, over each sequence's own cached tokens as well, with
the weight every own token receives accumulated; and the eviction of the
lowest accumulated weights.

A case is a dict of sizes.  `prepare` makes its inputs, `run` makes one pass:
in elementary torch operations, or, where `own` is true, through
kv_cache_compression_hkv_b200.SharedPrefixCache.  `exact` is the definition in
64 bits, sequence by sequence.

attend   queries [S, H, T, d] are the newest T cached tokens of their
         sequences.  Query t of a sequence sees its whole prompt (one of G
         shared ones, or none) and the own slots before len - T + t + 1.  Out:
         the attention outputs, the log of each row's sum of exponentials, and
         (accumulate) weight[slot] += the softmax weights over the queries and
         the query heads of the slot's key head.
evict    appends a block of tokens with their weights, then brings every head
         of at least budget + block tokens back to its budget: the lowest
         (weight, position) go, tokens at a distance below `recent` from the
         newest last of all and oldest first; survivors behind the budget fill
         the holes before it, both in slot order.
"""
import math

import torch

own = False

#: What an eviction's pass leaves: the whole state of the cache.
EVICTED = ("k", "v", "pos", "weight", "lens", "next_pos")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# -- cases ---------------------------------------------------------------------

def _attend(name, dtype, seqs, heads, kv_heads, dim, queries, prefixes, prefix_len, own_len, capacity,
            least_len=0, accumulate=True, slot_major=False):
    case = dict(op="attend", dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, queries=queries,
                prefixes=prefixes, prefix_len=prefix_len, own_len=own_len, capacity=capacity,
                least_len=least_len, accumulate=accumulate, slot_major=slot_major)
    return dict(case, name=name) if name else case


def _evict(name, dtype, seqs, kv_heads, dim, budget, block, recent, least_budget, slot_major=False):
    case = dict(op="evict", dtype=dtype, seqs=seqs, kv_heads=kv_heads, dim=dim, budget=budget, block=block,
                recent=recent, least_budget=least_budget, slot_major=slot_major)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one layer of the 16x16 class-conditional model in fp32: a handful of
        # tokens, where the time is the calls'
        _attend("decode_tiny_f32", "f32", 2, 20, 20, 64, 1, 2, 1, 80, 80, 20),
        # one decode step of a 7B image model: 16 images of one prompt with
        # their unconditional halves, heads of 28 (window) to 138 tokens
        _attend("decode_janus_7b", "bf16", 32, 32, 32, 128, 1, 2, 64, 138, 138, 28),
        # the 48x49 image grid's caches: 56 to 477 own tokens a head
        _attend("decode_lumina", "bf16", 16, 32, 32, 128, 1, 2, 128, 477, 477, 56),
        # many samples of one long prompt, four query heads to a key head
        _attend("decode_long_prompt_gqa", "bf16", 48, 32, 8, 128, 1, 1, 16384, 1000, 1024, 700),
        # few sequences, long caches of their own, prompts of odd lengths
        _attend("decode_long_own_gqa", "bf16", 3, 32, 4, 128, 1, 2, 777, 32001, 32768, 9000, slot_major=True),
        # a row of image tokens and its line break at once
        _attend("block_image_row", "bf16", 16, 32, 32, 128, 49, 2, 128, 462, 480, 49),
        # the first image tokens behind a shared prompt, before any eviction
        _attend("prefill_lumina", "bf16", 16, 32, 32, 128, 256, 2, 128, 256, 480, 256),
        # a long own prompt behind a shared one, odd lengths
        _attend("prefill_long_gqa", "bf16", 2, 32, 8, 128, 4001, 2, 1000, 4001, 4096, 4001),
        # the 36-layer stack's prefill of a layer in fp32
        _attend("prefill_f32", "f32", 8, 20, 20, 64, 96, 2, 33, 96, 113, 96),
        # one token in, one out, as budgets are held in steady decoding
        _evict("evict_one_janus_7b", "bf16", 32, 32, 128, 106, 1, 28, 28),
        # a block of 64 out of 477
        _evict("evict_block_lumina", "bf16", 16, 32, 128, 413, 64, 56, 413),
        # a long context cut to two thirds
        _evict("evict_long", "bf16", 8, 8, 128, 16384, 8192, 512, 9000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    dim = rng.choice((64, 128))
    slot_major = rng.random() < 0.3
    kind = rng.choice(("decode", "decode", "block", "prefill", "evict", "evict"))
    if kind == "evict":
        seqs, kv_heads, budget = _log(rng, 1, 64), rng.choice((1, 2, 4, 8, 20, 32)), _log(rng, 16, 16384)
        while seqs * kv_heads * budget > 1 << (19 if dtype == "f32" else 20):
            budget = max(16, budget // 2 + 1)
            seqs = max(1, seqs - seqs // 4)
        block = _log(rng, 1, max(1, budget // 2))
        return _evict(None, dtype, seqs, kv_heads, dim, budget, block, rng.randint(0, budget // 2),
                      rng.choice((budget, budget // 2)), slot_major)
    kv_heads = rng.choice((1, 2, 4, 8, 16, 20, 32))
    rep = rng.choice((1, 1, 2, 4, 7, 8))
    rep = rep if kv_heads * rep <= 64 else 1
    prefixes = rng.choice((0, 1, 2, 2, 3))
    accumulate = rng.random() < 0.8
    if kind == "decode":
        queries, seqs, prefix_len, own_len = 1, _log(rng, 1, 64), _log(rng, 1, 16384), _log(rng, 1, 32768)
        most = 1 << 20
    elif kind == "block":
        queries, seqs, prefix_len = _log(rng, 2, 64), _log(rng, 1, 16), _log(rng, 1, 2048)
        own_len = queries + _log(rng, 1, 2048)
        most = 1 << 18
    else:
        queries, seqs, prefix_len = _log(rng, 65, 2500), _log(rng, 1, 16), _log(rng, 1, 1500)
        own_len = queries
        most = 1 << 16
    # no drawn case reads more slots than the largest listed decode, nor forms
    # more logits than the largest listed prefill
    most >>= dtype == "f32"
    while seqs * kv_heads * own_len > most and seqs > 1:
        seqs = max(1, seqs // 2)
    while prefixes * kv_heads * prefix_len > most // 2:
        prefix_len = prefix_len // 2 + 1
    while seqs * kv_heads * rep * queries * (own_len + prefix_len * max(1, prefixes)) > 1 << 29:
        if rep > 1:
            rep = 1
        elif kv_heads > 1:
            kv_heads //= 2
        else:
            seqs = max(1, seqs - 1)
    least = queries if kind != "decode" else rng.choice((0, own_len // 3, own_len))
    return _attend(None, dtype, seqs, kv_heads * rep, kv_heads, dim, queries, prefixes,
                   prefix_len if prefixes else 0, own_len, own_len + rng.randint(0, 40), least, accumulate,
                   slot_major)


# -- inputs --------------------------------------------------------------------

def _cache(g, dev, dtype, S, H, n, d, slot_major):
    """[S, H, n, d] unit-normal rows; slot_major: the slots of a sequence lie
    together in memory, [S, n, H, d]."""
    x = torch.randn((S, n, H, d) if slot_major else (S, H, n, d), generator=g, device=dev).to(dtype)
    return x.transpose(1, 2) if slot_major else x


def _lens(g, dev, S, H, lo, hi):
    n = torch.randint(lo, hi + 1, (S, H), generator=g, device=dev, dtype=torch.int32)
    n.view(-1)[0] = hi  # the longest one is there
    return n


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    S, Hk, d = case["seqs"], case["kv_heads"], case["dim"]
    st = {"case": case}
    if case["op"] == "evict":
        M, B = case["block"], case["budget"]
        cap = B + M
        st["k"] = _cache(g, dev, dt, S, Hk, cap, d, case["slot_major"])
        st["v"] = _cache(g, dev, dt, S, Hk, cap, d, case["slot_major"])
        st["budget"] = _lens(g, dev, S, Hk, case["least_budget"], B)
        st["lens"] = st["budget"].clone()  # as the last eviction left them
        # what a head's tokens have gathered: few heavy ones, many light
        st["weight"] = torch.empty(S, Hk, cap, device=dev).exponential_(generator=g).square_()
        # a thinned history in the order that evictions left
        order = torch.rand(S, Hk, 2 * cap, generator=g, device=dev).argsort(-1)[..., :cap]
        st["pos"] = order.to(torch.int32)
        st["next_pos"] = torch.full((S, Hk), 2 * cap, dtype=torch.int32, device=dev)
        st["k_t"] = _cache(g, dev, dt, S, Hk, M, d, case["slot_major"])
        st["v_t"] = _cache(g, dev, dt, S, Hk, M, d, case["slot_major"])
        st["w_t"] = torch.empty(S, Hk, M, device=dev).exponential_(generator=g)
        return st
    H, T, G, P, cap = case["heads"], case["queries"], case["prefixes"], case["prefix_len"], case["capacity"]
    st["k"] = _cache(g, dev, dt, S, Hk, cap, d, case["slot_major"])
    st["v"] = _cache(g, dev, dt, S, Hk, cap, d, case["slot_major"])
    st["lens"] = _lens(g, dev, S, Hk, case["least_len"], case["own_len"])
    st["pos"] = torch.arange(cap, dtype=torch.int32, device=dev).expand(S, Hk, cap).contiguous()
    st["weight"] = torch.rand(S, Hk, cap, generator=g, device=dev)
    st["prefix_k"] = _cache(g, dev, dt, G, Hk, P, d, False)
    st["prefix_v"] = _cache(g, dev, dt, G, Hk, P, d, False)
    st["prefix_lens"] = torch.full((G,), P, dtype=torch.int32, device=dev)
    if G > 1:
        st["prefix_lens"][1] = max(1, P - P // 3)  # prompts of unequal length
    # batches laid out as [conditional | unconditional], G ranges
    st["prefix_of"] = (torch.arange(S, device=dev) * max(G, 1) // S).to(torch.int32)
    # a query looks for one of its own tokens and one of its prompt's
    rep = H // Hk
    q = torch.randn(S, Hk, rep, T, d, generator=g, device=dev)
    at = (torch.rand(S, Hk, rep * T, generator=g, device=dev) * st["lens"].clamp(min=1)[..., None]).long()
    q += 0.35 * st["k"].gather(2, at[..., None].expand(-1, -1, -1, d)).float().view(S, Hk, rep, T, d)
    if G:
        of = st["prefix_of"].long()
        at = (torch.rand(S, Hk, rep * T, generator=g, device=dev) * st["prefix_lens"][of][:, None, None]).long()
        near = st["prefix_k"][of[:, None, None], torch.arange(Hk, device=dev)[None, :, None], at]
        q += 0.35 * near.float().view(S, Hk, rep, T, d)
    st["q"] = q.view(S, H, T, d).to(dt)
    return st


# -- one pass ------------------------------------------------------------------

def _handle(st):
    """The cache object over the state's buffers, made once as a program does."""
    if "cache" not in st:
        import kv_cache_compression_hkv_b200 as hkv
        c = st["case"]
        cfg = hkv.SharedConfig(
            num_seqs=c["seqs"], num_heads=c.get("heads", c["kv_heads"]), num_kv_heads=c["kv_heads"],
            head_dim=c["dim"], capacity=st["k"].shape[2], num_prefixes=c.get("prefixes", 0),
            prefix_capacity=c.get("prefix_len", 0), dtype=hkv.DTYPE_F32 if c["dtype"] == "f32" else hkv.DTYPE_BF16)
        st["cache"] = hkv.SharedPrefixCache(
            cfg, device=st["k"].device, k=st["k"], v=st["v"], pos=st["pos"], weight=st["weight"], lens=st["lens"],
            next_pos=st.get("next_pos"), prefix_k=st.get("prefix_k"), prefix_v=st.get("prefix_v"), prefix_lens=st.get("prefix_lens"),
            prefix_of=st.get("prefix_of"))
    return st["cache"]


def _run_own(st):
    cache, c = _handle(st), st["case"]
    if c["op"] == "evict":
        cache.append(st["k_t"], st["v_t"], st["w_t"])
        cache.evict(st["budget"], c["recent"], slack=c["block"])
        return {n: st[n] for n in EVICTED}
    out, lse = cache.attend(st["q"], accumulate=c["accumulate"])
    return {"out": out, "lse": lse, "weight": st["weight"]}


def _plain_attend(st):
    c = st["case"]
    S, H, Hk, T, d, G = c["seqs"], c["heads"], c["kv_heads"], c["queries"], c["dim"], c["prefixes"]
    rep, cap = H // Hk, c["capacity"]
    dev = st["q"].device
    q = st["q"].float().view(S, Hk, rep * T, d) * (1.0 / math.sqrt(d))
    first = st["lens"].long() - T + 1                                             # slots that query 0 sees
    sees = (first[..., None] + torch.arange(T, device=dev)).repeat(1, 1, rep)     # [S, Hk, rep T]
    hidden = torch.arange(cap, device=dev) >= sees[..., None]
    x = torch.matmul(q, st["k"].float().transpose(-1, -2)).masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    if G:
        of = st["prefix_of"].long()
        # every sequence against every prompt, then its own prompt's part
        qg = q.transpose(0, 1).reshape(1, Hk, S * rep * T, d)
        y = torch.matmul(qg, st["prefix_k"].float().transpose(-1, -2)).view(G, Hk, S, rep * T, -1)
        y = y.permute(2, 0, 1, 3, 4)[torch.arange(S, device=dev), of]
        past = torch.arange(y.shape[-1], device=dev) >= st["prefix_lens"][of][:, None]
        y = y.masked_fill(past[:, None, None, :], -math.inf)
        m = torch.maximum(m, y.amax(-1, keepdim=True))
    m = m.masked_fill(m == -math.inf, 0.0)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, st["v"].float())
    if G:
        y = (y - m).exp_()
        total = total + y.sum(-1, keepdim=True)
        mine = of[None, :] == torch.arange(G, device=dev)[:, None]                # [G, S]
        yg = y.permute(1, 0, 2, 3)[None] * mine[:, None, :, None, None]
        yg = yg.reshape(G, Hk, S * rep * T, -1)
        o = o + torch.matmul(yg, st["prefix_v"].float()).sum(0).view(Hk, S, rep * T, d).transpose(0, 1)
    lse = m + total.log()
    inv = torch.where(total > 0, 1.0 / total, total)
    if c["accumulate"]:
        st["weight"] += x.mul_(inv).sum(2)
    return {"out": (o * inv).view(S, H, T, d).to(st["q"].dtype), "lse": lse.view(S, H, T), "weight": st["weight"]}


def _plain_evict(st):
    c = st["case"]
    M, cap = c["block"], c["budget"] + c["block"]
    dev = st["k"].device
    # the block behind each head's last token
    slot = st["lens"].long()[..., None] + torch.arange(M, device=dev)
    for name in ("k", "v"):
        st[name].scatter_(2, slot[..., None].expand(st[name + "_t"].shape), st[name + "_t"])
    st["weight"].scatter_(2, slot, st["w_t"])
    st["pos"].scatter_(2, slot, st["next_pos"][..., None] + torch.arange(M, dtype=torch.int32, device=dev))
    st["next_pos"] += M
    n = st["lens"].long() + M
    budget = st["budget"].long()
    due = n >= budget + M
    idx = torch.arange(cap, device=dev)
    valid = idx < n[..., None]
    pos = st["pos"].long()
    newest = pos.masked_fill(~valid, -1 << 40).amax(-1, keepdim=True)
    recent = pos > newest - c["recent"]
    # (class, weight, position, slot) ascending by stable sorts, last key first
    order = pos.argsort(dim=-1, stable=True)
    w = st["weight"].masked_fill(recent, 0.0).gather(-1, order)
    order = order.gather(-1, w.argsort(dim=-1, stable=True))
    kind = torch.where(valid, recent.long(), 2).gather(-1, order)
    order = order.gather(-1, kind.argsort(dim=-1, stable=True))
    rank = torch.empty_like(order).scatter_(-1, order, idx.expand_as(order).contiguous())
    gone = due[..., None] & (rank < (n - budget)[..., None])
    hole = gone & (idx < budget[..., None])
    mover = due[..., None] & valid & ~gone & (idx >= budget[..., None])
    movers = (~mover).to(torch.int8).argsort(dim=-1, stable=True)
    src = movers.gather(-1, (hole.long().cumsum(-1) - 1).clamp_(min=0))
    at = hole.nonzero(as_tuple=True)
    frm = (at[0], at[1], src[at])
    for name in ("k", "v", "pos", "weight"):
        st[name][at] = st[name][frm]
    st["lens"].copy_(torch.where(due, budget, n))
    return {n: st[n] for n in EVICTED}


def run(state):
    if own:
        return _run_own(state)
    return _plain_evict(state) if state["case"]["op"] == "evict" else _plain_attend(state)


# -- what a pass cannot do without ---------------------------------------------

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    S, Hk, d = case["seqs"], case["kv_heads"], case["dim"]
    if case["op"] == "evict":
        B, M = (case["least_budget"] + case["budget"]) / 2, case["block"]
        rows = S * Hk
        # the block in (k, v, weight; position made) and out; every token's
        # weight and position read; the rows that move: of M evicted ones
        # M B / (B + M) lie before the budget where all slots are alike
        moved = M * B / (B + M)
        return {"bytes": rows * (M * (4 * d * es + 12) + (B + M) * 8 + moved * (4 * d * es + 16) + 8),
                "flops": rows * (B + M)}
    H, T, G, P = case["heads"], case["queries"], case["prefixes"], case["prefix_len"]
    n = (case["least_len"] + case["own_len"]) / 2
    lens = [P if g != 1 else max(1, P - P // 3) for g in range(G)]
    prefix = sum(lens) / G if G else 0.0
    seen = prefix + max(n - (T - 1) / 2, n / 2)
    acc = 2 * S * Hk * n * 4 if case["accumulate"] else 0
    return {"bytes": 2 * S * H * T * d * es + 2 * S * Hk * n * d * es + 2 * sum(lens) * Hk * d * es + S * H * T * 4 + acc,
            "flops": 4.0 * S * H * T * seen * d}


# -- the definition in 64 bits -------------------------------------------------

def _exact_attend(st):
    c = st["case"]
    S, H, Hk, T, d, G = c["seqs"], c["heads"], c["kv_heads"], c["queries"], c["dim"], c["prefixes"]
    rep = H // Hk
    out = torch.zeros(S, H, T, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.empty(S, H, T, dtype=torch.float64, device=out.device)
    weight = st["weight"].double()
    lens, pl, of = st["lens"].tolist(), st["prefix_lens"].tolist(), st["prefix_of"].tolist()
    for s in range(S):
        p = pl[of[s]] if G else 0
        for h in range(Hk):
            n = lens[s][h]
            keys, vals = st["k"][s, h, :n].double(), st["v"][s, h, :n].double()
            if p:
                keys = torch.cat([st["prefix_k"][of[s], h, :p].double(), keys])
                vals = torch.cat([st["prefix_v"][of[s], h, :p].double(), vals])
            x = st["q"][s, h * rep:(h + 1) * rep].double() @ keys.T / math.sqrt(d)    # [rep, T, p + n]
            # query t stands at own slot n - T + t
            last = p + n - T + torch.arange(T, device=x.device)
            x[:, torch.arange(p + n, device=x.device)[None, :] > last[:, None]] = -math.inf
            e = torch.logsumexp(x, -1)
            lse[s, h * rep:(h + 1) * rep] = e
            w = (x - e[..., None]).exp().nan_to_num(0.0)
            out[s, h * rep:(h + 1) * rep] = w @ vals
            if c["accumulate"]:
                weight[s, h, :n] += w[..., p:].sum((0, 1))
    return {"out": out, "lse": lse, "weight": weight}


def _exact_evict(st):
    import numpy as np
    c = st["case"]
    M = c["block"]
    pos, weight, lens = (st[n].cpu().numpy() for n in ("pos", "weight", "lens"))
    budget, t, w_t = (st[n].cpu().numpy() for n in ("budget", "next_pos", "w_t"))
    k, v = st["k"].double(), st["v"].double()
    for s in range(c["seqs"]):
        for h in range(c["kv_heads"]):
            a, B = int(lens[s, h]), int(budget[s, h])
            n = a + M
            k[s, h, a:n], v[s, h, a:n] = st["k_t"][s, h].double(), st["v_t"][s, h].double()
            pos[s, h, a:n], weight[s, h, a:n] = t[s, h] + np.arange(M), w_t[s, h]
            lens[s, h] = n
            if n < B + M:
                continue
            p, w = pos[s, h, :n].astype(np.int64), weight[s, h, :n].astype(np.float64)
            near = p.max() - p < c["recent"]
            order = np.lexsort((np.arange(n), p, np.where(near, 0.0, w), near))
            gone = np.zeros(n, bool)
            gone[order[: n - B]] = True
            holes, movers = np.nonzero(gone[:B])[0], B + np.nonzero(~gone[B:])[0]
            pos[s, h, holes], weight[s, h, holes] = pos[s, h, movers], weight[s, h, movers]
            hi, mi = torch.from_numpy(holes).to(k.device), torch.from_numpy(movers).to(k.device)
            k[s, h, hi], v[s, h, hi] = k[s, h, mi], v[s, h, mi]
            lens[s, h] = B
    return {"k": k, "v": v, "pos": torch.from_numpy(pos), "weight": torch.from_numpy(weight).double(),
            "lens": torch.from_numpy(lens), "next_pos": torch.from_numpy(t + M)}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_evict(st) if case["op"] == "evict" else _exact_attend(st)
