"""Cases that measure the paged-cache operators: kv_append, forward_paged and
forward_shared_prefix.

Each case is one pass through one operator, at sizes a serving program meets.
`run` computes it in plain fp32 torch operations (own = False) or through the
framework's public calls (own = True), and `exact` in 64 bits.

The key/value cache is a pool of pages, [pages, Hkv, page, D], and a table
gives the pages of each sequence in order.  `lo` and `hi` bound the sequences'
own lengths, the tokens of the pass included.
"""
import math

import torch

own = False

# The multiples of this number, modulo 1, are spread evenly: they give a batch's
# lengths in [lo, hi], the same for every seed, so that a case fixes its work.
_GOLDEN = 0.6180339887498949

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(name, op, dtype, B, T, Hq, Hkv, D, page, lo, hi, prefix=0, rot=0, interleaved=False):
    return dict(name=name, op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, lo=lo, hi=hi,
                prefix=prefix, rot=rot, interleaved=interleaved)


def listed():
    return [
        # one user, one new token: the smallest call, where latency is all
        _case("append_one", "append", "bf16", 1, 1, 32, 8, 128, 16, 1000, 1000, rot=128),
        # one decoding step of a large batch
        _case("append_step", "append", "bf16", 256, 1, 32, 8, 128, 64, 1, 4096, rot=128),
        # two long prompts written at once: limited by memory bandwidth
        _case("append_prompt", "append", "bf16", 2, 8192, 32, 8, 128, 64, 8192, 8192, rot=128),
        # odd prompt lengths, pages of 24, neighbouring pairs over half of the head
        _case("append_ragged", "append", "f16", 3, 777, 16, 16, 64, 24, 500, 1777, rot=32, interleaved=True),
        # one user, one token, a short context
        _case("paged_one", "paged", "bf16", 1, 1, 32, 8, 128, 16, 1000, 1000),
        # one user, one token, a context of 128 k tokens
        _case("paged_long", "paged", "bf16", 1, 1, 32, 8, 128, 64, 131072, 131072),
        # a decoding step of a batch of very different lengths, a free slot (length 0) among them
        _case("paged_step", "paged", "bf16", 64, 1, 32, 8, 128, 64, 0, 8191),
        # five drafted tokens verified at once, every head with keys of its own
        _case("paged_draft", "paged", "f16", 16, 5, 16, 16, 64, 16, 700, 4095),
        # the last 1024 tokens of a prompt that is read in pieces
        _case("paged_chunk", "paged", "bf16", 1, 1024, 32, 8, 128, 64, 16384, 16384),
        # four samples that continue one prompt
        _case("shared_few", "shared", "f16", 4, 1, 16, 16, 64, 16, 1, 200, prefix=1000),
        # a batch over one long document
        _case("shared_long", "shared", "bf16", 64, 1, 32, 8, 128, 64, 0, 1023, prefix=16384),
        # many requests with the same instructions in front
        _case("shared_wide", "shared", "bf16", 256, 1, 32, 8, 128, 64, 1, 511, prefix=4097),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    limit = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("append", "paged", "shared")}
    while True:
        op = rng.choice(["append", "paged", "shared"])
        Hkv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8])
        D = rng.choice([40, 64, 64, 80, 96, 128, 128, 128, 256])
        T = rng.choice([1, 1, 1, 2, 5, 8, _log(rng, 16, 1024)])
        hi = _log(rng, 16, 32768)
        case = dict(op=op, dtype=rng.choice(["bf16", "f16"]), B=_log(rng, 1, 256), T=min(T, hi), Hq=Hkv * group,
                    Hkv=Hkv, D=D, page=rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]),
                    lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, prefix=0, rot=0, interleaved=False)
        if op == "append":
            case["T"] = rng.choice([1, 1, min(hi, _log(rng, 2, 8192))])
            case["rot"] = rng.choice([D, D // 2 // 2 * 2])
            case["interleaved"] = rng.choice([False, True])
        if op == "shared":
            case["T"] = min(case["T"], 8)
            case["prefix"] = _log(rng, 64, 32768)
            case["hi"] = min(hi, 4096)
            case["lo"] = min(case["lo"], case["hi"])
            case["T"] = min(case["T"], case["hi"])
        pool = case["Hkv"] * D * (case["prefix"] + sum(_lengths(case)))
        scores = case["B"] * case["Hq"] * case["T"] * (case["prefix"] + case["hi"])
        padded = case["B"] * case["Hkv"] * case["hi"] * D
        if _cost(case) <= limit[op] and max(pool, scores, padded) <= 1 << 29:
            return case


def _lengths(case):
    """The own lengths of the batch's sequences: fixed by the case, spread over [lo, hi]."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    if B == 1:
        return [hi]
    return [lo + int((b * _GOLDEN) % 1.0 * (hi - lo + 1)) for b in range(B)]


def _cost(case):
    """About the seconds of a pass, by what the work alone costs."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.8e15)


def work(case):
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    lens = _lengths(case)
    if case["op"] == "append":
        tokens = sum(min(T, n) for n in lens)
        # every value is read once and written once; a rotated pair costs 6 operations
        return {"bytes": 4 * tokens * (Hq + 2 * Hkv) * D, "flops": 3 * tokens * (Hq + Hkv) * case["rot"]}
    P = case["prefix"]
    # a query of the last T tokens sees the keys up to its own position
    seen = sum(min(T, n) * (P + n) - min(T, n) * (min(T, n) - 1) // 2 for n in lens)
    io = 2 * B * Hq * T * D * 2 + 4 * B * Hq * T
    return {"bytes": io + 4 * Hkv * D * (P + sum(lens)), "flops": 4 * Hq * D * seen}


def _pages(n, page):
    return -(-n // page)


def prepare(case, seed):
    B, T, Hq, Hkv, D, page, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page", "prefix"))
    dtype, lens = _TYPES[case["dtype"]], _lengths(case)
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    width = max(1, _pages(case["hi"], page))
    need = [_pages(n, page) for n in lens]
    first = _pages(P, page)
    pool = first + sum(need) + 3                       # a few pages are free
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros((B, width), dtype=torch.int32)
    at = first
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state = {"case": case, "table": table.cuda(), "seq_len": torch.tensor(lens, dtype=torch.int32).cuda(),
             "prefix_table": order[:first].cuda(), "spare": int(order[-1])}
    # the pool is made slice by slice, so that its fp32 draws stay small
    state["k_cache"], state["v_cache"] = (torch.empty((pool, Hkv, page, D), dtype=dtype, device="cuda") for _ in range(2))
    step = max(1, (1 << 27) // (Hkv * page * D))
    for c in (state["k_cache"], state["v_cache"]):
        for i in range(0, pool, step):
            n = min(step, pool - i)
            c[i:i + n] = normal(n, Hkv, page, D)
    # the projection's output holds q, k and v of a token side by side
    if case["op"] == "append":
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        state["q"], state["k"], state["v"] = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
        half = case["rot"] // 2
        state["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(1, half))).float().cuda()
    else:
        state["q"] = normal(B, T, Hq, D).transpose(1, 2)
    if own:
        import exact_tiled_attention_23_gb300 as fa
        # the handle that a serving program keeps beside its cache
        state["cache"] = fa.PagedKV(state["k_cache"], state["v_cache"], state["table"], state["seq_len"])
    return state


def run(state):
    if own:
        import exact_tiled_attention_23_gb300 as fa
        case, cache = state["case"], state["cache"]
        if case["op"] == "append":
            q = fa.kv_append(cache, state["k"], state["v"], q=state["q"], inv_freq=state["inv_freq"],
                             interleaved=case["interleaved"])
            return q, state["k_cache"], state["v_cache"]
        if case["op"] == "paged":
            return fa.forward_paged(state["q"], cache)
        return fa.forward_shared_prefix(state["q"], cache, state["prefix_table"], case["prefix"])
    if state["case"]["op"] == "append":
        return _append(state, torch.float32, state["k_cache"], state["v_cache"])
    return _attention(state, torch.float32)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "append":
        return _exact_append(state)
    if work(case)["flops"] > 6e11:
        return None
    return _exact_attention(state)


# ------------------------------------------------------------ the plain forms
def _append(state, wide, k_cache, v_cache):
    """Rotate k and q by their positions and put k, v into the sequences' pages."""
    case = state["case"]
    B, T, rot, page = case["B"], case["T"], case["rot"], case["page"]
    pos = state["seq_len"].long()[:, None] - T + torch.arange(T, device="cuda")      # [B, T]; below 0: no token
    angle = pos.double()[..., None] * state["inv_freq"].double()                       # far positions need 64 bits
    cos, sin = angle.cos().to(wide)[:, None], angle.sin().to(wide)[:, None]

    def turn(x):
        x = x.to(wide)
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    live = pos >= 0
    q = torch.where(live[:, None, :, None], turn(state["q"]), 0).to(state["q"].dtype)
    k = turn(state["k"]).to(k_cache.dtype).transpose(1, 2)                             # [B, T, Hkv, D]
    v = state["v"].to(v_cache.dtype).transpose(1, 2)
    at = pos.clamp_min(0)
    pages = state["table"].long().gather(1, at // page)
    # a slot without a token writes back what the first token's slot holds
    slot = at % page
    first = torch.where(live, torch.arange(T, device="cuda"), T).amin(dim=1, keepdim=True).clamp_max(T - 1)
    which = torch.where(live, torch.arange(T, device="cuda"), first)
    rows = torch.arange(B, device="cuda")[:, None]
    pages, slot = pages.gather(1, which), slot.gather(1, which)
    some = live.any(dim=1)[:, None, None, None]
    pages = torch.where(some[:, :, 0, 0], pages, state["spare"])
    k_cache[pages, :, slot] = torch.where(some, k[rows, which], k_cache[pages, :, slot])
    v_cache[pages, :, slot] = torch.where(some, v[rows, which], v_cache[pages, :, slot])
    return q, k_cache, v_cache


def _attention(state, wide):
    """softmax(q k^T / sqrt(D)) v over the prefix and the sequence's own pages."""
    case = state["case"]
    B, T, Hq, Hkv, D, page, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page", "prefix"))
    G = Hq // Hkv
    q = state["q"].to(wide).reshape(B, Hkv, G, T, D).reshape(B, Hkv, G * T, D)
    table, n = state["table"].long(), state["seq_len"].long()
    own_k, own_v = (c[table].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :case["hi"]].to(wide)
                    for c in (state["k_cache"], state["v_cache"]))
    pos = torch.arange(T, device="cuda") + n[:, None] - T                                  # [B, T]
    seen = torch.arange(own_k.shape[2], device="cuda") <= pos[..., None]                   # [B, T, keys]
    seen = seen[:, None].expand(B, G, T, -1).reshape(B, 1, G * T, -1)
    scores = (q @ own_k.transpose(2, 3) / math.sqrt(D)).masked_fill(~seen, -math.inf)
    if P:
        pages = state["prefix_table"].long()
        pre_k, pre_v = (c[pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :P].to(wide)
                        for c in (state["k_cache"], state["v_cache"]))
        stacked = q.transpose(0, 1).reshape(Hkv, B * G * T, D)
        front = (stacked @ pre_k.transpose(1, 2) / math.sqrt(D)).reshape(Hkv, B, G * T, P).transpose(0, 1)
        front = front.masked_fill((pos < 0)[:, None].expand(B, G, T).reshape(B, 1, G * T, 1), -math.inf)
        top = torch.maximum(front.amax(dim=3, keepdim=True), scores.amax(dim=3, keepdim=True))
    else:
        top = scores.amax(dim=3, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    p = (scores - top).exp()
    total, o = p.sum(dim=3, keepdim=True), p @ own_v
    if P:
        p = (front - top).exp()
        total = total + p.sum(dim=3, keepdim=True)
        o = o + (p.transpose(0, 1).reshape(Hkv, B * G * T, P) @ pre_v).reshape(Hkv, B, G * T, D).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0).to(state["q"].dtype)
    lse = (top + total.log()).squeeze(3)
    return o.reshape(B, Hq, T, D), lse.reshape(B, Hq, T)


# ------------------------------------------------------------------- 64 bits
def _exact_append(state):
    """One sequence at a time: the rotation as a product of complex numbers."""
    case = state["case"]
    T, rot, page, Hkv, D = (case[k] for k in ("T", "rot", "page", "Hkv", "D"))
    f = state["inv_freq"].double()
    q = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()

    def turned(x, pos):                                    # [H, t, D], [t]
        x = x.double().clone()
        z = torch.polar(torch.ones_like(pos[:, None] * f), pos[:, None] * f)
        r = x[..., :rot]
        pairs = r.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        x[..., :rot] = w.flatten(-2) if case["interleaved"] else w.transpose(-1, -2).flatten(-2)
        return x

    for b, n in enumerate(_lengths(case)):
        t = min(T, n)
        if t == 0:
            continue
        pos = torch.arange(n - t, n, device="cuda")
        q[b, :, T - t:] = turned(state["q"][b, :, T - t:], pos.double())
        pages = state["table"][b].long()[pos // page]
        k_cache[pages, :, pos % page] = turned(state["k"][b, :, T - t:], pos.double()).transpose(0, 1)
        v_cache[pages, :, pos % page] = state["v"][b, :, T - t:].double().transpose(0, 1)
    return q, k_cache, v_cache


def _exact_attention(state):
    """One sequence and one key head at a time, over exactly the keys it has."""
    case = state["case"]
    B, T, Hq, Hkv, D, page, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page", "prefix"))
    G = Hq // Hkv
    o = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")

    def rows(pages, n, h):
        return [c[pages.long()[:_pages(n, page)], h].reshape(-1, D)[:n].double()
                for c in (state["k_cache"], state["v_cache"])]

    for h in range(Hkv):
        pre = rows(state["prefix_table"], P, h)
        for b, n in enumerate(_lengths(case)):
            t = min(T, n)
            if t == 0:
                continue
            own_k, own_v = rows(state["table"][b], n, h)
            k, v = torch.cat([pre[0], own_k]), torch.cat([pre[1], own_v])
            s = state["q"][b, h * G:(h + 1) * G, T - t:].double() @ k.T / math.sqrt(D)      # [G, t, keys]
            ends = torch.arange(P + n - t, P + n, device="cuda")
            s = s.masked_fill(torch.arange(P + n, device="cuda") > ends[:, None], -math.inf)
            lse[b, h * G:(h + 1) * G, T - t:] = s.logsumexp(dim=2)
            o[b, h * G:(h + 1) * G, T - t:] = s.softmax(dim=2) @ v
    return o, lse
