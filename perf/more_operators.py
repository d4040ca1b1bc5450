"""Cases that measure the 4-bit paged cache (kv_append and forward_paged over a
PagedKV4, kv_read), positions of several axes (rotary, kv_append) and the cache's
pages (kv_grow, kv_fork, kv_free, kv_compact).

Each case is one pass through one operator, at sizes a serving or training
program meets.  `run` computes it in plain fp32 torch operations (own = False) or
through the framework's public calls (own = True), and `exact` in 64 bits.

A 16-bit cache is a pool of pages, [pages, Hkv, page, D], and a table gives the
pages of each sequence in order.  A 4-bit cache holds a row of a key or value in
groups of 16 elements, each a number of 4 bits (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times the group's scale, an unsigned
number of 8 bits (5 exponent bits, 3 mantissa bits: the upper bits of an IEEE
half).  Rows are padded to 64, 128 or 256 elements.  `lo` and `hi` bound the
sequences' lengths, the tokens of the pass included.
"""
import math

import torch

own = False

# The multiples of this number, modulo 1, are spread evenly: they give a batch's
# lengths in [lo, hi], the same for every seed, so that a case fixes its work.
_GOLDEN = 0.6180339887498949

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

_BASE = dict(dtype="bf16", B=1, T=1, Hq=32, Hkv=8, D=128, page=64, lo=1, hi=1, rot=0, axes=1, interleaved=False, spare=0)


def _case(name, op, **more):
    return {**_BASE, "name": name, "op": op, **more}


def listed():
    return [
        # queries and keys of a short video, turned by time, height and width, with the gradients
        _case("rotary_video", "rotary", T=32760, Hq=16, Hkv=16, rot=128, axes=3),
        # three images of odd sizes in a batch, neighbouring pairs over half of the head
        _case("rotary_image", "rotary", dtype="f16", B=3, T=777, Hq=16, Hkv=4, D=80, rot=40, axes=2, interleaved=True),
        # a decoding step whose tokens follow images: positions of three axes
        _case("append_axes", "append", B=64, hi=512, rot=128, axes=3),
        # one decoding step of a large batch into a 4-bit cache
        _case("append4_step", "append4", B=256, hi=4096, rot=128),
        # two long prompts written to a 4-bit cache at once, in 16-bit heads with text positions
        _case("append4_prompt", "append4", B=2, T=8192, lo=8192, hi=8192, rot=128),
        # one user, one token, a short context: the smallest call, where latency is all
        _case("paged4_one", "paged4", page=16, lo=1000, hi=1000),
        # one user, one token, a context of 128 k tokens
        _case("paged4_long", "paged4", lo=131072, hi=131072),
        # a decoding step of a batch of very different lengths, a free slot (length 0) among them
        _case("paged4_step", "paged4", B=64, lo=0, hi=8191),
        # the last 1024 tokens of a prompt that is read in pieces
        _case("paged4_chunk", "paged4", T=1024, lo=16384, hi=16384),
        # requests end and others take their places: pages freed and taken, no data moved
        _case("pages_admit", "admit", B=256, T=8, Hkv=1, D=64, page=16, lo=1, hi=4096, spare=2000),
        # a step of a beam search: half of the rows dropped, the others forked
        _case("pages_beam", "beam", dtype="f16", B=128, T=64, lo=1, hi=1024, spare=100),
        # a pool with holes, made dense again
        _case("pages_compact", "compact", B=96, page=16, lo=1, hi=3600, spare=5000),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    ops = ("rotary", "append", "append4", "paged4", "admit", "beam", "compact")
    limit = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ops}
    limit["append"] = limit["append4"]
    while True:
        op = rng.choice(ops)
        Hkv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8])
        D = rng.choice([40, 64, 64, 80, 96, 128, 128, 128, 256])
        hi = _log(rng, 16, 32768)
        case = {**_BASE, "op": op, "dtype": rng.choice(["bf16", "f16"]), "B": _log(rng, 1, 256), "Hq": Hkv * group,
                "Hkv": Hkv, "D": D, "page": rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256]),
                "lo": rng.choice([0, 1, hi // 2, hi]), "hi": hi}
        if op == "paged4":
            case["T"] = min(hi, rng.choice([1, 1, 1, 2, 5, 8, _log(rng, 16, 1024)]))
        elif op in ("rotary", "append", "append4"):
            case["T"] = rng.choice([1, min(hi, _log(rng, 2, 8192))]) if op != "rotary" else _log(rng, 1, 40000)
            case["rot"] = rng.choice([D, D // 2 // 2 * 2])
            case["interleaved"] = rng.choice([False, True])
            case["axes"] = rng.choice([1, 2, 3, 4]) if op != "append4" else rng.choice([1, 1, 3])
        else:
            case["B"] = max(2, case["B"])
            case["T"] = rng.randint(1, case["B"] - 1)
            case["lo"] = max(1, case["lo"])
            case["spare"] = _log(rng, case["T"], 20000)
        values = case["B"] * case["T"] * (case["Hq"] + 2 * Hkv) * D
        pool = case["Hkv"] * D * (sum(_lengths(case)) + case["spare"] * case["page"])
        scores = case["B"] * case["Hq"] * case["T"] * hi if op == "paged4" else 0
        padded = case["B"] * case["Hkv"] * hi * D if op == "paged4" else 0
        if _cost(case) <= limit[op] and max(values, pool if op != "rotary" else 0, scores, padded) <= 1 << 29:
            return case


def _lengths(case):
    """The lengths of the batch's sequences: fixed by the case, spread over [lo, hi]."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    if B == 1:
        return [hi]
    return [lo + int((b * _GOLDEN) % 1.0 * (hi - lo + 1)) for b in range(B)]


def _cost(case):
    """About the seconds of a pass, by what the work alone costs."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.8e15)


def _row4(D):
    """Bytes of a row of D elements in 4 bits, scales included: the padding is not work."""
    return D / 2 + math.ceil(D / 16)


def work(case):
    op, B, T, Hq, Hkv, D, page = (case[k] for k in ("op", "B", "T", "Hq", "Hkv", "D", "page"))
    lens = _lengths(case)
    if op == "rotary":
        # forward and backward: every value is read once and written once; a pair costs 6 operations
        return {"bytes": 8 * B * T * (Hq + Hkv) * D, "flops": 6 * B * T * (Hq + Hkv) * case["rot"]}
    tokens = sum(min(T, n) for n in lens)
    if op == "append":
        return {"bytes": 4 * tokens * (Hq + 2 * Hkv) * D, "flops": 3 * tokens * (Hq + Hkv) * case["rot"]}
    if op == "append4":
        # q is read and written, k and v read and written in 4 bits, and these read back into 16
        return {"bytes": tokens * (4 * Hq * D + 2 * Hkv * (2 * D + 2 * _row4(D) + 2 * D)),
                "flops": 3 * tokens * (Hq + Hkv) * case["rot"]}
    if op == "paged4":
        # a query of the last T tokens sees the keys up to its own position
        seen = sum(min(T, n) * n - min(T, n) * (min(T, n) - 1) // 2 for n in lens)
        return {"bytes": 4 * B * Hq * T * D + 4 * B * Hq * T + 2 * Hkv * _row4(D) * sum(lens), "flops": 4 * Hq * D * seen}
    # counts of all pages, and the entries that change
    moved = [_pages(n, page) for n in lens]
    pool = sum(moved) + case["spare"]
    if op == "admit":
        return {"bytes": 4 * pool + 16 * sum(moved[:T]), "flops": 0}
    data = 4 * Hkv * page * D                          # of a page's keys and values, read or written
    if op == "beam":
        tails = [lens[i % (B - T)] % page > 0 for i in range(T)]
        return {"bytes": 4 * pool + 16 * sum(moved[i % (B - T)] for i in range(T)) + 2 * data * sum(tails), "flops": 0}
    # about the share of the live pages that lie behind as many as there are live ones
    return {"bytes": 8 * pool + 8 * sum(moved) + 2 * data * sum(moved) * case["spare"] / pool, "flops": 0}


def _pages(n, page):
    return -(-n // page)


def _padded(D):
    return 64 if D <= 64 else 128 if D <= 128 else 256


# ------------------------------------------------------------------ 4-bit rows
def _round_scale(t):
    """To the nearest scale (5 exponent bits, 3 mantissa bits), at most 10240."""
    m, e = torch.frexp(t)
    normal = torch.ldexp(torch.round(m * 16) / 16, e)
    return torch.where(t < 2.0 ** -14, torch.round(t * 2.0 ** 17) * 2.0 ** -17, normal).clamp_max(10240.0)


def _quantise(x):
    """Rows [..., n * 16] in 4 bits: bytes [..., n * 8] (an even element is the lower half) and scales [..., n]."""
    g = x.unflatten(-1, (-1, 16))
    s = _round_scale(g.abs().amax(-1) / 6)
    u = torch.where(s[..., None] > 0, g / s[..., None], 0)
    a = u.abs()
    # halfway goes to the number whose mantissa bit is 0
    c = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
         + (a >= 3.5).byte() + (a > 5).byte())
    c = (c | ((u < 0) & (c > 0)).byte() << 3).flatten(-2)
    return c[..., 0::2] | c[..., 1::2] << 4, (s.half().view(torch.int16) >> 7).byte()


def _decode(data, scales, wide):
    """What rows in 4 bits stand for."""
    of = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=wide, device=data.device)
    u = torch.stack([of[(data & 15).long()], of[(data >> 4).long()]], -1).flatten(-2)
    s = (scales.short() << 7).view(torch.float16).to(wide)
    return (u.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------- inputs
def _positions(case):
    """Positions of each axis, [axes, B, T]: the raster of a video or an image."""
    A, B, T = case["axes"], case["B"], case["T"]
    width = max(1, int(math.sqrt(T / (1 if A < 3 else 20))))
    n = torch.arange(T, device="cuda")
    axes = [n // (width * width) if A >= 3 else n // width, n // width % width if A >= 3 else n % width, n % width, n]
    first = 100 * torch.arange(B, device="cuda")[:, None]
    return torch.stack([a.expand(B, T) + first for a in axes[:A]]).to(torch.int32)


def prepare(case, seed):
    op, B, T, Hq, Hkv, D, page = (case[k] for k in ("op", "B", "T", "Hq", "Hkv", "D", "page"))
    dtype, lens = _TYPES[case["dtype"]], _lengths(case)
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    state = {"case": case}
    half = case["rot"] // 2
    if half:
        state["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    if half and (op != "append4" or case["axes"] > 1):
        state["positions"] = _positions(case)
        # which axis a pair turns by: one after another where there are three, else in sections
        p = torch.arange(half, device="cuda")
        state["pair_axis"] = (p % case["axes"] if case["axes"] == 3 else p * case["axes"] // half).to(torch.int32)
    # the projection's output holds q, k and v of a token side by side
    if op in ("rotary", "append", "append4"):
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        state["q"], state["k"], state["v"] = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], dim=2))
    if op == "rotary":
        state["d_q"], state["d_k"] = normal(B, Hq, T, D), normal(B, Hkv, T, D)
        return state
    if op == "paged4":
        state["q"] = normal(B, T, Hq, D).transpose(1, 2)

    need = [_pages(n, page) for n in lens]
    width = max(1, max(need))
    pool = sum(need) + max(3, case["spare"])           # some pages are free
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    have = torch.tensor(need, device="cuda")
    first = have.cumsum(0) - have
    at = torch.arange(width, device="cuda")
    used = at < have[:, None]
    state["table"] = torch.where(used, order[(first[:, None] + at).clamp_max(pool - 1)], -1)
    state["seq_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    state["spare"] = int(order[-1])

    # the pool is made slice by slice, so that its fp32 draws stay small
    step = max(1, (1 << 26) // (Hkv * page * D))
    if op in ("append4", "paged4"):
        P = _padded(D)
        for x in "kv":
            data = torch.zeros((pool, Hkv, page, P // 2), dtype=torch.uint8, device="cuda")
            scales = torch.zeros((pool, Hkv, page, P // 16), dtype=torch.uint8, device="cuda")
            for i in range(0, pool, step):
                rows = torch.nn.functional.pad(normal(min(step, pool - i), Hkv, page, D).float(), (0, P - D))
                data[i:i + step], scales[i:i + step] = _quantise(rows)
            state[x + "_cache"], state[x + "_scales"] = data, scales
    else:
        for x in "kv":
            c = state[x + "_cache"] = torch.empty((pool, Hkv, page, D), dtype=dtype, device="cuda")
            for i in range(0, pool, step):
                c[i:i + step] = normal(min(step, pool - i), Hkv, page, D)
    if op in ("admit", "beam", "compact"):
        state["refs"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        state["refs"][state["table"][used].long()] = 1
    if op == "admit":
        # the first T requests end; as many of other lengths take their places
        state["rows"] = torch.arange(T, dtype=torch.int32, device="cuda")
        state["tokens"] = torch.where(torch.arange(B, device="cuda") < T, state["seq_len"], 0)
    if op == "beam":
        state["parent"] = (torch.arange(T, device="cuda") % (B - T)).to(torch.int32)
        state["child"] = torch.arange(B - T, B, dtype=torch.int32, device="cuda")
    if op == "compact":
        state["scattered"] = state["table"].clone(), state["refs"].clone()
    if own:
        import exact_tiled_attention_23_gb300 as fa
        # the handle that a serving program keeps beside its cache
        if op in ("append4", "paged4"):
            state["cache"] = fa.PagedKV4(state["k_cache"], state["v_cache"], state["k_scales"], state["v_scales"],
                                         state["table"], state["seq_len"], D=D, dtype=dtype)
        else:
            state["cache"] = fa.PagedKV(state["k_cache"], state["v_cache"], state["table"], state["seq_len"])
    return state


def run(state):
    case = state["case"]
    op = case["op"]
    if op == "compact":
        # a pass makes it dense: the requests that came and went since the last one left these holes
        state["table"].copy_(state["scattered"][0])
        state["refs"].copy_(state["scattered"][1])
    if not own:
        if op in ("rotary", "append", "append4", "paged4"):
            return {"rotary": _rotary, "append": _append, "append4": _append4, "paged4": _attention}[op](state, torch.float32)
        return {"admit": _admit, "beam": _beam, "compact": _compact}[op](state)
    import exact_tiled_attention_23_gb300 as fa
    if op == "rotary":
        q, k = state["q"].detach().requires_grad_(), state["k"].detach().requires_grad_()
        turned = fa.rotary(q, state["inv_freq"], state["positions"], k=k, pair_axis=state["pair_axis"],
                           interleaved=case["interleaved"])
        return turned[0].detach(), turned[1].detach(), *torch.autograd.grad(turned, (q, k), (state["d_q"], state["d_k"]))
    cache = state["cache"]
    if op in ("append", "append4"):
        q = fa.kv_append(cache, state["k"], state["v"], q=state["q"], inv_freq=state.get("inv_freq"),
                         interleaved=case["interleaved"], positions=state.get("positions"), pair_axis=state.get("pair_axis"))
        return (q, state["k_cache"], state["v_cache"]) if op == "append" else (q, *fa.kv_read(cache, case["T"]))
    if op == "paged4":
        return fa.forward_paged(state["q"], cache)
    if op == "admit":
        fa.kv_free(cache, state["refs"], state["rows"])
        taken = fa.kv_grow(cache, state["refs"], state["tokens"])
        return taken, state["table"], state["seq_len"], state["refs"]
    if op == "beam":
        fa.kv_free(cache, state["refs"], state["child"])
        taken = fa.kv_fork(cache, state["refs"], state["parent"], state["child"])
        return taken, state["table"], state["seq_len"], state["refs"], state["k_cache"], state["v_cache"]
    moved = fa.kv_compact(cache, state["refs"])
    return moved, state["table"], state["refs"], state["k_cache"], state["v_cache"]


def exact(case, seed):
    global own
    op = case["op"]
    if op in ("admit", "beam", "compact") or op == "paged4" and work(case)["flops"] > 6e11:
        return None
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    if op == "rotary":
        pos = state["positions"].double()
        return tuple(_exact_turn(state, x, pos, back) for back, names in ((False, ("q", "k")), (True, ("d_q", "d_k")))
                     for x in (state[n] for n in names))
    return _exact_append(state) if op != "paged4" else _exact_attention(state)


# ------------------------------------------------------------ the plain forms
def _turn(case, x, cos, sin):
    """Pairs of x [B, H, T, D] by the angles of cos, sin [B, 1, T, rot / 2]."""
    rot = case["rot"]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _angles(state, text, wide):
    """cos and sin [B, 1, T, rot / 2] of the tokens' positions: the axes', or `text` [B, T]."""
    if not state["case"]["rot"]:
        return None, None
    if "positions" in state:
        pos = state["positions"].double()[state["pair_axis"].long()].permute(1, 2, 0)
    else:
        pos = text.double()[..., None]
    angle = pos * state["inv_freq"].double()                                # far positions need 64 bits
    return angle.cos().to(wide)[:, None], angle.sin().to(wide)[:, None]


def _rotary(state, wide):
    case = state["case"]
    cos, sin = _angles(state, None, wide)
    forward = [_turn(case, state[x].to(wide), cos, sin).to(state[x].dtype) for x in ("q", "k")]
    return (*forward, *(_turn(case, state[x].to(wide), cos, -sin).to(state[x].dtype) for x in ("d_q", "d_k")))


def _slots(state):
    """Index, page and slot of the last T tokens, [B, T], and which exist; a token
    that does not has the place of the sequence's first one, or of a spare page."""
    case = state["case"]
    T, page = case["T"], case["page"]
    t = torch.arange(T, device="cuda")
    pos = state["seq_len"].long()[:, None] - T + t
    live = pos >= 0
    which = torch.where(live, t, torch.where(live, t, T).amin(dim=1, keepdim=True).clamp_max(T - 1))
    at = pos.gather(1, which).clamp_min(0)
    some = live.any(dim=1, keepdim=True)
    pages = torch.where(some, state["table"].long().gather(1, at // page), state["spare"])
    return pos, pages, at % page, which, live


def _put(state, name, rows, slots):
    """Rows [B, Hkv, T, n] of the tokens into a pool."""
    _, pages, slot, which, live = slots
    B = torch.arange(rows.shape[0], device="cuda")[:, None]
    some = live.any(dim=1)[:, None, None, None]
    pool = state[name]
    pool[pages, :, slot] = torch.where(some, rows.transpose(1, 2)[B, which], pool[pages, :, slot])


def _append(state, wide):
    """Rotate k and q by their positions and put k, v into the sequences' pages."""
    case, slots = state["case"], _slots(state)
    live = slots[4][:, None, :, None]
    cos, sin = _angles(state, slots[0], wide)
    q, k = (_turn(case, state[x].to(wide), cos, sin) for x in "qk")
    _put(state, "k_cache", k.to(state["k"].dtype), slots)
    _put(state, "v_cache", state["v"], slots)
    return torch.where(live, q, 0).to(state["q"].dtype), state["k_cache"], state["v_cache"]


def _append4(state, wide):
    """The same into a 4-bit cache, and what it holds for these tokens."""
    case, slots, dtype, D = state["case"], _slots(state), state["q"].dtype, state["case"]["D"]
    _, pages, slot, _, live = slots
    live = live[:, None, :, None]
    cos, sin = _angles(state, slots[0], wide)
    q, k = (state[x].to(wide) if cos is None else _turn(case, state[x].to(wide), cos, sin) for x in "qk")
    held = []
    for x, rows in (("k", k), ("v", state["v"].to(wide))):
        data, scales = _quantise(torch.nn.functional.pad(rows, (0, _padded(D) - D)))
        _put(state, x + "_cache", data, slots)
        _put(state, x + "_scales", scales, slots)
        back = _decode(state[x + "_cache"][pages, :, slot], state[x + "_scales"][pages, :, slot], wide)
        held.append(torch.where(live, back.transpose(1, 2)[..., :D], 0).to(dtype))
    return torch.where(live, q, 0).to(dtype), *held


def _attention(state, wide):
    """softmax(q k^T / sqrt(D)) v over the sequence's pages of a 4-bit cache."""
    case = state["case"]
    B, T, Hq, Hkv, D = (case[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q = state["q"].to(wide).reshape(B, Hkv, G * T, D)
    table, n = state["table"].long().clamp_min(0), state["seq_len"].long()

    def rows(x):
        held = [state[x + y][table].transpose(1, 2).flatten(2, 3)[:, :, :case["hi"]] for y in ("_cache", "_scales")]
        return _decode(*held, wide)[..., :D]

    pos = torch.arange(T, device="cuda") + n[:, None] - T                                  # [B, T]
    scores = q @ rows("k").transpose(2, 3) / math.sqrt(D)
    seen = torch.arange(scores.shape[3], device="cuda") <= pos[..., None]                  # [B, T, keys]
    scores = scores.masked_fill(~seen[:, None].expand(B, G, T, -1).reshape(B, 1, G * T, -1), -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    p = (scores - top).exp()
    total, o = p.sum(dim=3, keepdim=True), p @ rows("v")
    o = torch.where(total > 0, o / total, 0).to(state["q"].dtype)
    return o.reshape(B, Hq, T, D), (top + total.log()).reshape(B, Hq, T)


def _give_up(state, rows):
    """The pages of table rows are used once less, and the rows empty."""
    rows = rows.long()
    have = (state["seq_len"][rows].long() + state["case"]["page"] - 1) // state["case"]["page"]
    held = torch.arange(state["table"].shape[1], device="cuda") < have[:, None]
    state["refs"].index_add_(0, state["table"][rows].long().clamp_min(0).flatten(), -held.int().flatten())
    state["table"][rows] = -1
    state["seq_len"][rows] = 0


def _free_pages(refs):
    """Pages in order, the free ones in front."""
    return torch.argsort((refs > 0).byte(), stable=True)


def _admit(state):
    """Rows give up their pages, and sequences grow by their tokens."""
    _give_up(state, state["rows"])
    page, n, table, refs = state["case"]["page"], state["seq_len"].long(), state["table"], state["refs"]
    have, then = (n + page - 1) // page, (n + state["tokens"] + page - 1) // page
    need = then - have
    first = need.cumsum(0) - need
    at = torch.arange(table.shape[1], device="cuda")
    new = (at >= have[:, None]) & (at < then[:, None])
    pages = _free_pages(refs)[(first[:, None] + at - have[:, None]).clamp(0, refs.numel() - 1)]
    refs.index_add_(0, pages.flatten(), new.int().flatten())
    table.copy_(torch.where(new, pages.int(), table))
    state["seq_len"] += state["tokens"]
    return need.int(), table, state["seq_len"], refs


def _beam(state):
    """Rows give up their pages, and others are forked into them: full pages are
    shared, a page that is part full is copied."""
    _give_up(state, state["child"])
    page, table, refs = state["case"]["page"], state["table"], state["refs"]
    parent, child = state["parent"].long(), state["child"].long()
    n = state["seq_len"][parent].long()
    full, part = n // page, n % page > 0
    rank = part.long().cumsum(0) - 1
    new = torch.where(part, _free_pages(refs)[rank.clamp_min(0)], -1)
    rows = table[parent]
    at = torch.arange(table.shape[1], device="cuda")
    shared = at < full[:, None]
    refs.index_add_(0, rows.long().clamp_min(0).flatten(), shared.int().flatten())
    refs.index_add_(0, new.clamp_min(0), part.int())
    # (where nothing is copied, a page onto itself)
    src = rows.gather(1, (_last(n, page)).clamp_min(0)[:, None])[:, 0].long()
    dst = torch.where(part, new, src)
    for x in ("k_cache", "v_cache"):
        state[x][dst] = state[x][src]
    table[child] = torch.where(shared, rows, torch.where((at == full[:, None]) & part[:, None], new[:, None].int(), -1))
    state["seq_len"][child] = n.int()
    return new.int(), table, state["seq_len"], refs, state["k_cache"], state["v_cache"]


def _last(n, page):
    return (n + page - 1) // page - 1


def _compact(state):
    """The live pages from the far end move into the holes in front, both in order."""
    table, refs = state["table"], state["refs"]
    live = refs > 0
    pages = torch.arange(refs.numel(), device="cuda")
    front = pages < live.sum()
    src, dst = torch.nonzero(live & ~front)[:, 0], torch.nonzero(~live & front)[:, 0]
    moved = torch.where(live, pages, -1).int()
    moved[src] = dst.int()
    for x in ("k_cache", "v_cache"):
        state[x][dst] = state[x][src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, moved[table.long().clamp_min(0)], table))
    return moved, table, refs, state["k_cache"], state["v_cache"]


# ------------------------------------------------------------------- 64 bits
def _exact_turn(state, x, pos, back=False):
    """Rotation of x [B, H, T, D] as a product of complex numbers; pos [axes, B, T]."""
    case = state["case"]
    rot = case["rot"]
    x = x.double().clone()
    if not rot:
        return x
    axis = state["pair_axis"].long() if "pair_axis" in state else torch.zeros(rot // 2, dtype=torch.long, device="cuda")
    angle = torch.stack([pos[a] * f for a, f in zip(axis.tolist(), state["inv_freq"].double())], -1)[:, None]
    z = torch.polar(torch.ones_like(angle), -angle if back else angle)
    r = x[..., :rot]
    pairs = r.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    x[..., :rot] = w.flatten(-2) if case["interleaved"] else w.transpose(-1, -2).flatten(-2)
    return x


def _exact_four(x):
    """What rows [..., D] stand for after they were put into 4 bits."""
    D = x.shape[-1]
    g = torch.nn.functional.pad(x, (0, -D % 16)).unflatten(-1, (-1, 16))
    t = g.abs().amax(-1, keepdim=True) / 6
    step = torch.exp2(torch.floor(torch.log2(t.clamp_min(2.0 ** -14))) - 3)     # of the scales around t
    s = torch.round(t / step) * step
    u = g / s.clamp_min(2.0 ** -17)
    # 0 to 2 in halves, to 4 in ones, to 6 in twos
    a = u.abs()
    to = torch.where(a <= 2, torch.round(a * 2) / 2, torch.where(a <= 4, torch.round(a), torch.round(a / 2).clamp_max(3) * 2))
    return torch.where(s > 0, to * u.sign() * s, 0).flatten(-2)[..., :D]


def _exact_append(state):
    case = state["case"]
    T, page = case["T"], case["page"]
    n = state["seq_len"].long()
    pos = n[:, None] - T + torch.arange(T, device="cuda")
    at = state["positions"].double() if "positions" in state else pos.double()[None]
    live = (pos >= 0)[:, None, :, None]
    q, k, v = torch.where(live, _exact_turn(state, state["q"], at), 0), _exact_turn(state, state["k"], at), state["v"].double()
    if case["op"] == "append4":
        return q, torch.where(live, _exact_four(k), 0), torch.where(live, _exact_four(v), 0)
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()
    for b, length in enumerate(_lengths(case)):
        t = min(T, length)
        if t:
            p = torch.arange(length - t, length, device="cuda")
            pages = state["table"][b].long()[p // page]
            k_cache[pages, :, p % page] = k[b, :, T - t:].transpose(0, 1)
            v_cache[pages, :, p % page] = v[b, :, T - t:].transpose(0, 1)
    return q, k_cache, v_cache


def _exact_attention(state):
    """One sequence and one key head at a time, over exactly the keys it has."""
    case = state["case"]
    B, T, Hq, Hkv, D, page = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    o = torch.zeros((B, Hq, T, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device="cuda")

    def rows(x, pages, h, n):
        data, scales = (state[x + y][pages, h].flatten(0, 1)[:n] for y in ("_cache", "_scales"))
        code = torch.stack([data % 16, data // 16], -1).flatten(-2).double()
        e, m = torch.floor(code % 8 / 2), code % 2
        u = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2)) * torch.where(code >= 8, -1, 1)
        big = scales.double()
        e, m = torch.floor(big / 8), big % 8
        s = torch.where(e == 0, m * 2.0 ** -17, torch.exp2(e - 15) * (1 + m / 8))
        return (u.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)[:, :D]

    for b, n in enumerate(_lengths(case)):
        t = min(T, n)
        if t == 0:
            continue
        pages = state["table"][b].long()[:_pages(n, page)]
        for h in range(Hkv):
            k, v = rows("k", pages, h, n), rows("v", pages, h, n)
            s = state["q"][b, h * G:(h + 1) * G, T - t:].double() @ k.T / math.sqrt(D)      # [G, t, keys]
            ends = torch.arange(n - t, n, device="cuda")
            s = s.masked_fill(torch.arange(n, device="cuda") > ends[:, None], -math.inf)
            lse[b, h * G:(h + 1) * G, T - t:] = s.logsumexp(dim=2)
            o[b, h * G:(h + 1) * G, T - t:] = s.softmax(dim=2) @ v
    return o, lse
