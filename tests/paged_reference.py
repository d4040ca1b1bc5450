"""Plain 64-bit implementations of the paged-cache operators for the tests:
one sequence, head and query at a time, over exactly the keys it sees.  They
share nothing with the CUDA path."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def lengths(seq_len, width, page):
    return [max(0, min(int(n), width * page)) for n in seq_len]


def key_rows(cache, table, n, page, num_pages, h):
    """([n, D] values, [n] whether the key's page exists) of one sequence and key head."""
    rows, ok = [], []
    for i in range(n):
        p = int(table[i // page])
        ok.append(0 <= p < num_pages)
        rows.append(cache[p if ok[-1] else 0, h, i % page].double())
    if not rows:
        return cache.new_zeros((0, cache.shape[3]), dtype=torch.float64), torch.zeros(0, dtype=torch.bool)
    return torch.stack(rows), torch.tensor(ok)


def attention(q, k_cache, v_cache, table, seq_len, causal=True, scale=None, prefix_table=None, prefix_len=0):
    """O, LSE in 64 bits and, for the tolerances, A = sum p |v| / sum p, the
    largest sum |q k| scale of a visible key, and the largest visible |v|.
    All arguments on the CPU."""
    B, Hq, T, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G, scale = Hq // Hkv, 1 / math.sqrt(D) if scale is None else scale
    o = torch.zeros(q.shape, dtype=torch.float64)
    a = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    size = torch.zeros((B, Hq, T), dtype=torch.float64)
    vmax = torch.zeros((B, Hq, T), dtype=torch.float64)
    for h in range(Hkv):
        kp, okp = key_rows(k_cache, [] if prefix_table is None else prefix_table, prefix_len, page, pages, h)
        vp, _ = key_rows(v_cache, [] if prefix_table is None else prefix_table, prefix_len, page, pages, h)
        for b, n in enumerate(lengths(seq_len, table.shape[1], page)):
            ko, oko = key_rows(k_cache, table[b], n, page, pages, h)
            vo, _ = key_rows(v_cache, table[b], n, page, pages, h)
            k, v, ok = torch.cat([kp, ko]), torch.cat([vp, vo]), torch.cat([okp, oko])
            for t in range(T):
                own = n - T + t + 1 if causal else n
                if causal and own <= 0:
                    continue
                seen = ok.clone()
                seen[prefix_len + own:] = False
                if not bool(seen.any()):
                    continue
                ks, vs = k[seen], v[seen]
                for hq in range(h * G, (h + 1) * G):
                    x = q[b, hq, t].double()
                    s = ks @ x * scale
                    p = torch.softmax(s, dim=0)
                    o[b, hq, t], a[b, hq, t] = p @ vs, p @ vs.abs()
                    lse[b, hq, t] = torch.logsumexp(s, dim=0)
                    size[b, hq, t] = (ks.abs() @ x.abs()).max() * scale
                    vmax[b, hq, t] = vs.abs().max()
    return o, lse, a, size, vmax


def check_attention(got_o, got_lse, ref, keys, dtype):
    """Compare with `attention()`'s answer.

    A score is a sum of D products in fp32: off by at most (D + 4) 2^-24
    sum |q k| scale, and by 2^-21 of an exponent of up to 2^6 in the base-2
    form, so every weight is off by e = that + 2^-20 relative.  A weight that
    multiplies V as one 16-bit number is off by half a step u, and the sum it
    is divided by as well: |dO| <= 2 (e + u) A.  Weights below fp16's normal
    range are off by 2^-25 of the largest instead, each.  The output is rounded
    once more, half a step of itself.  The LSE is off by e and its own rounding.
    """
    o, lse, a, size, vmax = ref
    D = o.shape[3]
    u = HALF_STEP[dtype]
    e = (D + 4) * 2.0 ** -24 * size + 2.0 ** -20
    tiny = 2.0 ** -25 * keys * vmax + 2.0 ** -25 if dtype == torch.float16 else 0.0 * vmax
    bound = u * o.abs() + 1.01 * (2 * (e + u)[..., None] * a + tiny[..., None])
    got_o, empty = got_o.double().cpu(), torch.isneginf(lse)
    assert got_o.isfinite().all()
    assert (got_o[empty] == 0).all() and not torch.signbit(got_o[empty]).any()
    over = (got_o - o).abs() - bound
    assert (over <= 0).all(), f"O off by {(got_o - o).abs().max():.3e}, {over.max():.3e} over its bound"
    if got_lse is None:
        return
    got_lse = got_lse.double().cpu()
    assert torch.equal(torch.isneginf(got_lse), empty)
    off = (got_lse[~empty] - lse[~empty]).abs()
    assert (off <= e[~empty] + 2.0 ** -22 * (1 + lse[~empty].abs())).all(), f"LSE off by {off.max():.3e}"


def rotated(x, pos, inv_freq, interleaved):
    """[H, T, D] turned by positions [T], in 64 bits."""
    x = x.double().clone()
    half = inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()
    c, s = angle.cos(), angle.sin()
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first].clone(), x[..., second].clone()
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x
