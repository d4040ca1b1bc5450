"""How exact the weights of the paged forward are.

The row kernel (up to 32 stacked rows, alone or as a team) and the tensor-core
kernel over the prefix of such rows multiply V by each weight as two 16-bit
numbers, p = hi + lo.  The bounds here count that, and not
the single rounding of a weight that tests/paged_reference.py allows every
kernel: a kernel without its second product does not keep them (which a model
on the CPU shows first).
"""
import math

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference as ref
from test_paged_gpu import BF16, F16, Pool

# fp16: a row's largest weight is at least 2^LIFT in the row kernel's units, and
# 2^LIFT_TILES in the tensor-core kernel's
LIFT, LIFT_TILES = 12, 7


def bound_of(want, keys, dtype, lift=LIFT):
    """|O - exact| with weights of two numbers.

    A weight is off by e as in check_attention().  hi is off by half a step u of
    p, and lo by half a step of that: u^2.  fp16 numbers below the normal range
    are off by 2^-25 instead, 2^-(25 + lift) of the row's largest weight.  One
    accumulator takes keys / 16 products of hi and as many of lo, each a sum of
    17 terms that are off by 2^-24 of the sum of magnitudes; the sum of weights
    is off by keys 2^-24.  The result is rounded once, half a step of itself."""
    o, _, a, size, vmax = want
    u = ref.HALF_STEP[dtype]
    e = (o.shape[3] + 4) * 2.0 ** -24 * size + 2.0 ** -20
    c = (2 * -(-keys // 16) * 17 + keys) * 2.0 ** -24
    tiny = keys * 2.0 ** -(25 + lift) * vmax + 2.0 ** -25 if dtype == F16 else 0 * vmax
    return u * o.abs() + 1.01 * ((2 * e[..., None] + u * u + c) * a + tiny[..., None])


def modelled(q, pool, dtype, second):
    """O of a pool's sequences with weights of one or two 16-bit numbers, the rest in 64 bits."""
    out = torch.zeros(q.shape, dtype=torch.float64)
    G = q.shape[1] // pool.Hkv
    for b, n in enumerate(pool.lens.tolist()):
        for hq in range(q.shape[1]):
            k, _ = ref.key_rows(pool.k, pool.table[b], n, pool.page, pool.k.shape[0], hq // G)
            v, _ = ref.key_rows(pool.v, pool.table[b], n, pool.page, pool.k.shape[0], hq // G)
            s = k @ q[b, hq, 0].double() / math.sqrt(q.shape[3])
            p = torch.exp(s - s.max()) * (2.0 ** LIFT if dtype == F16 else 1.0)
            hi = p.to(dtype).double()
            lo = (p - hi).to(dtype).double() if second else 0 * p
            out[b, hq, 0] = (hi + lo) @ v / p.sum()
    return out.to(dtype).double()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_bound_tells_one_number_from_two(dtype):
    pool = Pool([20, 33], 2, 64, 16, dtype, seed=3)
    q = pool.queries(8, 1)
    want = ref.attention(q, pool.k, pool.v, pool.table, pool.lens)
    bound = bound_of(want, 33, dtype)
    assert ((modelled(q, pool, dtype, True) - want[0]).abs() <= bound).all()
    assert not ((modelled(q, pool, dtype, False) - want[0]).abs() <= bound).all()


ROWS = [
    # lens, Hkv, group, T, D, page, width (None: as narrow as it can be), prefix
    ([20, 33], 2, 4, 1, 64, 16, None, 0),
    ([20, 33], 2, 4, 1, 128, 16, 2000, 0),
    ([130, 7, 64], 1, 8, 1, 128, 8, 2000, 0),
    ([50, 9], 1, 5, 1, 96, 7, None, 0),
    ([50, 9], 1, 5, 1, 96, 7, 3000, 0),
    ([40, 18], 2, 4, 4, 64, 16, None, 0),
    ([40, 18], 1, 4, 3, 128, 12, None, 0),
    ([60, 33], 1, 4, 8, 128, 16, None, 0),
    ([60, 33], 1, 8, 3, 64, 100, None, 0),
    ([30, 41], 1, 4, 2, 256, 16, None, 0),
    ([30, 41], 1, 4, 9, 256, 16, None, 0),
    ([12, 30], 2, 4, 1, 64, 16, None, 21),
    ([12, 30], 1, 4, 2, 128, 16, 2000, 37),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,Hkv,group,T,D,page,width,prefix", ROWS)
def test_rows_keep_two_numbers_of_a_weight(lens, Hkv, group, T, D, page, width, prefix, dtype):
    pool = Pool(lens, Hkv, D, page, dtype, seed=D + T + page, prefix=prefix, width=width)
    q = pool.queries(Hkv * group, T)
    fa.build()
    cache = pool.gpu()
    o, _ = (fa.forward_shared_prefix(q.cuda(), cache, pool.prefix_table.cuda(), prefix) if prefix
            else fa.forward_paged(q.cuda(), cache))
    want = ref.attention(q, pool.k, pool.v, pool.table, pool.lens, prefix_table=pool.prefix_table, prefix_len=prefix)
    over = (o.double().cpu() - want[0]).abs() - bound_of(want, prefix + max(lens), dtype)
    assert (over <= 0).all(), over.max()


# Prefixes that the tensor cores read: more than 32 rows of all sequences together,
# up to 32 of each.
STACKED = [
    # prefix, lens, Hkv, group, T, D, page
    (40, [5, 30, 1, 0, 17, 9, 22, 3, 40], 1, 4, 1, 64, 16),
    (130, [12] * 6, 1, 8, 1, 128, 16),
    (17, [20, 1, 3], 2, 4, 3, 96, 8),
    (64, [33, 2], 1, 4, 8, 128, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("prefix,lens,Hkv,group,T,D,page", STACKED)
def test_a_prefix_is_as_exact_as_the_own_keys(prefix, lens, Hkv, group, T, D, page, dtype):
    pool = Pool(lens, Hkv, D, page, dtype, seed=D + T + prefix, prefix=prefix, width=20000 // page)
    q = pool.queries(Hkv * group, T)
    fa.build()
    o, _ = fa.forward_shared_prefix(q.cuda(), pool.gpu(), pool.prefix_table.cuda(), prefix)
    want = ref.attention(q, pool.k, pool.v, pool.table, pool.lens, prefix_table=pool.prefix_table, prefix_len=prefix)
    over = (o.double().cpu() - want[0]).abs() - bound_of(want, prefix + max(lens), dtype, LIFT_TILES)
    assert (over <= 0).all(), over.max()
