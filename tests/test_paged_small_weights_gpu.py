"""Rows of which one key has nearly all the weight and a value of 0, so that the
output is made of very many small weights, all alike.  fp16 numbers are multiples
of 2^-24: what a weight loses by that must not be a share of the output."""
import math

import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

# fp16: a row's largest weight is at least 2^LIFT in the row kernel's units, and
# 2^LIFT_TILES in the tensor-core kernel's
LIFT, LIFT_TILES = 12, 7

# sequences, keys of each (all share their pages), how far the first key lies
# above the others in powers of 2, query tokens, D, page
ROWS = [
    (2048, 8192, 20.5, 1, 64, 16),         # a warp has whole sequences
    (2048, 8192, 23.6, 1, 128, 16),
    (1024, 8192, 23.6, 1, 256, 16),
    (1024, 8192, 20.5, 1, 64, 12),
    (1024, 8192, 23.6, 4, 128, 16),        # tiles of 16 rows
    (1024, 8192, 20.5, 3, 256, 16),
    (512, 8192, 20.5, 6, 64, 16),          # tiles of 32 rows
    (512, 8192, 23.6, 8, 128, 16),
    (1, 8192, 20.5, 1, 64, 16),            # a team
    (1, 131072, 26.0, 1, 128, 16),         # one sequence, cut among all warps
]


def check(B, n, gap, T, D, page, dtype, one_number, lift, prefix=False):
    """A weight is off by 2^-20 of itself (the exponent's rounding) and by its
    16-bit form: half a step u, or u^2 as two numbers; in fp16 by 2^-25 against
    a largest weight of 2^lift where that is more.  One accumulator takes at most
    n / 16 products with either number, each a sum of 17 terms that are off by
    2^-24 of the sum, and the sum of weights n terms; the merge joins up to 2048
    states.  O divides two such sums and is rounded once."""
    fa.build()
    group = 4
    k = torch.zeros((-(-n // page), 1, page, D), dtype=dtype)
    v = torch.ones_like(k)
    k[..., 0] = -gap * math.log(2)
    k[0, 0, 0, 0] = 0
    v[0, 0, 0] = 0
    q = torch.zeros((B, group, T, D), dtype=dtype)
    q[..., 0] = 8
    table = torch.arange(k.shape[0], dtype=torch.int32).expand(B, -1).contiguous()
    cache = fa.PagedKV(k.cuda(), v.cuda(), table.cuda(),
                       torch.full((B,), 0 if prefix else n, dtype=torch.int32, device="cuda"))
    scale = 1 / 8                                              # a score is the key's first element
    if prefix:
        o, lse = fa.forward_shared_prefix(q.cuda(), cache, table[0].cuda(), n, causal=False, scale=scale)
    else:
        o, lse = fa.forward_paged(q.cuda(), cache, causal=False, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    tail = (n - 1) * math.exp(float(k[0, 0, 1, 0]))
    want = tail / (1 + tail)
    u = ref.HALF_STEP[dtype]
    mine = min(n, 8192)                                        # keys of one accumulator
    off = 2.0 ** -20 + (u if one_number else u * u) + (2 * mine / 16 * 17 + mine + 2048) * 2.0 ** -24
    bound = want * (u + 2 * off) + (n * 2.0 ** -(25 + lift) + 2.0 ** -25 if dtype == F16 else 0.0)
    worst = (o.double() - want).abs().max().item()
    assert worst <= bound, f"{worst / want:.2e} of O off, {bound / want:.2e} allowed"
    assert (lse.double() - math.log1p(tail)).abs().max() <= off + 2.0 ** -20


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,n,gap,T,D,page", ROWS)
def test_rows_keep_small_weights(B, n, gap, T, D, page, dtype):
    check(B, n, gap, T, D, page, dtype, False, LIFT)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,n,gap,T,D,page", [
    (256, 8192, 20.5, 40, 64, 16),         # a CTA has whole tiles
    (256, 8192, 23.6, 40, 128, 16),
    (128, 8192, 23.6, 32, 96, 64),
    (1, 131072, 24.4, 40, 128, 16),        # a tile is cut among all CTAs
])
def test_tiles_keep_small_weights(B, n, gap, T, D, page, dtype):
    check(B, n, gap, T, D, page, dtype, True, LIFT_TILES)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,n,gap,T,D,page", [(8192, 8192, 20.5, 1, 64, 16), (4096, 8192, 23.6, 2, 128, 16)])
def test_a_prefix_keeps_small_weights(B, n, gap, T, D, page, dtype):
    """All keys are the prefix's, which the tensor cores read with weights of two numbers."""
    check(B, n, gap, T, D, page, dtype, False, LIFT_TILES, prefix=True)
