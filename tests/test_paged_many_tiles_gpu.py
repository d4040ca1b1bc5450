"""More tiles than pieces of the line: only tiles that a piece's border cuts have
a state, in a workspace of two slots a piece.  Tolerances are those of
tests/paged_reference.py."""
import pytest
import torch

import exact_tiled_attention_23_gb300 as fa
import paged_reference as ref
from test_paged_gpu import BF16, F16, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    fa.build()
    fa.load()


@pytest.mark.parametrize("B,Hkv,group,T,D,page,dtype,long", [
    (200, 1, 1, 33, 64, 8, BF16, 3000),        # tensor-core tiles, one cut into many pieces
    (90, 2, 1, 40, 128, 16, F16, 700),
    (40, 1, 2, 300, 64, 16, BF16, 300),        # several tiles a sequence
    (2000, 1, 1, 1, 64, 8, BF16, 2500),        # tiles of 8, 16 and 32 rows
    (1000, 2, 3, 1, 128, 12, F16, 900),
    (1000, 2, 3, 4, 64, 8, BF16, 700),
    (1300, 1, 4, 5, 64, 100, F16, 300),
    (500, 2, 2, 8, 256, 16, BF16, 300),
])
def test_cut_tiles_among_many(B, Hkv, group, T, D, page, dtype, long):
    lens = [(b * 7) % 5 for b in range(B)]
    lens[B // 3], lens[B // 3 + 1], lens[-1] = long, long // 2, long // 3
    pool = Pool(lens, Hkv, D, page, dtype, seed=B)
    q, cache = pool.queries(Hkv * group, T), pool.gpu()
    need = cache.workspace_bytes(Hkv * group, T)
    rows = B * Hkv * group * T
    assert need < max(rows * D * 4, 2 * 160 * 256 * (D + 1) * 4) + 16 * B * Hkv * T      # not a state for every row
    got = []
    for fill in (0, 255):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        got.append(fa.forward_paged(q.cuda(), cache, workspace=ws[:need]))
        assert (ws[need:] == fill).all()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    # the long sequences and a sample of the others, in 64 bits
    some = sorted({B // 3, B // 3 + 1, B - 1, 0, 1, 2, 3, 4, B // 2, B - 2})
    want = ref.attention(q[some], pool.k, pool.v, pool.table[some], pool.lens[some])
    o, lse = (x.cpu()[some] for x in got[0])
    ref.check_attention(o, lse, want, long, dtype)
    # and the others against the same sequences alone
    for part in range(0, B, 50):
        few = fa.PagedKV(cache.k_cache, cache.v_cache, cache.block_table[part:part + 50], cache.seq_len[part:part + 50])
        o, lse = fa.forward_paged(q[part:part + 50].cuda(), few)
        assert (o.float() - got[0][0][part:part + 50].float()).abs().max() <= 4 * ref.HALF_STEP[dtype] * 5
        a, b = lse, got[0][1][part:part + 50]
        assert torch.equal(torch.isneginf(a), torch.isneginf(b))
        assert (a - b)[~torch.isneginf(a)].abs().max() <= 1e-4
