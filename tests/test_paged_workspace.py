"""The workspace of the paged forward: what it grows with, on the host."""
import pytest

import exact_tiled_attention_23_gb300 as fa
from test_paged_abi import cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    fa.build()
    return fa.load()


def pool(keys, Hkv, D, page=64):
    return cache(num_pages=1 << 20, page_size=page, Hkv=Hkv, D=D, stride_slot=D, stride_head=page * D,
                 stride_page=Hkv * page * D, table_width=-(-keys // page), table_stride=-(-keys // page))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page", [(16, 4096, 32, 32, 128, 64), (1, 16384, 32, 8, 128, 64), (64, 4096, 32, 8, 64, 16),
                                               (4, 4096, 32, 8, 256, 64), (8, 4096, 32, 8, 128, 100), (8192, 1, 32, 8, 128, 64)])
def test_many_tiles_need_no_slot_each(B, T, Hq, Hkv, D, page):
    """Without a prefix only a tile that a piece's border cuts leaves a state: two
    a piece at most.  148 to 160 SMs of up to 12 pieces of 8 rows, 8 of 32 rows or
    one of 128, and 8 bytes for a tile."""
    need = fa.fa_fwd_paged_workspace_bytes(pool(max(T, 4096), Hkv, D, page), B, Hq, T)
    tiles = B * Hkv * -(-(Hq // Hkv * T) // 8)
    assert 0 < need <= 2 * 160 * 256 * (D + 1) * 4 + 8 * tiles + 1024


def test_few_tiles_need_one_state_a_piece():
    one = fa.fa_fwd_paged_workspace_bytes(pool(131072, 8, 128), 1, 32, 1)
    assert 0 < one <= (160 * 12 + 8) * 4 * 129 * 4 + 1024
    # behind a prefix every tile leaves a state for the merge
    assert fa.fa_fwd_shared_prefix_workspace_bytes(pool(4096, 8, 128), 1000, 64, 32, 1) > 64 * 8 * 4 * 129 * 4


def test_slots_of_cut_tiles_are_their_own():
    """Two slots a piece: where the kernels put a tile's states, where the merge
    looks for them, and that no two tiles share one (a model of Partials in
    csrc/fa_paged.h)."""
    import random

    from test_paged_line import cut_line
    rng = random.Random(7)
    for _ in range(600):
        tiles = [rng.choice([0, 1, rng.randint(0, 30)]) for _ in range(rng.randint(1, 60))]
        if not sum(tiles):
            continue
        cut = rng.randint(1, 24)
        pieces, records = cut_line(tiles, cut, rng.choice([1, 5]))
        taken = {}
        for piece, mine in enumerate(pieces):
            for i in {i for i, _ in mine}:
                chunks = [c for j, c in mine if j == i]
                if len(chunks) == tiles[i]:
                    assert records[i][1] == 1                      # written directly
                    continue
                slot = 2 * piece + (0 if chunks[0] > 0 else 1)
                assert slot not in taken and slot < 2 * cut
                taken[slot] = i
        for i, (first, count) in records.items():
            if count > 1:
                slots = [2 * first + 2 * n + (1 if n == 0 else 0) for n in range(count)]
                assert [taken.pop(x) for x in slots] == [i] * count
                assert count <= (2 * cut - 2 * first) >> 1         # what the merge clamps a count to
        assert not taken
