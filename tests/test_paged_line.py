"""Model of how the paged kernels cut their line of chunks into pieces
(csrc/fa_paged_line.cuh), in plain Python: every chunk is in exactly one piece,
what a piece copies is what it computes, and a tile's record names exactly the
pieces that leave a state of it."""
import random

import pytest


def cut_line(tiles, cut, heavy):
    """tiles: chunks of each, in the line's order.  Returns the pieces' chunks
    and the records {tile: (first piece, count)}."""
    chunks, filled = sum(tiles), sum(n > 0 for n in tiles)
    weight = heavy if chunks // cut >= 2 * heavy else 0

    def span(n):
        return n + weight if n else 0

    def start_of(c):
        return c + weight if c else 0

    def following(i):
        i += 1
        while i < len(tiles) and not tiles[i]:
            i += 1
        return i

    starts = [sum(map(span, tiles[:i])) for i in range(len(tiles))]
    total = chunks + filled * weight
    per = -(-total // cut)
    pieces, records = [[] for _ in range(cut)], {}
    for piece in range(cut):
        start = per * piece
        if start >= total:
            continue
        size = min(per, total - start)
        i = max(j for j in range(len(tiles)) if tiles[j] and starts[j] <= start)
        x = start - starts[i]
        c = 0 if x == 0 else max(1, x - weight)
        if c < tiles[i]:
            before = start_of(c) - x
        else:
            before = span(tiles[i]) - x
            i, c = following(i), 0
            if i == len(tiles):
                continue
        units = max(0, size - before)
        # what is copied, one chunk at a time
        copied, left, li, lc = [], units, i, c
        while left > 0:
            copied.append((li, lc))
            left -= 1 if lc else 1 + weight
            lc += 1
            if lc == tiles[li]:
                li, lc = following(li), 0
                if li == len(tiles):
                    assert left <= 0
                    break
        # what is computed, tile by tile
        used, end = before, before + units
        while used < end:
            within = end - used if c else max(1, end - used - weight)
            count = min(tiles[i] - c, within)
            if c == 0:
                records[i] = (piece, (used + start_of(tiles[i] - 1)) // per + 1)
            pieces[piece] += [(i, c + k) for k in range(count)]
            used += start_of(c + count) - start_of(c)
            c += count
            if c == tiles[i]:
                i, c = following(i), 0
                if i == len(tiles):
                    break
        assert pieces[piece] == copied
    return pieces, records


@pytest.mark.parametrize("heavy", [1, 5])
@pytest.mark.parametrize("longest", [1, 3, 40])
def test_every_chunk_is_in_one_piece(heavy, longest):
    rng = random.Random(heavy * 100 + longest)
    for _ in range(400):
        tiles = [rng.choice([0, 1, rng.randint(0, longest)]) for _ in range(rng.randint(1, 30))]
        if not sum(tiles):
            continue
        pieces, records = cut_line(tiles, rng.randint(1, 24), heavy)
        owner = {}
        for piece, mine in enumerate(pieces):
            for chunk in mine:
                assert chunk not in owner
                owner[chunk] = piece
        assert len(owner) == sum(tiles)
        for i, n in enumerate(tiles):
            states = sorted({owner[i, c] for c in range(n)})
            assert states == (list(range(records[i][0], sum(records[i]))) if n else [])


def test_equal_pieces():
    """Tiles of one chunk cost two, so that a piece of them has half as many."""
    pieces, _ = cut_line([64] * 4 + [1] * 128, 8, 1)
    assert max(map(len, pieces)) <= 65 and max(len({t for t, _ in p}) for p in pieces) <= 33
