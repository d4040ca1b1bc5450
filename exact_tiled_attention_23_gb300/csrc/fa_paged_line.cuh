// fa_paged_line.cuh -- the line of key chunks that the paged kernels share out.
//
// A group is one row tile of one sequence (its index is sequence * tiles + row
// tile); each of the Hkv key heads has a tile of the group, with the same
// number of chunks.  The line runs over groups, then key heads, then chunks;
// every CTA (or warp) takes an equal piece of it, whatever the sequences' lengths.
#pragma once

#include "fa_paged.h"

namespace fa {

// seq_len[b] as it counts: within what the table can hold.
__device__ __forceinline__ int clamped_length(const PagedParams &p, int n)
{
    const int64_t cap = (int64_t)p.c.table_width * p.c.page_size;
    return n < 0 ? 0 : (n > cap ? (int)cap : n);
}

__device__ __forceinline__ int keys_of_sequence(const PagedParams &p, int b)
{
    return p.c.seq_len ? clamped_length(p, p.c.seq_len[b]) : p.c.fixed_len;
}

// Keys that at least one row of row tile `rt` sees, of a sequence of `len`.
__device__ __forceinline__ int keys_of_tile(int len, int rt, int rows, int R, FastDiv by_g, int T, bool causal)
{
    if (!causal) return len;
    const int last = min((rt + 1) * rows, R) - 1;
    return max(0, min(len, len - T + by_g.quotient(last) + 1));
}

__device__ __forceinline__ int chunks_of(int keys, int chunk) { return (int)(((int64_t)keys + chunk - 1) / chunk); }

// A place on the line.
struct LineCursor {
    int g, h;      // group, key head
    int c, n;      // chunk, chunks of the tile
    int keys;      // keys that the tile sees
    int len;       // keys of the sequence
};

// Pieces are equal in units: a chunk is one, and where pieces are long a tile's
// first chunk counts kTile more, for what a tile costs beside its keys.  A chunk
// belongs to the piece in which it begins.
template <int kChunk, int kTile>
struct Line {
    const PagedParams &p;
    int R;         // stacked rows per (sequence, key head)
    int groups;
    bool masked;   // rows see different keys
    int weight = 0;                // kTile or 0, set by share()

    __device__ __forceinline__ explicit Line(const PagedParams &q) : p(q)
    {
        R = p.G * p.T * (p.part.stacked ? p.B : 1);
        groups = (p.part.stacked ? 1 : p.B) * p.part.tiles;
        masked = p.causal && !p.part.stacked;
    }

    __device__ __forceinline__ void enter(LineCursor &u, int g) const
    {
        const int b = p.part.tiles == 1 ? g : g / p.part.tiles;
        u.g = g;
        u.len = keys_of_sequence(p, b);
        u.keys = keys_of_tile(u.len, g - b * p.part.tiles, p.part.rows, R, p.by_g, p.T, masked);
        u.n = chunks_of(u.keys, kChunk);
    }

    // To the next chunk; past the line's end n is 0.
    __device__ __forceinline__ void advance(LineCursor &u) const
    {
        if (++u.c < u.n) return;
        u.c = 0;
        if (++u.h < p.c.Hkv) return;
        u.h = 0;
        do {
            if (u.g + 1 >= groups) {
                u.n = 0;
                return;
            }
            enter(u, u.g + 1);
        } while (u.n == 0);
    }

    __device__ __forceinline__ int units_of(int chunks) const { return chunks ? chunks + weight : 0; }
    // Where a tile's chunk c begins.
    __device__ __forceinline__ int start_of(int c) const { return c ? c + weight : 0; }
    // How many chunks from `c` on begin within `units` (> 0) of chunk c's start.
    __device__ __forceinline__ int chunks_within(int c, int units) const { return c ? units : max(1, units - weight); }

    // Chunks of a tile of the groups base + 32 i + lane; their lengths are loaded
    // together.
    static constexpr int kHeld = 2;
    __device__ __forceinline__ void chunks_of_groups(int base, int (&n)[kHeld]) const
    {
        int b[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int g = base + 32 * i + (int)threadIdx.x % 32;
            b[i] = g >= groups ? -1 : p.part.tiles == 1 ? g : g / p.part.tiles;
            n[i] = b[i] >= 0 && p.c.seq_len ? p.c.seq_len[b[i]] : p.c.fixed_len;
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int g = base + 32 * i + (int)threadIdx.x % 32;
            const int len = p.c.seq_len ? clamped_length(p, n[i]) : n[i];
            const int keys = b[i] < 0 ? 0 : keys_of_tile(len, g - b[i] * p.part.tiles, p.part.rows, R, p.by_g, p.T, masked);
            n[i] = chunks_of(keys, kChunk);
        }
    }

    // How many pieces a line is cut into: `most`, or fewer where another kernel
    // works beside.  `own`: its chunks and tiles.  (Whole warps call it, and
    // share().)
    __device__ __forceinline__ int pieces(unsigned own, int most) const
    {
        const Beside &s = p.beside;
        if (!s.on) return most;
        if (p.part.stacked) {
            own = 0;
            for (int b = threadIdx.x % 32; b < s.B; b += 32) {
                const int n = chunks_of(min(max(s.seq_len[b], 0), s.cap), s.chunk);
                own += n ? n + 1 : 0;
            }
            own = __reduce_add_sync(0xffffffffu, own) * s.tiles;
        }
        if (own == 0) return most;
        const int front = beside_front(s, own);
        return min(p.part.stacked ? front : (s.sms - front) * s.per_sm, most);
    }

    // Piece `piece` of the line: its first chunk, how many units there are from
    // that chunk's start to the piece's end (none: no chunk is the piece's), how
    // many before it, and how many in a full piece.  The lanes sum the groups'
    // chunks, 64 groups at a time (256: more code to fetch, 54 us where 64 take 53
    // behind a shared prefix; 32: 256 sequences 53.6 where 64 take 52.7); then
    // the row of 32 groups to start in is found from the rows' sums, and the group
    // from that row's prefix sums.  Every warp does it for itself: no barrier, and
    // little code to fetch.  (The host keeps the line below 2^32 units.)
    __device__ __forceinline__ void share(int piece, int most, LineCursor &at, int &before, int &units, int &per)
    {
        const int lane = threadIdx.x % 32;
        int n[kHeld];
        unsigned chunks = 0, tiles = 0;
#pragma unroll 1
        for (int base = 0; base < groups; base += 32 * kHeld) {
            chunks_of_groups(base, n);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                chunks += n[i];
                tiles += n[i] > 0;
            }
        }
        chunks = __reduce_add_sync(0xffffffffu, chunks) * p.c.Hkv;
        tiles = __reduce_add_sync(0xffffffffu, tiles) * p.c.Hkv;
        const int cut = pieces(chunks + tiles, most);
        // (short pieces: equal in chunks)
        weight = chunks / (unsigned)cut >= 2 * kTile ? kTile : 0;
        const unsigned total = chunks + tiles * weight;
        // (a full piece is longer than kTile, so that a chunk begins in it)
        per = (int)((total + cut - 1) / (unsigned)cut);
        const unsigned start = (unsigned)per * (unsigned)piece;
        before = units = 0;
        if (piece >= cut || start >= total) return;
        const int size = (int)min((unsigned)per, total - start);
        const unsigned target = start / (unsigned)p.c.Hkv;      // of the units of one key head
        unsigned sums = 0;                                       // units of the groups in front
        int here = 0, row = -1;
#pragma unroll 1
        for (int base = 0; base < groups && row < 0; base += 32 * kHeld) {
            if (groups > 32 * kHeld) chunks_of_groups(base, n);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const unsigned all = __reduce_add_sync(0xffffffffu, (unsigned)units_of(n[i]));
                if (row < 0 && target - sums < all) {
                    row = base + 32 * i;
                    here = units_of(n[i]);
                }
                if (row < 0) sums += all;
            }
        }
        // (a second read of lengths that are being changed may find none)
        if (row < 0) return;
        const int mine = here;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, here, d);
            if (lane >= d) here += v;
        }
        const int at_lane = __ffs(__ballot_sync(0xffffffffu, target - sums < (unsigned)here)) - 1;
        sums += __shfl_sync(0xffffffffu, here - mine, at_lane);
        enter(at, row + at_lane);
        if (at.n == 0) return;
        const int span = units_of(at.n), left = (int)(start - sums * p.c.Hkv);
        at.h = min(left / span, p.c.Hkv - 1);
        const int x = min(left - at.h * span, span - 1);
        at.c = x == 0 ? 0 : max(1, x - weight);
        if (at.c < at.n) {
            before = start_of(at.c) - x;
        } else {                                                 // in the tile's last chunk: the next tile
            before = span - x;
            at.c = at.n - 1;
            advance(at);
            if (at.n == 0) return;
        }
        units = max(0, size - before);
    }

    // The piece that has the first chunk of a tile says where its states will be;
    // `before`: units of the piece in front of the tile.
    __device__ __forceinline__ void record(const LineCursor &u, int piece, int before, int per) const
    {
        const int tile = u.g * p.c.Hkv + u.h;
        p.part.tile[tile] = TileSlots{p.part.first_of(piece, tile), (before + start_of(u.n - 1)) / per + 1};
    }
};

// Row `idx` of the stacked rows of a tile's (sequence, key head): its place in
// [B, H, T].
struct RowPlace {
    int b, hq, t;
};

__device__ __forceinline__ RowPlace row_place(const PagedParams &p, int b, int h, int idx)
{
    if (p.part.stacked) {
        b = p.by_gt.quotient(idx);
        idx -= b * (int)p.by_gt.by;
    }
    const int t = p.by_g.quotient(idx);
    return RowPlace{b, h * p.G + idx - t * p.G, t};
}

}  // namespace fa
