// fa_paged_line.cuh -- the line of key chunks that the paged kernels share out.
//
// A group is one row tile of one sequence (its index is sequence * tiles + row
// tile); each of the Hkv key heads has a tile of the group, with the same
// number of chunks.  The line runs over groups, then key heads, then chunks;
// every CTA takes an equal piece of it, whatever the sequences' lengths.
#pragma once

#include "fa_paged.h"

namespace fa {

__device__ __forceinline__ int keys_of_sequence(const PagedParams &p, int b)
{
    if (!p.c.seq_len) return p.c.fixed_len;
    const int64_t cap = (int64_t)p.c.table_width * p.c.page_size;
    const int n = p.c.seq_len[b];
    return n < 0 ? 0 : (n > cap ? (int)cap : n);
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

template <int kChunk>
struct Line {
    const PagedParams &p;
    int R;         // stacked rows per (sequence, key head)
    int groups;
    bool masked;   // rows see different keys

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

    // This CTA's piece of the line: where it starts, its first chunk counted
    // along the line, how many it has, and how many a full piece has.  The
    // whole CTA calls it; `scratch` holds kThreads / 32 + 2 numbers.  Thread i
    // sums the chunks of a strip of groups, and the strips' prefix sums find the
    // group to start in.  (The host keeps the line below 2^31 chunks.)
    template <int kThreads>
    __device__ __forceinline__ void share(int *scratch, LineCursor &at, int &first, int &count, int &per) const
    {
        constexpr int kWarps = kThreads / 32;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        int total, base = 0;
        at.h = at.c = 0;
        if (groups == 1) {
            enter(at, 0);
            total = at.n * p.c.Hkv;
            per = (int)(((unsigned)total + gridDim.x - 1) / gridDim.x);
        } else {
            const int strip = (groups + kThreads - 1) / kThreads;
            const int g0 = min(tid * strip, groups), g1 = min(g0 + strip, groups);
            int sum = 0;
            LineCursor u;
            for (int g = g0; g < g1; ++g) {
                enter(u, g);
                sum += u.n;
            }
            int scan = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, scan, d);
                if (lane >= d) scan += v;
            }
            if (lane == 31) scratch[warp] = scan;
            __syncthreads();
            int all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) scan += scratch[w];
                all += scratch[w];
            }
            total = all * p.c.Hkv;
            per = (int)(((unsigned)total + gridDim.x - 1) / gridDim.x);
            const unsigned start = (unsigned)per * blockIdx.x;
            if (start < (unsigned)total && (unsigned)((scan - sum) * p.c.Hkv) <= start &&
                start < (unsigned)(scan * p.c.Hkv)) {
                int before = scan - sum;
                int g = g0;
                for (;; ++g) {
                    enter(u, g);
                    if (start < (unsigned)((before + u.n) * p.c.Hkv)) break;
                    before += u.n;
                }
                scratch[kWarps] = g;
                scratch[kWarps + 1] = before * p.c.Hkv;
            }
            __syncthreads();
            if (start < (unsigned)total) {
                enter(at, scratch[kWarps]);
                base = scratch[kWarps + 1];
            }
        }
        const unsigned start = (unsigned)per * blockIdx.x;
        count = start < (unsigned)total ? min(per, total - (int)start) : 0;
        first = (int)start;
        if (count > 0) {
            at.h = (first - base) / at.n;
            at.c = (first - base) - at.h * at.n;
        }
    }

    // The CTA that has the first chunk of a tile says where its states will be.
    __device__ __forceinline__ void record(const LineCursor &u, int first_chunk, int per) const
    {
        const int tile = u.g * p.c.Hkv + u.h;
        const int last = (int)((unsigned)(first_chunk + u.n - 1) / (unsigned)per);
        p.part.tile[tile] = TileSlots{(int)blockIdx.x + tile, last - (int)blockIdx.x + 1};
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
