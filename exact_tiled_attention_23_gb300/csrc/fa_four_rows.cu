// fa_four_rows.cu -- attention of few query rows over a paged cache of 4 bits
// (fa_four.cuh): softmax(scale q k^T) v with k and v decoded on the way to the
// products.
//
// The keys are shared out as in fa_paged_rows.cu: one line of chunks, an equal piece
// of it per warp, partial states joined by the merge.  A tile is 8 or 16 rows, the
// products' columns.
//
// A key and its value are 144 bytes a head at D = 128 where 16 bits take 512, so that
// beside memory the issue slots count: 2 D numbers a key to decode, each pair a
// conversion and a product with its scale.  For that
//   * K: keys are the product's rows and a lane has neighbouring elements of a key,
//     whole words of the cache, as the product's k: any order of k will do, as long
//     as the queries have the same;
//   * V: a product's k is the keys, so that a pair's halves come from two keys.  The
//     halves of bytes of two keys' words are exchanged before they are converted, two
//     operations for 8 numbers; a lane has 2 DP / 16 neighbouring columns of V, and
//     so of O;
//   * decoded numbers are exact in IEEE halves, whatever the queries' type, and so
//     are bf16 queries times a power of two per row (but what lies 2^-39 below the
//     row's largest): all products are of halves, added in fp32;
//   * a weight p is one half, with 11 bits against the 8 of a bf16 output, and for
//     fp16 outputs the sum of two, as in fa_paged_rows.cu.
//
// Measured (D = 128, 8 key heads of 4 queries, bf16): a token of 64 sequences of up to
// 8191 keys, 303 MB, 67 us, 4.5 TB/s (16 bits: 165 us); of one sequence of 131072 keys,
// 151 MB, 38 us (90); of one of 1000, a team per tile, 6.0 us.  4096 keys more a
// sequence take 52 us where their copies alone take 43 and their numbers alone 44: a
// pair of numbers is a conversion (2 clk of an SM's quarter) and a product (2 clk), with
// the products on the tensor cores 21 clk for 8 pairs and 2 products, 340 of the 780
// clk of a step of 32 keys; the rest is the exchange of V's halves, the softmax, shared
// memory and control.  No unit is full: 59 % of the issue slots, 51 % of the integer pipe
// and two thirds of DRAM are used.  12 us are spent before the first and behind the last
// keys.  fp16 queries, with a second product per value, take 73 and 40 us; D = 256, with
// chunks of 16 keys, 161 and 85 (16 bits: 330 and 170), in fp16 171 and 91.  Not kept: a
// step's scores beside the values of the step before (71 us), two accumulators per score
// (68), 16 or 14 warps an SM instead of 12 (68, 74).
#include "fa_four.cuh"
#include "fa_four_rows.h"
#include "fa_paged_line.cuh"
#include "fa_paged_team.cuh"
#include "fa_tc_common.cuh"

#include <atomic>
#include <cmath>

namespace fa {

__device__ uint32_t g_status_four;

namespace {

// Weights are p = 2^(s - m); m is raised where a score lies 2^(kLift + kRise) above
// it, to 2^kLift below the largest one then: halves are multiples of 2^-24, so that a
// weight is off by 2^-37 of the row's largest at most, where not by half a step.
constexpr float kLift = 12.f, kRise = 3.f;

// kTeam: all warps of a cluster work on one tile and join it in shared memory, as in
// fa_paged_rows.cu; else every warp has a piece of the line.
template <int DP, int J, bool kTeam>
struct FourLayout {
    static constexpr int kWarps = kTeam ? kTeamWarps : kRowsWarps;
    static constexpr int kRows = 8 * J;
    static constexpr int kChunk = DP == 256 ? 16 : 32;            // keys of a step
    static constexpr int kRowBytes = DP / 2, kScaleBytes = DP / 16;
    static constexpr int kTileBytes = kChunk * kRowBytes;         // K or V of a step
    static constexpr int kScaleTile = kChunk * kScaleBytes;
    static constexpr int kScales = 2 * kTileBytes;                // where the scales are
    static constexpr int kStageBytes = 2 * kTileBytes + 2 * kScaleTile;
    static constexpr int kStages = DP == 64 ? 4 : 3;
    // what registers and shared memory hold
    static constexpr int kCtas = kTeam ? 1 : J == 2 && DP == 128 ? 4 : J == 2 || DP == 256 ? 5 : DP == 128 ? 6 : 8;
    static constexpr int kMaskOff = kWarps * kStages * kStageBytes;
    static constexpr int kBarOff = kMaskOff + kWarps * kStages * 4;
    static constexpr int kAbortOff = kBarOff + kWarps * kStages * 8;
    // team: (m, l) of every warp's rows, and 24 bytes for each row and four columns
    static constexpr int kStatOff = kAbortOff + kWarps * 4;
    static constexpr int kMailOff = kStatOff + kWarps * kRows * 8;
    static constexpr int kSmemBytes = kTeam ? kMailOff + kRows * DP / 4 * 24 : kStatOff;
    static_assert(kBarOff % 8 == 0 && (!kTeam || kMailOff % 16 == 0), "barriers, states");
    static_assert(!kTeam || (J == 1 && DP <= 128 && kRows * DP * 4 <= kStageBytes), "a team's states fit a stage");
    static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
    static_assert(kStageBytes % 128 == 0 && kTileBytes % 16 == 0 && kScaleTile % 16 == 0, "alignment");
};

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src, bool on)
{
    const uint32_t n = on ? kBytes : 0;             // else zeros
    if constexpr (kBytes == 16)
        ptx::cp_async16(dst, src, n);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}

template <int kWords>
__device__ __forceinline__ void words_of(const uint8_t *at, uint32_t (&w)[kWords])
{
    if constexpr (kWords == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(at);
    } else if constexpr (kWords == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    }
}

__device__ __forceinline__ uint32_t two_bytes(const uint8_t *at) { return *reinterpret_cast<const uint16_t *>(at); }

// A copy of `bytes` (a multiple of 16) between 16-byte boundaries, counted by `bar`.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const uint8_t *src, uint32_t bytes, uint64_t *bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar)), "l"(policy) : "memory");
}

__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t scale)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&scale));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// A chunk's rows are in this order as the products' rows, by eights, so that a
// matrix load's lanes find their banks free: 0 5 1 4 2 7 3 6.
__device__ __forceinline__ int key_of_row(int r) { return r & 1 ? 4 + ((r >> 1) ^ 1) : r >> 1; }

// kBulk: a chunk's rows are one block of each array, which one lane copies.
template <int DP, int J, bool kF16, bool kBulk, bool kTeam>
__global__ void __launch_bounds__((32 * FourLayout<DP, J, kTeam>::kWarps), (FourLayout<DP, J, kTeam>::kCtas))
four_rows_kernel(const FourParams f)
{
    using Lay = FourLayout<DP, J, kTeam>;
    constexpr int S = Lay::kStages, KS = Lay::kChunk, RM = Lay::kRows, KJ = KS / 16;
    constexpr bool kTwo = kF16;                     // weights of two halves
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : 0xffffu;
    constexpr int kUnits = DP == 256 ? 2 : 1;       // of a lane's elements of a key
    constexpr int kWords = DP == 64 ? 2 : 4;        // of a unit
    constexpr int KT = DP / 16;                     // 16-column steps of a score, tiles of O
    constexpr int kVWords = DP / 64;                // of a lane's elements of a value
    extern __shared__ __align__(128) uint8_t smem[];
    const PagedParams &p = f.p;
    const PagedCache4 &c = f.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * S * Lay::kStageBytes;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + Lay::kMaskOff) + warp * S;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff) + warp * S;
    // the warp's own: a warp that gave up a wait stops nobody else
    volatile int *abort_word = reinterpret_cast<int *>(smem + Lay::kAbortOff) + warp;
    const Abort ab{abort_word, &g_status_four};
    if constexpr (kBulk) {
        // (set-up that reads no memory overlaps the end of the kernel before)
        if (lane == 0) {
            for (int i = 0; i < S; ++i) ptx::mbar_init(&full[i], 1);
            *abort_word = 0;
            ptx::fence_mbarrier_init();
        }
        __syncwarp();
    }
    if constexpr (kTeam) ptx::cluster_arrive();
    ptx::wait_for_primary();
    ptx::launch_dependents();
    Line<KS, kRowsTile> line(p);
    const int piece = (int)blockIdx.x * Lay::kWarps + warp;
    LineCursor at;
    int units, used, per;       // of the piece, those in front of `at`, a full piece's (team: chunks)
    if constexpr (kTeam) {
        const int tile = (int)blockIdx.x / p.team, g = tile / p.c.Hkv;
        line.enter(at, g);
        at.h = tile - g * p.c.Hkv;
        const int warps = p.team * Lay::kWarps, mine = ((int)blockIdx.x - tile * p.team) * Lay::kWarps + warp;
        per = (at.n + warps - 1) / warps;
        at.c = min(mine * per, at.n);
        units = min(per, at.n - at.c);
        used = 0;
    } else {
        line.share(piece, (int)gridDim.x * Lay::kWarps, at, used, units, per);
        units += used;
    }
    const int R = line.R;

    // ---- loads -----------------------------------------------------------
    LineCursor ld = at;
    int ld_left = units - used;
    int issued = 0;             // steps copied
    // kBulk: a run is up to 32 steps in one tile.  A lane finds where one of them is and
    // copies it when its turn comes, so that what a step costs beside its numbers is a
    // few instructions (with every lane looking up every step: 71 us where this takes
    // 68, 64 sequences of up to 8191 keys).
    int run = 0, run_at = 0;    // steps of the run, those copied
    int64_t run_off = 0, run_scale = 0;
    uint32_t run_mask = 0;      // keys of this lane's step that are visible
    auto next_run = [&] {
        run = min(min(ld.n - ld.c, kTeam ? ld_left : line.chunks_within(ld.c, ld_left)), 32);
        run_at = 0;
        run_mask = 0;
        if (lane < run) {
            const int key = (ld.c + lane) * KS, which = p.c.by_page.quotient(key);
            const int b = p.part.tiles == 1 ? ld.g : ld.g / p.part.tiles;
            const int slot = key - which * p.c.page_size, keys = ld.keys - key;
            const int page = p.c.table[(int64_t)b * p.c.table_stride + which];
            if (page >= 0 && page < p.c.num_pages) {
                run_mask = keys >= KS ? kAll : (1u << keys) - 1u;
                run_off = page * c.s_page + ld.h * c.s_head + slot * Lay::kRowBytes;
                run_scale = page * c.t_page + ld.h * c.t_head + slot * Lay::kScaleBytes;
            }
        }
        if constexpr (kTeam) {
            ld.c += run;
            ld_left -= run;
        } else {
            ld_left -= line.start_of(ld.c + run) - line.start_of(ld.c);
            ld.c += run - 1;
            line.advance(ld);
        }
        __syncwarp();
    };
    // Else: where this lane's key of a step is (lane % KS).  Its page number is fetched
    // at least one step before its use.
    struct Place {
        int page, slot, h;      // page < 0: not a key that the tile sees
    };
    auto look_up = [&]() -> Place {
        if (kBulk || ld_left <= 0) return Place{-1, 0, 0};
        Place x{-1, 0, ld.h};
        const int key = ld.c * KS + lane % KS;
        if (key < ld.keys) {
            const int which = p.c.by_page.quotient(key);
            const int b = p.part.tiles == 1 ? ld.g : ld.g / p.part.tiles;
            x.slot = key - which * p.c.page_size;
            x.page = p.c.table[(int64_t)b * p.c.table_stride + which];
        }
        if constexpr (kTeam) {
            ++ld.c;
            --ld_left;
        } else {
            ld_left -= ld.c ? 1 : 1 + line.weight;
            line.advance(ld);
        }
        return x;
    };
    const uint64_t policy = kBulk ? ptx::l2_policy(!kTeam && p.part.tiles == 1) : 0;
    Place next = look_up();
    // The next step into `stage` (past the piece, nothing).
    auto load = [&](int stage) {
        const uint32_t dst = ptx::smem_u32(ring) + stage * Lay::kStageBytes;
        if constexpr (kBulk) {
            if (run_at == run) {
                if (ld_left <= 0) return;
                next_run();
            }
            ++issued;
            if (lane == run_at++) {
                s_mask[stage] = run_mask;
                if (run_mask == 0) {
                    ptx::mbar_arrive(&full[stage]);                 // nothing comes
                } else {
                    ptx::mbar_arrive_expect_tx(&full[stage], Lay::kStageBytes);
                    copy_bulk(dst, c.k + run_off, Lay::kTileBytes, &full[stage], policy);
                    copy_bulk(dst + Lay::kTileBytes, c.v + run_off, Lay::kTileBytes, &full[stage], policy);
                    copy_bulk(dst + Lay::kScales, c.ks + run_scale, Lay::kScaleTile, &full[stage], policy);
                    copy_bulk(dst + Lay::kScales + Lay::kScaleTile, c.vs + run_scale, Lay::kScaleTile, &full[stage], policy);
                }
            }
        } else {
            const Place x = next;
            next = look_up();
            const bool ok = x.page >= 0 && x.page < p.c.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAll;
            if (lane == 0) s_mask[stage] = mask;
            constexpr int kLanes = Lay::kRowBytes / 16, kPer = 32 / kLanes;     // lanes per row, rows at a time
            const int unit = lane % kLanes;
            int64_t off = 0, scale = 0;
            if (ok) {
                off = x.page * c.s_page + x.h * c.s_head + x.slot * c.s_slot;
                scale = x.page * c.t_page + x.h * c.t_head + x.slot * c.t_slot;
            }
#pragma unroll
            for (int i = 0; i < KS / kPer; ++i) {
                const int row = i * kPer + lane / kLanes;
                const bool on = (mask >> row) & 1u;
                const int64_t from = __shfl_sync(0xffffffffu, off, row);
                const int64_t o = on ? from + unit * 16 : 0;
                const uint32_t to = dst + row * Lay::kRowBytes + unit * 16;
                copy_async<16>(to, c.k + o, on);
                copy_async<16>(to + Lay::kTileBytes, c.v + o, on);
            }
            if (lane < KS) {
                const uint32_t to = dst + Lay::kScales + lane * Lay::kScaleBytes;
                copy_async<Lay::kScaleBytes>(to, c.ks + scale, ok);
                copy_async<Lay::kScaleBytes>(to + Lay::kScaleTile, c.vs + scale, ok);
            }
            ptx::cp_async_commit();
        }
    };
#pragma unroll 1
    for (int s = 0; s < S; ++s) load(s);

    // ---- the piece, tile by tile -------------------------------------------
    const int qr = lane >> 2, qc = lane & 3;        // this lane's row (and + 8) and columns (2 qc, + 1) of a product
    const int k_row = key_of_row(qr), v_first = key_of_row(2 * qc), v_second = key_of_row(2 * qc + 1);
    int stage = 0;
    uint32_t phase = 0;
    // Waits for a step's keys; returns which of them are visible.  After a wait that
    // gave up (the results are undefined then) the warp computes nothing and, above
    // all, copies nothing more: its stages still have copies in flight.
    bool gave_up = false;
    auto landed = [&]() -> uint32_t {
        if constexpr (kBulk) {
            if (!gave_up)
                gave_up = !__all_sync(0xffffffffu, wait_bounded(&full[stage], phase, p.wait_limit_ns, kSiteSlotFull, ab));
            if (gave_up) return 0u;
        } else {
            ptx::cp_async_wait<S - 1>();
            __syncwarp();
        }
        return s_mask[stage];
    };
    // A block brings what its page holds behind the last key: scales that may be no
    // numbers, whose values have weights of 0.
    auto clear_rest = [&](uint32_t mask, uint8_t *scales) {
        if constexpr (kBulk) {
            if (mask == kAll || gave_up) return;
            if (lane < KS && !((mask >> lane) & 1u))
#pragma unroll
                for (int i = 0; i < Lay::kScaleBytes; i += 4)
                    *reinterpret_cast<uint32_t *>(scales + lane * Lay::kScaleBytes + i) = 0u;
            ptx::fence_proxy_async_smem();          // before the next copy into the stage
            __syncwarp();
        }
    };
    // The step is done: its stage takes the next one (past the piece, nothing).
    auto refill = [&] {
        __syncwarp();
        if (gave_up) return;
        load(stage);
        if (++stage == S) {
            stage = 0;
            phase ^= 1;
        }
    };
    // No copy may still be landing in shared memory at exit.
    auto drain = [&] {
        if constexpr (kBulk) {
            for (int i = max(0, issued - S); i < issued; ++i)
                wait_bounded(&full[i % S], (i / S) & 1, p.wait_limit_ns, kSiteDrain, ab, false);
        } else {
            ptx::cp_async_wait<0>();
        }
    };
#pragma unroll 1
    while (kTeam || used < units) {
        const int rest = units - used;
        const int count = kTeam ? rest : min(at.n - at.c, line.chunks_within(at.c, rest));
        const int b = p.part.tiles == 1 ? at.g : at.g / p.part.tiles;
        const int row0 = (at.g - b * p.part.tiles) * RM, h = at.h;
        const int tile = at.g * p.c.Hkv + h;
        if (!kTeam && at.c == 0 && lane == 0) line.record(at, piece, used, per);
        const int lim_all = line.masked ? at.len - p.T + p.by_g.quotient(row0) + 1 : at.len;   // seen by every row

        // Q: this lane's row 8 n + qr, the elements that it has of a key, as halves
        uint32_t qb[J][KT][2];
        float to_log2[J][2];                        // of the scores of rows 8 n + 2 qc and the next
        int lim[J][2];                              // keys that these rows see
#pragma unroll
        for (int n = 0; n < J; ++n) {
            const int tr = row0 + 8 * n + qr;
#pragma unroll
            for (int k = 0; k < KT; ++k) qb[n][k][0] = qb[n][k][1] = 0u;
            if (tr < R) {
                const RowPlace x = row_place(p, b, h, tr);
                const uint16_t *src = p.q + x.b * p.q_s[0] + x.hq * p.q_s[1] + x.t * p.q_s[2];
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    const int d = (k / 8) * 128 + qc * (DP == 64 ? 16 : 32) + 4 * (k % 8);
                    if (d < p.c.D) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(src + d);
                        qb[n][k][0] = w.x;
                        qb[n][k][1] = w.y;
                    }
                }
            }
            float mine = 1.f;
            if constexpr (!kF16) {
                // times the power of two that takes the row's largest to 2^14 .. 2^15
                float largest = 0.f;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        largest = fmaxf(largest, fabsf(__uint_as_float(qb[n][k][e] << 16)));
                        largest = fmaxf(largest, fabsf(__uint_as_float(qb[n][k][e] & 0xffff0000u)));
                    }
                largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
                largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
                const RowScale scale = row_scale(largest);
                const float by = scale.up;
                mine = scale.down;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qb[n][k][e] = ptx::pack_f16x2(__uint_as_float(qb[n][k][e] << 16) * by,
                                                      __uint_as_float(qb[n][k][e] & 0xffff0000u) * by);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                to_log2[n][r] = p.scale_log2;
                if constexpr (!kF16) to_log2[n][r] *= __shfl_sync(0xffffffffu, mine, 4 * (2 * qc + r));
                lim[n][r] = line.masked ? at.len - p.T + p.by_g.quotient(row0 + 8 * n + 2 * qc + r) + 1 : at.len;
            }
        }
        // o[n][i]: columns qr DP / 8 + 2 i and the next, of rows 8 n + 2 qc and the next
        float o[J][KT][4], m[J][2], l[J][2];
#pragma unroll
        for (int n = 0; n < J; ++n) {
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[n][r] = -INFINITY;
                l[n][r] = 0.f;
            }
        }

        float s[J][KJ][4];                          // scores of keys 16 j + k_row (and + 8) and the rows 2 qc, + 1
        uint32_t hi[J][KJ][2], lo[J][KJ][2];        // weights, of products' lanes
        auto scores = [&](int j, const uint8_t *kt) {
            const uint8_t *const ks = kt + Lay::kScales;
#pragma unroll
            for (int n = 0; n < J; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][j][e] = 0.f;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                uint32_t w[2][kWords], sc[2][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * j + 8 * e + k_row;
                    words_of<kWords>(kt + row * Lay::kRowBytes + u * 64 + qc * (4 * kWords), w[e]);
                    if constexpr (DP == 64) {
                        sc[e][0] = ks[row * Lay::kScaleBytes + qc] * 0x800080u;
                    } else {
                        const uint32_t two = two_bytes(ks + row * Lay::kScaleBytes + u * 8 + 2 * qc);
                        sc[e][0] = (two & 0xffu) * 0x800080u;
                        sc[e][1] = (two >> 8) * 0x800080u;
                    }
                }
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    uint32_t x[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ptx::unpack_e2m1x8(w[e][i], x[e]);
#pragma unroll
                        for (int a = 0; a < 4; ++a) x[e][a] = times(x[e][a], sc[e][DP == 64 ? 0 : i / 2]);
                    }
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const uint32_t ka[4] = {x[0][2 * a], x[1][2 * a], x[0][2 * a + 1], x[1][2 * a + 1]};
#pragma unroll
                        for (int n = 0; n < J; ++n)
                            ptx::mma_16816<true>(s[n][j], ka, qb[n][8 * u + 2 * i + a][0], qb[n][8 * u + 2 * i + a][1]);
                    }
                }
            }
        };
        auto values = [&](int j, const uint8_t *vt) {
            const uint8_t *const vs = vt + (Lay::kScales + Lay::kScaleTile - Lay::kTileBytes);
            // keys 16 j + v_first, + v_second, and 8 further
            uint32_t w[2][2][kVWords], sc[2][2];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = 16 * j + 8 * a + (e ? v_second : v_first);
                    words_of<kVWords>(vt + row * Lay::kRowBytes + qr * (4 * kVWords), w[a][e]);
                    if constexpr (DP == 256)
                        sc[a][e] = two_bytes(vs + row * Lay::kScaleBytes + 2 * qr);
                    else
                        sc[a][e] = vs[row * Lay::kScaleBytes + (DP == 64 ? qr / 2 : qr)];
                }
#pragma unroll
            for (int i = 0; i < kVWords; ++i) {
                uint32_t x[2][2][4];        // [keys][even and odd columns]
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    uint32_t both = 0;      // the two keys' scales
                    if constexpr (DP == 256)
                        both = i < 2 ? (sc[a][0] & 0xffu) * 0x80u + (sc[a][1] & 0xffu) * 0x800000u
                                     : (sc[a][0] >> 8) * 0x80u + (sc[a][1] >> 8) * 0x800000u;
                    else
                        both = sc[a][0] * 0x80u + sc[a][1] * 0x800000u;
                    const uint32_t even = (w[a][0][i] & 0x0f0f0f0fu) | ((w[a][1][i] * 16u) & 0xf0f0f0f0u);
                    const uint32_t odd = ((w[a][0][i] >> 4) & 0x0f0f0f0fu) | (w[a][1][i] & 0xf0f0f0f0u);
                    ptx::unpack_e2m1x8(even, x[a][0]);
                    ptx::unpack_e2m1x8(odd, x[a][1]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        x[a][0][y] = times(x[a][0][y], both);
                        x[a][1][y] = times(x[a][1][y], both);
                    }
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t va[4] = {x[0][0][y], x[0][1][y], x[1][0][y], x[1][1][y]};
#pragma unroll
                    for (int n = 0; n < J; ++n) {
                        ptx::mma_16816<true>(o[n][4 * i + y], va, hi[n][j][0], hi[n][j][1]);
                        if constexpr (kTwo) ptx::mma_16816<true>(o[n][4 * i + y], va, lo[n][j][0], lo[n][j][1]);
                    }
                }
            }
        };
        auto weights = [&](int step, uint32_t mask, uint8_t *vs) {
            const int key0 = (at.c + step) * KS;
            if (mask != kAll || key0 + KS > lim_all) {
                clear_rest(mask, vs);
#pragma unroll
                for (int n = 0; n < J; ++n)
#pragma unroll
                    for (int j = 0; j < KJ; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = 16 * j + 8 * (e >> 1) + k_row;
                            if (!((mask >> key) & 1u) || key0 + key >= lim[n][e & 1]) s[n][j][e] = -INFINITY;
                        }
            }
#pragma unroll
            for (int n = 0; n < J; ++n) {
                float mx[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    mx[r] = fmaxf(s[n][0][r], s[n][0][r + 2]);
#pragma unroll
                    for (int j = 1; j < KJ; ++j) mx[r] = ptx::max3(mx[r], s[n][j][r], s[n][j][r + 2]);
                    mx[r] *= to_log2[n][r];
                }
                if (__any_sync(0xffffffffu, mx[0] > m[n][0] + (kLift + kRise) || mx[1] > m[n][1] + (kLift + kRise))) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], d));
                        const float m_new = fmaxf(m[n][r], mx[r] - kLift);
                        const float alpha = ptx::ex2_approx(m[n][r] - (m_new == -INFINITY ? 0.f : m_new));
                        l[n][r] *= alpha;
#pragma unroll
                        for (int i = 0; i < KT; ++i) {
                            o[n][i][r] *= alpha;
                            o[n][i][r + 2] *= alpha;
                        }
                        m[n][r] = m_new;
                    }
                }
                const float ref0 = m[n][0] == -INFINITY ? 0.f : m[n][0], ref1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
                for (int j = 0; j < KJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = ptx::ex2_approx(fmaf(s[n][j][2 * e], to_log2[n][0], -ref0));
                        const float p1 = ptx::ex2_approx(fmaf(s[n][j][2 * e + 1], to_log2[n][1], -ref1));
                        l[n][0] += p0;
                        l[n][1] += p1;
                        const uint32_t w = ptx::pack_f16x2(p0, p1);
                        // keys of a lane's weights become those of a product's lane
                        hi[n][j][e] = ptx::transpose8(w);
                        if constexpr (kTwo) {
                            float r0, r1;
                            ptx::unpack2(ptx::widen16x2<true>(w), r0, r1);
                            lo[n][j][e] = ptx::transpose8(ptx::pack_f16x2(p0 - r0, p1 - r1));
                        }
                    }
            }
        };
#pragma unroll 1
        for (int step = 0; step < count; ++step) {
            const uint32_t mask = landed();
            uint8_t *const now = ring + stage * Lay::kStageBytes;
            if (mask) {
#pragma unroll
                for (int j = 0; j < KJ; ++j) scores(j, now);
                weights(step, mask, now + Lay::kScales + Lay::kScaleTile);
#pragma unroll
                for (int j = 0; j < KJ; ++j) values(j, now + Lay::kTileBytes);
            }
            refill();
        }

        if constexpr (kTeam) {
            drain();
            __syncwarp();
            // O over the warp's first stage: four columns of all rows after four
            // columns of all rows
            float2 *stat = reinterpret_cast<float2 *>(smem + Lay::kStatOff) + warp * RM;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[0][r];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (qr == 0) stat[2 * qc + r] = make_float2(m[0][r], sum);
#pragma unroll
                for (int i = 0; i < KT / 2; ++i)
                    reinterpret_cast<float4 *>(ring)[(qr * (DP / 32) + i) * RM + 2 * qc + r] =
                        make_float4(o[0][2 * i][r], o[0][2 * i][r + 2], o[0][2 * i + 1][r], o[0][2 * i + 1][r + 2]);
            }
            join_team<DP, kF16>(p, smem, S * Lay::kStageBytes, reinterpret_cast<const float2 *>(smem + Lay::kStatOff),
                                reinterpret_cast<float4 *>(smem + Lay::kMailOff), b, h, at.len);
            return;
        }

        // ---- the tile's state ----
        const bool direct = count == at.n;
        const int64_t slot = p.part.slot_of(piece, tile, at.c > 0);
        const int col0 = qr * (DP / 8);
#pragma unroll
        for (int n = 0; n < J; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[n][r];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const int tr = 8 * n + 2 * qc + r;
                if (row0 + tr >= R) continue;
                // (a NaN among the scores reaches the output)
                const bool empty = sum == 0.f;
                const float inv = empty ? 0.f : 1.f / sum;
                const float lse2 = empty ? -INFINITY : m[n][r] + log2f(sum);
                if (direct) {
                    const RowPlace x = row_place(p, b, h, row0 + tr);
                    uint16_t *dst = p.o + x.b * p.o_s[0] + x.hq * p.o_s[1] + x.t * p.o_s[2] + col0;
#pragma unroll
                    for (int i = 0; i < KT / 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = empty ? 0u : ptx::pack16x2<kF16>(o[n][4 * i + y][r] * inv, o[n][4 * i + y][r + 2] * inv);
                        if (col0 + 8 * i < p.c.D) *reinterpret_cast<uint4 *>(dst + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (p.lse && qr == 0) p.lse[((int64_t)x.b * p.Hq + x.hq) * p.T + x.t] = lse2 * kLn2;
                } else {
                    if (qr == 0) p.part.lse[slot * p.part.slot_rows + tr] = lse2;
#pragma unroll
                    for (int i = 0; i < KT / 2; ++i)
                        if (col0 + 4 * i < p.c.D)
                            *reinterpret_cast<float4 *>(p.part.o + ((slot * (p.c.D / 4) + col0 / 4 + i) * p.part.slot_rows + tr) * 4) =
                                empty ? make_float4(0.f, 0.f, 0.f, 0.f)
                                      : make_float4(o[n][2 * i][r] * inv, o[n][2 * i][r + 2] * inv,
                                                    o[n][2 * i + 1][r] * inv, o[n][2 * i + 1][r + 2] * inv);
                }
            }
        __syncwarp();
        used += line.start_of(at.c + count) - line.start_of(at.c);
        at.c += count - 1;
        line.advance(at);
    }
    drain();
}

template <int DP, int J, bool kF16, bool kBulk, bool kTeam>
cudaError_t launch_one(const FourParams &f, int ctas, cudaStream_t stream)
{
    using Lay = FourLayout<DP, J, kTeam>;
    static SharedMemory allowed;
    const cudaError_t e = allowed.allow(four_rows_kernel<DP, J, kF16, kBulk, kTeam>, Lay::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_clusters(four_rows_kernel<DP, J, kF16, kBulk, kTeam>, kTeam ? f.p.team : 1, dim3((unsigned)ctas),
                           32 * Lay::kWarps, Lay::kSmemBytes, stream, f);
}

// Whether a chunk's rows are one block of each array, on 16-byte boundaries.  (64
// sequences of up to 8191 keys: 67 us, through 16-byte copies 68.5.)
template <int DP>
bool blocks(const PagedCache4 &c)
{
    using Lay = FourLayout<DP, 1, false>;
    return c.page_size % Lay::kChunk == 0 && c.s_slot == Lay::kRowBytes && c.t_slot == Lay::kScaleBytes &&
           (c.t_page % 16 == 0 || c.num_pages == 1) && (c.t_head % 16 == 0 || c.Hkv == 1);
}

template <int DP, int J, bool kTeam>
cudaError_t launch_rows(const FourParams &f, int ctas, cudaStream_t stream)
{
    if (blocks<DP>(f.c))
        return f.p.f16 ? launch_one<DP, J, true, true, kTeam>(f, ctas, stream) : launch_one<DP, J, false, true, kTeam>(f, ctas, stream);
    return f.p.f16 ? launch_one<DP, J, true, false, kTeam>(f, ctas, stream) : launch_one<DP, J, false, false, kTeam>(f, ctas, stream);
}

}  // namespace

// 9 to 16 rows a key head over 64 sequences of 2000 to 6000 keys: one tile of 16 88 us,
// two of 8 117; 20 rows over 8 of them 31.8 and 30.7, 32 rows 32.5 and 36.3.
int four_rows_per_tile(int D, int64_t rows) { return rows <= 8 || D > 128 ? 8 : 16; }

int four_rows_chunk(int D) { return D > 128 ? FourLayout<256, 1, false>::kChunk : FourLayout<128, 1, false>::kChunk; }

int four_rows_ctas_per_sm(int D, int rows)
{
    if (D > 128) return FourLayout<256, 1, false>::kCtas;
    if (rows == 8) return D > 64 ? FourLayout<128, 1, false>::kCtas : FourLayout<64, 1, false>::kCtas;
    return D > 64 ? FourLayout<128, 2, false>::kCtas : FourLayout<64, 2, false>::kCtas;
}

cudaError_t launch_four_rows(const FourParams &f, int ctas, cudaStream_t stream)
{
    if (f.p.c.D > 128) return launch_rows<256, 1, false>(f, ctas, stream);
    if (f.p.c.D > 64)
        return f.p.part.rows == 8 ? launch_rows<128, 1, false>(f, ctas, stream) : launch_rows<128, 2, false>(f, ctas, stream);
    return f.p.part.rows == 8 ? launch_rows<64, 1, false>(f, ctas, stream) : launch_rows<64, 2, false>(f, ctas, stream);
}

cudaError_t launch_four_team(const FourParams &f, int ctas, cudaStream_t stream)
{
    return f.p.c.D > 64 ? launch_rows<128, 1, true>(f, ctas, stream) : launch_rows<64, 1, true>(f, ctas, stream);
}

int four_teams_at_once(int device, int team)
{
    static std::atomic<int> known[64][kMostTeam + 1];
    if (device < 0 || device >= 64) return 0;
    std::atomic<int> &n = known[device][team];       // 1 + the answer
    if (n.load(std::memory_order_relaxed) == 0) {
        // (of the variants the one with the largest CTA)
        using Lay = FourLayout<128, 1, true>;
        const int clusters = clusters_at_once(four_rows_kernel<128, 1, false, true, true>, team, 32 * Lay::kWarps, Lay::kSmemBytes);
        n.store(1 + clusters, std::memory_order_relaxed);
    }
    return n.load(std::memory_order_relaxed) - 1;
}

cudaError_t read_and_clear_status_four(uint32_t *out)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_four, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_status_four, &zero, sizeof(zero));
        if (e != cudaSuccess) return e;
    }
    *out = v;
    return cudaSuccess;
}

}  // namespace fa
