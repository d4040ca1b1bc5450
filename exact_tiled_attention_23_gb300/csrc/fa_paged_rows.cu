// fa_paged_rows.cu -- attention of few query rows over a paged cache, and the
// merge of partial softmax states.
//
// A tile is up to 8, 16 or 32 stacked query rows of one (sequence, key head): the
// Hq / Hkv query heads that share the key head, times the query tokens.  Every
// key and value is read once for the whole tile, so a decoding step is bound
// by memory: 4 D bytes and 4 D * rows operations per key.  What the layout is
// for is to keep loads in flight:
//
//   * the keys of all tiles form one line of chunks (16 keys, 32 at D <= 64),
//     cut into equal pieces, one per warp, whatever the sequences' lengths (a
//     tile weighs as much as one chunk more, for what it costs to begin it).  A
//     tile that two or more warps had a share of leaves a partial state
//     (O_s, LSE_s) in a slot for each, and the merge joins them:
//         m = max LSE_s,  w_s = 2^(LSE_s - m),  O = sum w_s O_s / sum w_s.
//     Warps never meet.  (With four warps on a tile, joined in shared memory at
//     its end, the barriers and the code that runs once per tile, fetched anew
//     each time, took a third of the time of tiles of 512 keys.)  Where the work
//     is so little that the merge would be most of it, a cluster of CTAs takes a
//     tile instead and joins it by itself ("Teams" below);
//   * a warp has its own ring of shared-memory stages.  Where pages hold a
//     multiple of 8 keys, one lane copies boxes of 8 to 32 rows with TMA;
//     elsewhere all lanes copy 16 bytes at a time.  Either way the addresses
//     come from the page table, so any page, head and slot strides do;
//   * scores and outputs come from 16x8x16 warp products.  The tcgen05 unit
//     would have to multiply 128 rows whatever the tile holds, and its rate is
//     not what bounds this kernel;
//   * each weight p is split into two 16-bit numbers, p = hi + lo with an error
//     of 2^-16 p (fp16: 2^-22 p, or 2^-37 of the row's largest weight where that
//     is more, see kLift), and V is multiplied by both: the products are not the
//     bound.
//
// Measured (D = 128, 8 key heads of 4 queries, bf16): a token of 64 sequences of
// up to 8191 keys, 1.07 GB, 165 us, 6.5 TB/s (a copy: 6.8); of one sequence of
// 131072 keys, 537 MB, 92 us, 5.8 TB/s.  A quarter of the issue slots are used and
// 13 % of the products' rate: what is left is 3 us until the first keys land and
// 5 us from the last keys to the end of the merge.
//
// Keys at or past a sequence's length and keys of pages outside the pool get a
// score of -inf, and their rows of V are zero in shared memory (0 * NaN is NaN).
#include "fa_internal.h"
#include "fa_paged.h"
#include "fa_paged_line.cuh"
#include "fa_paged_team.cuh"
#include "fa_tc_common.cuh"
#include "sm103_ptx.cuh"

#include <atomic>
#include <cmath>

namespace fa {

__device__ uint32_t g_status_paged_rows;

namespace {

// A row's weights are p = 2^(s - m).  m is raised, and O rescaled, only where a
// score lies 2^(kLift + kRise) above it, to 2^kLift below the largest one then.
// bf16 has the exponents of fp32.  fp16 numbers are multiples of 2^-24, so hi +
// lo may be off by 2^-25 whatever p is: weights of up to 2^15 put that 2^-37 or
// more below the row's largest.  (At m = the largest, a first key that draws the
// attention lost the others: 8192 keys that share 0.5 % of the weight came out 2.6 %
// off.)
template <bool kF16> constexpr float kLift = kF16 ? 12.f : 0.f;
template <bool kF16> constexpr float kRise = kF16 ? 3.f : 8.f;

// kTeam: all warps of a cluster work on one tile and join it in shared memory
// (below); else every warp has a piece of the line.
template <int DP, int RM, bool kTeam>
struct RowsLayout {
    static constexpr int kWarps = kTeam ? kTeamWarps : kRowsWarps;
    // Up to 8 rows are the products' columns (keys and columns of V their rows:
    // half the products, weights and registers of 16 rows), more are their rows.
    static constexpr bool kColumns = RM == 8;
    static constexpr int MT = kColumns ? 1 : RM / 16;             // 16-row tiles of Q
    // Keys of a chunk, one step of a warp: 8 KB of K and V at D <= 128.
    static constexpr int kChunk = DP == 64 ? 32 : 16;
    static constexpr int kTileBytes = kChunk * DP * 2;            // K or V of a step
    static constexpr int kStageBytes = 2 * kTileBytes;
    // Q in registers, or where O leaves too few, in shared memory per warp
    static constexpr bool kQRegs = kColumns || (RM == 16 && DP <= 128);
    static constexpr int kQBytes = kQRegs ? 0 : RM * DP * 2;
    // CTAs per SM: what registers and shared memory hold
    static constexpr int kCtas = kTeam ? 1 : DP == 256 ? (RM == 8 ? 3 : 2) : RM == 32 ? 4 : 6;
    static constexpr int kStages = 2;
    static constexpr int kRingOff = 0;
    static constexpr int kQOff = kWarps * kStages * kStageBytes;
    static constexpr int kMaskOff = kQOff + kWarps * kQBytes;     // visible keys of every stage
    static constexpr int kBarOff = kMaskOff + kWarps * kStages * 4;
    static constexpr int kAbortOff = kBarOff + kWarps * kStages * 8;
    // team: (m, l) of every warp's rows, and 24 bytes for each row and four columns
    static constexpr int kStatOff = kAbortOff + kWarps * 4;
    static constexpr int kMailOff = kStatOff + kWarps * RM * 8;
    static constexpr int kSmemBytes = (kTeam ? kMailOff + RM * DP / 4 * 24 : kStatOff) + 1024;   // + alignment slack
    static_assert(RM == 8 || RM == 16 || (RM == 32 && DP <= 128), "rows");
    static_assert(kBarOff % 8 == 0 && (!kTeam || kMailOff % 16 == 0), "barriers, states");
    static_assert(!kTeam || (RM == 8 && DP <= 128 && RM * DP * 4 <= kStageBytes), "a team's states fit its stages");
    static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
};

// Byte offset of 16-byte unit `unit` of row `row` in a tile of `kTall` rows:
// 64 columns of all rows after 64 columns of all rows, and within a row's 128
// bytes the units permuted by the row's low bits (the layout that TMA's 128-byte
// swizzle gives), so that the eight rows of a matrix load touch all banks.
template <int kTall>
__device__ __forceinline__ uint32_t unit_at(int row, int unit)
{
    return (uint32_t)((unit >> 3) * (kTall * 128) + row * 128 + (((unit & 7) ^ (row & 7)) << 4));
}

// Teams.  Where there is little work, two launches and the way through memory
// between them are most of its time.  Then a cluster of up to eight CTAs takes a
// tile: every warp some of its chunks, and the states are joined through the
// cluster's shared memory.  A shared prefix, whose keys come first, is read by
// every tile: from the L2, and its rows are too few to fill the tensor cores.
// One sequence of 1000 keys, 8 key heads: 8.2 -> 5.1 us; 128 sequences of 512
// keys, one key head: 15.2 -> 8.0 us.
template <int DP, int RM, bool kF16, bool kTma, bool kTeam>
__global__ void __launch_bounds__((32 * RowsLayout<DP, RM, kTeam>::kWarps), (RowsLayout<DP, RM, kTeam>::kCtas))
paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedParams p)
{
    using Lay = RowsLayout<DP, RM, kTeam>;
    constexpr int kWarps = Lay::kWarps;
    constexpr int S = Lay::kStages, MT = Lay::MT, KS = Lay::kChunk;
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : 0xffffu;
    constexpr int NT = DP / 8;                      // 8-column tiles of O
    constexpr int KT = DP / 16;                     // 16-column steps of a score
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t s_base = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + Lay::kMaskOff) + warp * S;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff) + warp * S;
    // the warp's own: a warp that gave up a wait stops nobody else
    volatile int *abort_word = reinterpret_cast<int *>(smem + Lay::kAbortOff) + warp;
    const Abort ab{abort_word, &g_status_paged_rows};

    if constexpr (kTma) {
        // (set-up that reads no memory overlaps the end of the kernel before)
        if (lane == 0) {
            for (int i = 0; i < S; ++i) ptx::mbar_init(&full[i], 1);
            *abort_word = 0;
            ptx::fence_mbarrier_init();
            ptx::tma_prefetch_desc(&tm_k);
            ptx::tma_prefetch_desc(&tm_v);
        }
        __syncwarp();
    }
    if constexpr (kTeam) ptx::cluster_arrive();
    if (!p.second) ptx::wait_for_primary();
    ptx::launch_dependents();
    Line<KS, kRowsTile> line(p);
    const int piece = (int)blockIdx.x * kWarps + warp;
    LineCursor at;
    // of the piece: units, those in front of `at`; a full piece's.  Team: chunks.
    int units, used, per;
    int front = 0;              // team: chunks of the prefix, before the own ones
    if constexpr (kTeam) {
        const int tile = (int)blockIdx.x / p.team, g = tile / p.c.Hkv;
        line.enter(at, g);
        at.h = tile - g * p.c.Hkv;
        front = chunks_of(p.prefix_len, KS);
        at.n += front;
        const int warps = p.team * kWarps, mine = ((int)blockIdx.x - tile * p.team) * kWarps + warp;
        per = (at.n + warps - 1) / warps;
        at.c = min(mine * per, at.n);
        units = min(per, at.n - at.c);
        used = 0;
    } else {
        line.share(piece, (int)gridDim.x * kWarps, at, used, units, per);
        units += used;
    }
    const int R = line.R;

    // ---- loads -----------------------------------------------------------
    LineCursor ld = at;
    int ld_left = units - used;
    // Where this lane's key of a step is (lane % KS).  Its page number is
    // fetched at least one step before its use.
    struct Place {
        int page, slot, h;      // page < 0: not a key that the tile sees; h < 0: past the piece
    };
    auto look_up = [&]() -> Place {
        if (ld_left <= 0) return Place{-1, 0, -1};
        Place x{-1, 0, ld.h};
        const int key = (ld.c - front) * KS + lane % KS;
        if (kTeam && ld.c < front) {
            const int k = ld.c * KS + lane % KS;
            if (k < p.prefix_len) {
                const int which = p.c.by_page.quotient(k);
                x.slot = k - which * p.c.page_size;
                x.page = p.prefix_table[which];
            }
        } else if (key < ld.keys) {
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
    const uint32_t ring = s_base + Lay::kRingOff + warp * S * Lay::kStageBytes;
    // A sequence with one row tile has its keys read once, by that tile, unless
    // another sequence's table has the same pages.  They leave the L2 first, and a
    // prefix that other CTAs read again and again keeps its place (256 sequences
    // behind a prefix of 4097 keys: 77 -> 66 us; 64 sequences of up to 8191 keys of
    // their own: 169 -> 165).  Pages that tables share do not lose by it: 64
    // sequences with 4096 keys in common, 89.6 -> 89.3, 16 with 32768, 166.6 ->
    // 165.6, 256 with 1024, 95.8 -> 95.4.
    const uint64_t policy = kTma ? ptx::l2_policy(!kTeam && p.part.tiles == 1) : 0;
    int issued = 0;             // steps copied
    auto load = [&](int stage, const Place &x) {
        const bool ok = x.page >= 0 && x.page < p.c.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAll;
        if (lane == 0) s_mask[stage] = mask;
        const uint32_t dst = ring + stage * Lay::kStageBytes;
        if constexpr (kTma) {
            if (x.h < 0) return;
            ++issued;
            if (lane == 0) ptx::mbar_arrive_expect_tx(&full[stage], Lay::kStageBytes);
            const int page = ok ? x.page : p.c.num_pages;         // past the tensor's end: zeros
#pragma unroll 1
            for (int i = 0; i < KS; i += p.box_rows) {
                const int box_page = __shfl_sync(0xffffffffu, page, i), box_slot = __shfl_sync(0xffffffffu, x.slot, i);
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c) {
                        ptx::tma_load_4d_hint(dst + (c * KS + i) * 128, &tm_k, &full[stage], c * 64, box_slot, x.h,
                                              box_page, policy);
                        ptx::tma_load_4d_hint(dst + Lay::kTileBytes + (c * KS + i) * 128, &tm_v, &full[stage], c * 64,
                                              box_slot, x.h, box_page, policy);
                    }
                }
            }
        } else {
            const int64_t off =
                ok ? (int64_t)x.page * p.c.s_page + (int64_t)x.h * p.c.s_head + (int64_t)x.slot * p.c.s_slot : 0;
            constexpr int kLanes = DP / 8 < 32 ? DP / 8 : 32;      // lanes per row
            constexpr int kRowsPer = 32 / kLanes;
            const int unit = lane % kLanes;
#pragma unroll
            for (int i = 0; i < KS / kRowsPer; ++i) {
                const int row = i * kRowsPer + lane / kLanes;
                const int64_t o = __shfl_sync(0xffffffffu, off, row);
                const uint32_t bytes = ((mask >> row) & 1u) && unit * 8 < p.c.D ? 16u : 0u;
                const int64_t src = bytes ? o + unit * 8 : 0;
                const uint32_t to = dst + unit_at<KS>(row, unit);
                ptx::cp_async16(to, p.c.k + src, bytes);
                ptx::cp_async16(to + Lay::kTileBytes, p.c.v + src, bytes);
            }
            ptx::cp_async_commit();
        }
    };
    Place next = look_up();
#pragma unroll 1
    for (int s = 0; s < S; ++s) {
        const Place x = next;
        next = look_up();
        load(s, x);
    }

    // ---- the piece, tile by tile -------------------------------------------
    const int qr = lane >> 2, qc = lane & 3;        // this lane's rows (qr, qr + 8) and columns (2 qc, +1) of a product
    const uint32_t q_smem = s_base + Lay::kQOff + warp * Lay::kQBytes;
    int stage = 0;
    uint32_t phase = 0;
    // Waits for a step's keys; returns which of them are visible.  After a wait
    // that gave up (the results are undefined then) the warp computes nothing
    // and, above all, copies nothing more: its stages still have copies in
    // flight, and an arrival on a barrier whose phase they hold open is invalid.
    bool gave_up = false;
    auto landed = [&]() -> uint32_t {
        if constexpr (kTma) {
            if (!gave_up)
                gave_up = !__all_sync(0xffffffffu, wait_bounded(&full[stage], phase, p.wait_limit_ns, kSiteSlotFull, ab));
            if (gave_up) return 0u;
        } else {
            ptx::cp_async_wait<S - 1>();
            __syncwarp();
        }
        return s_mask[stage];
    };
    // A box brings what its page holds behind the last key.
    auto clear_rest = [&](uint32_t mask, uint32_t vt) {
        if constexpr (kTma) {
            if (mask == kAll) return;
#pragma unroll 1
            for (int e = lane; e < KS * (DP / 8); e += 32)
                if (!((mask >> (e % KS)) & 1u)) ptx::st_shared_v4(vt + unit_at<KS>(e % KS, e / KS), 0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();          // before the next copy into the stage
            __syncwarp();
        }
    };
    // The step is done: its stage takes the next one (past the piece, nothing).
    auto refill = [&] {
        __syncwarp();
        if (gave_up) return;
        const Place x = next;
        next = look_up();
        load(stage, x);
        if (++stage == S) {
            stage = 0;
            phase ^= 1;
        }
    };
    // No copy may still be landing in shared memory at exit.
    auto drain = [&] {
        if constexpr (kTma) {
            for (int i = max(0, issued - S); i < issued; ++i)
                wait_bounded(&full[i % S], (i / S) & 1, p.wait_limit_ns, kSiteDrain, ab, false);
        } else {
            ptx::cp_async_wait<0>();
        }
    };
#pragma unroll 1
    while (kTeam || used < units) {
        const int rest = units - used;
        const int count = kTeam ? rest : min(at.n - at.c, line.chunks_within(at.c, rest));      // chunks of this tile in the piece
        const int b = p.part.tiles == 1 ? at.g : at.g / p.part.tiles;
        const int row0 = (at.g - b * p.part.tiles) * RM, h = at.h;
        const int tile = at.g * p.c.Hkv + h;
        if (!kTeam && at.c == 0 && lane == 0) line.record(at, piece, used, per);

        const int lim_all = line.masked ? at.len - p.T + p.by_g.quotient(row0) + 1 : at.len;   // seen by every row

        if constexpr (Lay::kColumns) {
            // Q: this lane's row qr, columns 2 qc, +1 of every 8
            uint32_t qb[KT][2];
#pragma unroll
            for (int k = 0; k < KT; ++k) qb[k][0] = qb[k][1] = 0u;
            if (row0 + qr < R) {
                const RowPlace x = row_place(p, b, h, row0 + qr);
                const uint16_t *src = p.q + x.b * p.q_s[0] + x.hq * p.q_s[1] + x.t * p.q_s[2] + 2 * qc;
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (16 * k + 8 * e < p.c.D) qb[k][e] = *reinterpret_cast<const uint32_t *>(src + 16 * k + 8 * e);
            }
            int lim[2];                             // keys that rows 2 qc and 2 qc + 1 see
#pragma unroll
            for (int r = 0; r < 2; ++r)
                lim[r] = line.masked ? at.len - p.T + p.by_g.quotient(row0 + 2 * qc + r) + 1 : at.len;
            // o[n]: columns 16 n + qr (and + 8) of rows 2 qc and 2 qc + 1
            float o[KT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < KT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

#pragma unroll 1
            for (int step = 0; step < count; ++step) {
                const uint32_t mask = landed();
                const uint32_t kt = ring + stage * Lay::kStageBytes, vt = kt + Lay::kTileBytes;
                // (the prefix's keys come before every row's limit)
                const int key0 = at.c + step < front ? INT32_MIN / 2 : (at.c + step - front) * KS;
                if (mask) {
                    // scores of keys 16 j + qr (and + 8) and the two rows
                    float s[KS / 16][4];
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int j = 0; j < KS / 16; ++j) {
                            uint32_t ka[4];
                            ptx::ldmatrix4(ka, kt + unit_at<KS>(16 * j + (lane & 15), 2 * k + (lane >> 4)));
                            ptx::mma_16816<kF16>(s[j], ka, qb[k][0], qb[k][1]);
                        }
                    if (mask != kAll || key0 + KS > lim_all) {
                        clear_rest(mask, vt);
#pragma unroll
                        for (int j = 0; j < KS / 16; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = 16 * j + qr + 8 * (e >> 1);
                                if (!((mask >> key) & 1u) || key0 + key >= lim[e & 1]) s[j][e] = -INFINITY;
                            }
                    }
                    float ref[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float mx = fmaxf(s[0][r], s[0][r + 2]);
#pragma unroll
                        for (int j = 1; j < KS / 16; ++j) mx = ptx::max3(mx, s[j][r], s[j][r + 2]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        mx *= p.scale_log2;
                        if (__any_sync(0xffffffffu, mx > m[r] + (kLift<kF16> + kRise<kF16>))) {
                            const float m_new = fmaxf(m[r], mx - kLift<kF16>);
                            const float alpha = ptx::ex2_approx(m[r] - (m_new == -INFINITY ? 0.f : m_new));
                            l[r] *= alpha;
#pragma unroll
                            for (int n = 0; n < KT; ++n) {
                                o[n][r] *= alpha;
                                o[n][r + 2] *= alpha;
                            }
                            m[r] = m_new;
                        }
                        ref[r] = m[r] == -INFINITY ? 0.f : m[r];
                    }
                    uint32_t hi[KS / 16][2], lo[KS / 16][2];
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float p0 = ptx::ex2_approx(fmaf(s[j][2 * e], p.scale_log2, -ref[0]));
                            const float p1 = ptx::ex2_approx(fmaf(s[j][2 * e + 1], p.scale_log2, -ref[1]));
                            l[0] += p0;
                            l[1] += p1;
                            const uint32_t w = ptx::pack16x2<kF16>(p0, p1);
                            float r0, r1;
                            ptx::unpack2(ptx::widen16x2<kF16>(w), r0, r1);
                            // keys of a lane's weights become those of a product's lane
                            hi[j][e] = ptx::transpose8(w);
                            lo[j][e] = ptx::transpose8(ptx::pack16x2<kF16>(p0 - r0, p1 - r1));
                        }
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j)
#pragma unroll
                        for (int n = 0; n < KT; ++n) {
                            // columns 16 n .. of V as rows, keys 16 j .. as the product's k
                            uint32_t va[4];
                            ptx::ldmatrix4_trans(va, vt + unit_at<KS>(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * n + ((lane >> 3) & 1)));
                            ptx::mma_16816<kF16>(o[n], va, hi[j][0], hi[j][1]);
                            ptx::mma_16816<kF16>(o[n], va, lo[j][0], lo[j][1]);
                        }
                }
                refill();
            }

            if constexpr (kTeam) {
                drain();
                __syncwarp();
                // O over the warp's first stage: four columns of all rows after
                // four columns of all rows
                float *mine = reinterpret_cast<float *>(smem + Lay::kRingOff + warp * S * Lay::kStageBytes);
                float2 *stat = reinterpret_cast<float2 *>(smem + Lay::kStatOff) + warp * RM;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float sum = l[r];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    if (qr == 0) stat[2 * qc + r] = make_float2(m[r], sum);
#pragma unroll
                    for (int n = 0; n < KT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            mine[((4 * n + 2 * e + qr / 4) * RM + 2 * qc + r) * 4 + qr % 4] = o[n][2 * e + r];
                }
                join_team<DP, kF16>(p, smem + Lay::kRingOff, S * Lay::kStageBytes,
                                    reinterpret_cast<const float2 *>(smem + Lay::kStatOff),
                                    reinterpret_cast<float4 *>(smem + Lay::kMailOff), b, h, at.len);
                return;
            }

            // ---- the tile's state ----
            const bool direct = count == at.n && !p.joined;
            const int64_t slot = p.part.slot_of(piece, tile, at.c > 0);
            bool empty[2];
            float inv[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[r];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                // (a NaN among the scores reaches the output)
                empty[r] = sum == 0.f;
                inv[r] = empty[r] ? 0.f : 1.f / sum;
                const int tr = 2 * qc + r;
                if (qr == 0 && row0 + tr < R) {
                    const float lse2 = empty[r] ? -INFINITY : m[r] + log2f(sum);
                    if (!direct) {
                        p.part.lse[slot * p.part.slot_rows + tr] = lse2;
                    } else if (p.lse) {
                        const RowPlace x = row_place(p, b, h, row0 + tr);
                        p.lse[((int64_t)x.b * p.Hq + x.hq) * p.T + x.t] = lse2 * kLn2;
                    }
                }
            }
            if (direct) {
                // back to a row's neighbouring columns per lane
                const bool mine = row0 + qr < R;
                const RowPlace x = row_place(p, b, h, mine ? row0 + qr : row0);
                uint16_t *dst = p.o + x.b * p.o_s[0] + x.hq * p.o_s[1] + x.t * p.o_s[2] + 2 * qc;
#pragma unroll
                for (int n = 0; n < KT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w = ptx::transpose8(ptx::pack16x2<kF16>(empty[0] ? 0.f : o[n][2 * e] * inv[0],
                                                                               empty[1] ? 0.f : o[n][2 * e + 1] * inv[1]));
                        if (mine && 16 * n + 8 * e < p.c.D) *reinterpret_cast<uint32_t *>(dst + 16 * n + 8 * e) = w;
                    }
            } else {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (row0 + 2 * qc + r >= R) continue;
                    float *dst = p.part.o + ((slot * (p.c.D / 4) + qr / 4) * p.part.slot_rows + 2 * qc + r) * 4 + qr % 4;
#pragma unroll
                    for (int n = 0; n < KT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (16 * n + 8 * e < p.c.D)
                                dst[(4 * n + 2 * e) * 4 * p.part.slot_rows] = empty[r] ? 0.f : o[n][2 * e + r] * inv[r];
                }
            }
        } else {
            // Q: rows past R and columns past D are zero
            uint32_t qf[Lay::kQRegs ? KT : 1][4];
            if constexpr (Lay::kQRegs) {
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) qf[k][e] = 0u;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (row0 + qr + 8 * r >= R) continue;
                    const RowPlace x = row_place(p, b, h, row0 + qr + 8 * r);
                    const uint16_t *src = p.q + x.b * p.q_s[0] + x.hq * p.q_s[1] + x.t * p.q_s[2] + 2 * qc;
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (16 * k + 8 * e < p.c.D) qf[k][2 * e + r] = *reinterpret_cast<const uint32_t *>(src + 16 * k + 8 * e);
                }
            } else {
                __syncwarp();
#pragma unroll 4
                for (int e = lane; e < RM * (DP / 8); e += 32) {
                    const int row = e / (DP / 8), unit = e % (DP / 8);
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (row0 + row < R && unit * 8 < p.c.D) {
                        const RowPlace x = row_place(p, b, h, row0 + row);
                        w = *reinterpret_cast<const uint4 *>(p.q + x.b * p.q_s[0] + x.hq * p.q_s[1] + x.t * p.q_s[2] + unit * 8);
                    }
                    ptx::st_shared_v4(q_smem + unit_at<RM>(row, unit), w.x, w.y, w.z, w.w);
                }
                __syncwarp();
            }
            int lim[2 * MT];                            // keys that this lane's rows see
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                lim[i] = line.masked ? at.len - p.T + p.by_g.quotient(row0 + i * 8 + qr) + 1 : at.len;

            float o[MT][NT][4], m[2 * MT], l[2 * MT];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) { m[i] = -INFINITY; l[i] = 0.f; }

#pragma unroll 1
            for (int step = 0; step < count; ++step) {
                const uint32_t mask = landed();
                const uint32_t kt = ring + stage * Lay::kStageBytes, vt = kt + Lay::kTileBytes;
                const int key0 = (at.c + step) * KS;
                if (mask) {
                    float s[MT][KS / 8][4];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int n = 0; n < KS / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
                        uint32_t qa[MT][4];
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            if constexpr (Lay::kQRegs) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) qa[i][e] = qf[k][e];
                            } else {
                                ptx::ldmatrix4(qa[i], q_smem + unit_at<RM>(i * 16 + (lane & 15), 2 * k + (lane >> 4)));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < KS / 16; ++j) {
                            // K rows 16j .. +7 and +8 .. +15, columns 16k .. +7 and +8 .. +15
                            uint32_t kb[4];
                            ptx::ldmatrix4(kb, kt + unit_at<KS>(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                ptx::mma_16816<kF16>(s[i][2 * j], qa[i], kb[0], kb[1]);
                                ptx::mma_16816<kF16>(s[i][2 * j + 1], qa[i], kb[2], kb[3]);
                            }
                        }
                    }
                    if (mask != kAll || key0 + KS > lim_all) {
                        clear_rest(mask, vt);
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int n = 0; n < KS / 8; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int key = n * 8 + 2 * qc + (e & 1);
                                    if (!((mask >> key) & 1u) || key0 + key >= lim[2 * i + (e >> 1)]) s[i][n][e] = -INFINITY;
                                }
                    }
                    uint32_t hi[MT][KS / 16][4], lo[MT][KS / 16][4];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float &mr = m[2 * i + r], &lr = l[2 * i + r];
                            float mx = fmaxf(s[i][0][2 * r], s[i][0][2 * r + 1]);
#pragma unroll
                            for (int n = 1; n < KS / 8; ++n) mx = ptx::max3(mx, s[i][n][2 * r], s[i][n][2 * r + 1]);
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                            mx *= p.scale_log2;
                            if (__any_sync(0xffffffffu, mx > mr + (kLift<kF16> + kRise<kF16>))) {
                                const float m_new = fmaxf(mr, mx - kLift<kF16>), ref = m_new == -INFINITY ? 0.f : m_new;
                                const float alpha = ptx::ex2_approx(mr - ref);
                                lr *= alpha;
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    o[i][n][2 * r] *= alpha;
                                    o[i][n][2 * r + 1] *= alpha;
                                }
                                mr = m_new;
                            }
                            const float ref = mr == -INFINITY ? 0.f : mr;
#pragma unroll
                            for (int n = 0; n < KS / 8; ++n) {
                                const float p0 = ptx::ex2_approx(fmaf(s[i][n][2 * r], p.scale_log2, -ref));
                                const float p1 = ptx::ex2_approx(fmaf(s[i][n][2 * r + 1], p.scale_log2, -ref));
                                lr += p0 + p1;
                                const uint32_t w = ptx::pack16x2<kF16>(p0, p1);
                                float r0, r1;
                                ptx::unpack2(ptx::widen16x2<kF16>(w), r0, r1);
                                hi[i][n / 2][2 * (n & 1) + r] = w;
                                lo[i][n / 2][2 * (n & 1) + r] = ptx::pack16x2<kF16>(p0 - r0, p1 - r1);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j)
#pragma unroll
                        for (int n = 0; n < KT; ++n) {
                            // V rows 16j .. +7 and +8 .. +15 (the product's k), columns 16n .. +7 and +8 .. +15
                            uint32_t vb[4];
                            ptx::ldmatrix4_trans(vb, vt + unit_at<KS>(16 * j + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                ptx::mma_16816<kF16>(o[i][2 * n], hi[i][j], vb[0], vb[1]);
                                ptx::mma_16816<kF16>(o[i][2 * n + 1], hi[i][j], vb[2], vb[3]);
                                ptx::mma_16816<kF16>(o[i][2 * n], lo[i][j], vb[0], vb[1]);
                                ptx::mma_16816<kF16>(o[i][2 * n + 1], lo[i][j], vb[2], vb[3]);
                            }
                        }
                }
                refill();
            }

            // ---- the tile's state -------------------------------------------------
            const bool direct = count == at.n && !p.joined;
            const int64_t slot = p.part.slot_of(piece, tile, at.c > 0);
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                float sum = l[i];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int tr = i * 8 + qr;
                if (row0 + tr >= R) continue;
                // (a NaN among the scores reaches the output)
                const bool empty = sum == 0.f;
                const float inv = empty ? 0.f : 1.f / sum;
                const float lse2 = empty ? -INFINITY : m[i] + log2f(sum);
                if (direct) {
                    const RowPlace x = row_place(p, b, h, row0 + tr);
                    uint16_t *dst = p.o + x.b * p.o_s[0] + x.hq * p.o_s[1] + x.t * p.o_s[2] + 2 * qc;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (8 * n < p.c.D)
                            *reinterpret_cast<uint32_t *>(dst + 8 * n) =
                                empty ? 0u : ptx::pack16x2<kF16>(o[i / 2][n][2 * (i & 1)] * inv, o[i / 2][n][2 * (i & 1) + 1] * inv);
                    if (p.lse && qc == 0) p.lse[((int64_t)x.b * p.Hq + x.hq) * p.T + x.t] = lse2 * kLn2;
                } else {
                    // columns 8n + 2 qc and the next: half of four columns
                    float2 *dst = reinterpret_cast<float2 *>(p.part.o) +
                                  ((slot * (p.c.D / 4) + qc / 2) * p.part.slot_rows + tr) * 2 + (qc & 1);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (8 * n < p.c.D)
                            dst[n * 4 * p.part.slot_rows] =
                                empty ? make_float2(0.f, 0.f)
                                      : make_float2(o[i / 2][n][2 * (i & 1)] * inv, o[i / 2][n][2 * (i & 1) + 1] * inv);
                    if (qc == 0) p.part.lse[slot * p.part.slot_rows + tr] = lse2;
                }
            }
        }
        __syncwarp();
        used += line.start_of(at.c + count) - line.start_of(at.c);
        at.c += count - 1;
        line.advance(at);
    }
    drain();
    // the merge starts when this kernel has ended, and needs the one before too
    if (p.second) ptx::wait_for_primary();
}

template <int DP, int RM, bool kF16, bool kTma, bool kTeam = false>
cudaError_t launch_rows(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    using Lay = RowsLayout<DP, RM, kTeam>;
    static SharedMemory allowed;
    const cudaError_t e = allowed.allow(paged_rows_kernel<DP, RM, kF16, kTma, kTeam>, Lay::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_clusters(paged_rows_kernel<DP, RM, kF16, kTma, kTeam>, kTeam ? p.team : 1, dim3((unsigned)ctas),
                           32 * Lay::kWarps, Lay::kSmemBytes, stream, tk, tv, p);
}

template <int DP, int RM>
cudaError_t launch_rows_f(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    if (p.box_rows)
        return p.f16 ? launch_rows<DP, RM, true, true>(p, tk, tv, ctas, stream)
                     : launch_rows<DP, RM, false, true>(p, tk, tv, ctas, stream);
    return p.f16 ? launch_rows<DP, RM, true, false>(p, tk, tv, ctas, stream)
                 : launch_rows<DP, RM, false, false>(p, tk, tv, ctas, stream);
}

// ---------------------------------------------------------------- merge
// The sum of a row's partial outputs, weighted by their LSEs against the
// largest.  A CTA has kRows rows of a key head and 4 kCols of their columns, and
// kZ threads for each four columns, which take every kZ-th state and are joined in
// order: one thread's chain of loads through the 228 states of a row (one sequence
// of 131072 keys) took 18 us.  Where kZ = 1 there are many rows of few states: a
// thread has four columns twice, so that fewer CTAs wait for a place.  The lanes of
// a load are neighbours in the slots.  (The form of 32 threads spills 108 bytes of
// the 32 states that it joins at the end; read eight at a time they do not, and
// that sequence takes the same 90.5 us.)
constexpr int kMergeThreads = 256;

constexpr int merge_wide(int z) { return z == 1 ? 2 : 1; }
constexpr int merge_rows(int cols, int z) { return kMergeThreads * merge_wide(z) / (cols * z); }

template <int kCols, int kZ, bool kF16>
__global__ void __launch_bounds__(kMergeThreads, 4) paged_merge_kernel(const MergeParams p, const int groups)
{
    constexpr int kRows = merge_rows(kCols, kZ), kWide = merge_wide(kZ), kPart = kCols / kWide;
    const int row = threadIdx.x % kRows, col4 = threadIdx.x / kRows % kPart, z = threadIdx.x / (kRows * kPart);
    const int R = p.G * p.T, Hkv = p.Hq / p.G, h = blockIdx.y;
    // a sequence's rows take `groups` CTAs, or, if 0, a CTA has those of several
    const int several = groups ? 1 : kRows / R, sub = groups ? 0 : p.by_r.quotient(row);
    const int at_b = groups ? blockIdx.x / (unsigned)groups : blockIdx.x * several + sub;
    const int idx = groups ? (blockIdx.x - at_b * groups) * kRows + row : row - sub * R;
    const bool real = idx < R && sub < several && at_b < p.B;
    const int b = real ? at_b : 0;
    const int t = p.by_g.quotient(real ? idx : 0), hq = h * p.G + (real ? idx : 0) - t * p.G;

    // before the kernels that write the states have ended
    int len = p.seq_len[b];
    len = len < 0 ? 0 : (len > p.max_len ? p.max_len : len);
    const bool padding = p.causal && len - p.T + t < 0;        // no token here
    int keys[2], at[2], tile[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Partials &src = p.src[s];
        const int i = (real ? idx : 0) + (src.stacked ? b * R : 0);
        const int rt = s < p.n_src ? i / src.rows : 0;
        at[s] = i - rt * src.rows;
        tile[s] = ((src.stacked ? 0 : b) * src.tiles + rt) * Hkv + h;
        keys[s] = s >= p.n_src || padding || !real
                      ? 0
                      : src.stacked ? src.fixed_len
                                    : keys_of_tile(len, rt, src.rows, R, p.by_g, p.T, p.causal != 0);
    }
    ptx::wait_for_primary();

    // (read before it is known whether the tile has any keys: one wait less)
    TileSlots x[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) x[s] = s < p.n_src ? p.src[s].tile[tile[s]] : TileSlots{0, 0};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        // no read past the workspace, whatever a kernel that gave up has left
        x[s].first = min(max(x[s].first, 0), p.src[s].slots);
        x[s].count = keys[s] > 0 ? min(x[s].count, (p.src[s].slots - x[s].first) >> p.src[s].pairs) : 0;
    }
    // not a row, or one CTA had the whole tile and wrote the row itself
    const bool skip = !real || (!p.joined && x[0].count == 1);
    if constexpr (kZ == 1)
        if (skip) return;

    // A batch of states at a time, their LSEs and outputs loaded together; the
    // sums follow the largest LSE so far.
    constexpr int kBatch = kZ == 1 ? 2 : 4;
    const int c = blockIdx.z * kCols + col4;        // and every kPart-th
    float top = -INFINITY, sum = 0.f;
    float4 acc[kWide];
#pragma unroll
    for (int e = 0; e < kWide; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!skip && c < p.D / 4) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Partials &src = p.src[s];
            const float *lse = src.lse + at[s];
            const int64_t step = (int64_t)(p.D / 4) * src.slot_rows;
            const float4 *o = reinterpret_cast<const float4 *>(src.o) + (int64_t)c * src.slot_rows + at[s];
            for (int i = z; i < x[s].count; i += kBatch * kZ) {
                float y[kBatch];
                float4 v[kBatch][kWide];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    y[j] = -INFINITY;
                    const bool is = i + j * kZ < x[s].count;
                    const int64_t slot = src.slot_at(x[s].first, i + j * kZ);
                    if (is) y[j] = lse[slot * src.slot_rows];
#pragma unroll
                    for (int e = 0; e < kWide; ++e) {
                        v[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (is && c + e * kPart < p.D / 4) v[j][e] = o[slot * step + e * kPart * src.slot_rows];
                    }
                }
                float next = top;
#pragma unroll
                for (int j = 0; j < kBatch; ++j) next = fmaxf(next, y[j]);
                const float ref = next == -INFINITY ? 0.f : next;
                const float f = ptx::ex2_approx(top - ref);
                top = next;
                sum *= f;
#pragma unroll
                for (int e = 0; e < kWide; ++e) {
                    acc[e].x *= f;
                    acc[e].y *= f;
                    acc[e].z *= f;
                    acc[e].w *= f;
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const float w = ptx::ex2_approx(y[j] - ref);
                    sum += w;
#pragma unroll
                    for (int e = 0; e < kWide; ++e) {
                        acc[e].x = fmaf(w, v[j][e].x, acc[e].x);
                        acc[e].y = fmaf(w, v[j][e].y, acc[e].y);
                        acc[e].z = fmaf(w, v[j][e].z, acc[e].z);
                        acc[e].w = fmaf(w, v[j][e].w, acc[e].w);
                    }
                }
            }
        }
    }
    if constexpr (kZ > 1) {
        __shared__ float2 s_stat[kMergeThreads];
        __shared__ float4 s_acc[kMergeThreads];
        s_stat[threadIdx.x] = make_float2(top, sum);
        s_acc[threadIdx.x] = acc[0];
        __syncthreads();
        if (z != 0) return;
        float2 st[kZ];
#pragma unroll
        for (int j = 0; j < kZ; ++j) st[j] = s_stat[threadIdx.x + j * kRows * kCols];
#pragma unroll
        for (int j = 1; j < kZ; ++j) top = fmaxf(top, st[j].x);
        const float ref = top == -INFINITY ? 0.f : top;
        sum = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kZ; ++j) {
            const float w = ptx::ex2_approx(st[j].x - ref);
            const float4 v = s_acc[threadIdx.x + j * kRows * kCols];
            sum = fmaf(w, st[j].y, sum);
            acc[0].x = fmaf(w, v.x, acc[0].x);
            acc[0].y = fmaf(w, v.y, acc[0].y);
            acc[0].z = fmaf(w, v.z, acc[0].z);
            acc[0].w = fmaf(w, v.w, acc[0].w);
        }
    }
    if (skip || c >= p.D / 4) return;
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
    uint16_t *dst = p.o + b * p.o_s[0] + hq * p.o_s[1] + t * p.o_s[2];
#pragma unroll
    for (int e = 0; e < kWide; ++e)
        if (c + e * kPart < p.D / 4)
            *reinterpret_cast<uint2 *>(dst + 4 * (c + e * kPart)) =
                empty ? make_uint2(0u, 0u)
                      : make_uint2(ptx::pack16x2<kF16>(acc[e].x * inv, acc[e].y * inv),
                                   ptx::pack16x2<kF16>(acc[e].z * inv, acc[e].w * inv));
    if (p.lse && c == 0) p.lse[((int64_t)b * p.Hq + hq) * p.T + t] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int kCols, int kZ>
cudaError_t launch_merge(const MergeParams &p, cudaStream_t stream)
{
    constexpr int kRows = merge_rows(kCols, kZ);
    const int R = p.G * p.T, groups = 2 * R <= kRows ? 0 : (R + kRows - 1) / kRows;
    const int blocks = groups ? p.B * groups : (p.B + kRows / R - 1) / (kRows / R);
    const dim3 grid((unsigned)blocks, (unsigned)(p.Hq / p.G), (unsigned)((p.D / 4 + kCols - 1) / kCols));
    return p.f16 ? launch_behind(paged_merge_kernel<kCols, kZ, true>, grid, kMergeThreads, 0, stream, p, groups)
                 : launch_behind(paged_merge_kernel<kCols, kZ, false>, grid, kMergeThreads, 0, stream, p, groups);
}

template <int kCols>
cudaError_t launch_merge_z(const MergeParams &p, int z, cudaStream_t stream)
{
    switch (z) {
    case 1: return launch_merge<kCols, 1>(p, stream);
    case 2: return launch_merge<kCols, 2>(p, stream);
    case 4: return launch_merge<kCols, 4>(p, stream);
    default: return launch_merge<kCols, 8>(p, stream);
    }
}

}  // namespace

// 8 or 16 rows where they hold the tile, 16 where D = 256 leaves no registers
// for more, else 32.
int paged_rows_per_tile(int D, int64_t rows) { return rows <= 8 ? 8 : rows <= 16 || D > 128 ? 16 : 32; }

int paged_rows_chunk(int D) { return D <= 64 ? RowsLayout<64, 16, false>::kChunk : RowsLayout<128, 16, false>::kChunk; }

int paged_rows_ctas_per_sm(int D, int rows)
{
    if (D > 128) return rows == 8 ? RowsLayout<256, 8, false>::kCtas : RowsLayout<256, 16, false>::kCtas;
    return rows == 32 ? RowsLayout<128, 32, false>::kCtas : RowsLayout<128, 16, false>::kCtas;
}

cudaError_t launch_paged_rows(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                              cudaStream_t stream)
{
    if (p.c.D > 128)
        return p.part.rows == 8 ? launch_rows_f<256, 8>(p, tk, tv, ctas, stream)
                                : launch_rows_f<256, 16>(p, tk, tv, ctas, stream);
    if (p.c.D > 64)
        return p.part.rows == 8    ? launch_rows_f<128, 8>(p, tk, tv, ctas, stream)
               : p.part.rows == 16 ? launch_rows_f<128, 16>(p, tk, tv, ctas, stream)
                                   : launch_rows_f<128, 32>(p, tk, tv, ctas, stream);
    return p.part.rows == 8    ? launch_rows_f<64, 8>(p, tk, tv, ctas, stream)
           : p.part.rows == 16 ? launch_rows_f<64, 16>(p, tk, tv, ctas, stream)
                               : launch_rows_f<64, 32>(p, tk, tv, ctas, stream);
}

template <int DP>
cudaError_t launch_team(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    if (p.box_rows)
        return p.f16 ? launch_rows<DP, 8, true, true, true>(p, tk, tv, ctas, stream)
                     : launch_rows<DP, 8, false, true, true>(p, tk, tv, ctas, stream);
    return p.f16 ? launch_rows<DP, 8, true, false, true>(p, tk, tv, ctas, stream)
                 : launch_rows<DP, 8, false, false, true>(p, tk, tv, ctas, stream);
}

cudaError_t launch_paged_team(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    return p.c.D > 64 ? launch_team<128>(p, tk, tv, ctas, stream) : launch_team<64>(p, tk, tv, ctas, stream);
}

int paged_teams_at_once(int device, int team)
{
    static std::atomic<int> known[64][kMostTeam + 1];
    if (device < 0 || device >= 64) return 0;
    std::atomic<int> &n = known[device][team];       // 1 + the answer
    if (n.load(std::memory_order_relaxed) == 0) {
        // (every variant takes a whole SM per CTA)
        using Lay = RowsLayout<128, 8, true>;
        const int clusters = clusters_at_once(paged_rows_kernel<128, 8, false, true, true>, team, 32 * Lay::kWarps, Lay::kSmemBytes);
        n.store(1 + clusters, std::memory_order_relaxed);
    }
    return n.load(std::memory_order_relaxed) - 1;
}

cudaError_t read_and_clear_status_paged_rows(uint32_t *out)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_paged_rows, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_status_paged_rows, &zero, sizeof(zero));
        if (e != cudaSuccess) return e;
    }
    *out = v;
    return cudaSuccess;
}

cudaError_t launch_paged_merge(const MergeParams &p, int states, int sms, cudaStream_t stream)
{
    // Threads per column that share a row's states: as many as leave each two
    // or more, while the launch stays within a wave of CTAs.
    const int cols = p.D <= 64 ? 16 : 32;
    const auto ctas = [&](int z, int c) {
        const int rows = merge_rows(c, z);
        const int64_t R = p.G * p.T;
        return (2 * R <= rows ? (p.B + rows / R - 1) / (rows / R) : p.B * ((R + rows - 1) / rows)) * (p.Hq / p.G) *
               ((p.D / 4 + c - 1) / c);
    };
    if (states >= 32 && ctas(32, 8) <= 4 * sms) return launch_merge<8, 32>(p, stream);
    int z = 1;
    while (z < 8 && 4 * z <= states && ctas(2 * z, cols) <= 4 * sms) z *= 2;
    return p.D <= 64 ? launch_merge_z<16>(p, z, stream) : launch_merge_z<32>(p, z, stream);
}

}  // namespace fa
