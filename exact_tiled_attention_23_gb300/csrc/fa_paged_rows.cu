// fa_paged_rows.cu -- attention of few query rows over a paged cache, and the
// merge of partial softmax states.
//
// A tile is up to 16 or 32 stacked query rows of one (sequence, key head): the
// Hq / Hkv query heads that share the key head, times the query tokens.  Every
// key and value is read once for the whole tile, so a decoding step is bound
// by memory: 4 D bytes and 4 D * rows operations per key.  What the layout is
// for is to keep loads in flight:
//
//   * the keys of all tiles form one line of chunks of 64 keys, cut into equal
//     shares, one per CTA, whatever the sequences' lengths.  A tile that two
//     or more CTAs had a share of leaves a partial state (O_s, LSE_s) in a
//     slot for each, and the merge joins them:
//         m = max LSE_s,  w_s = 2^(LSE_s - m),  O = sum w_s O_s / sum w_s;
//   * a warp takes 16 keys of a chunk and has its own ring of shared-memory
//     stages, filled with 16-byte asynchronous copies from the addresses that
//     the page table gives, one per key row, so that any page size and any
//     page, head and slot strides do.  Warps meet only where a tile ends;
//   * scores and outputs come from 16x8x16 warp products.  The tcgen05 unit
//     would have to multiply 128 rows whatever the tile holds, and its rate is
//     not what bounds this kernel;
//   * each weight p is split into two 16-bit numbers, p = hi + lo with an error
//     of 2^-16 p (fp16: 2^-22), and V is multiplied by both: the products are
//     not the bound, and the output keeps fp32's error until it is rounded.
//
// Keys at or past a sequence's length and keys of pages outside the pool are
// never read; their shared-memory rows are zero and their scores -inf.
#include "fa_paged.h"
#include "fa_paged_line.cuh"
#include "fa_tc_common.cuh"
#include "sm103_ptx.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLn2 = 0.69314718055994530942f;

template <int DP, int MT>
struct RowsLayout {
    static constexpr int kRows = 16 * MT;
    // Keys of a warp per step: 8 KB of K and V at D <= 128.  (At D = 64 with 16
    // keys the chain of a step, not memory, set the pace: eight warps an SM.)
    static constexpr int kStepKeys = DP == 64 ? 32 : 16;
    static constexpr int kChunk = kWarps * kStepKeys;
    static constexpr int kRowBytes = 2 * DP;
    static constexpr int kTileBytes = kStepKeys * kRowBytes;      // K or V of a step
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kStages = 3;              // 96 KB: two CTAs per SM (192 KB, one CTA, at D = 256)
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = kRows * kRowBytes;
    static constexpr int kStatOff = kRingOff + kWarps * kStages * kStageBytes;
    static constexpr int kStatBytes = 2 * kWarps * kRows * 4;     // m and l of every warp
    static constexpr int kMaskOff = kStatOff + kStatBytes;        // valid keys of every stage
    static constexpr int kScanOff = kMaskOff + kWarps * kStages * 4;
    static constexpr int kSmemBytes = kScanOff + 128;
    static_assert((kWarps + 2) * 4 <= 128, "scratch of the line's share");
    static_assert(kStageBytes >= 16 * DP * 4, "an output tile fits a stage");
    static_assert(kSmemBytes * (DP == 256 ? 1 : 2) + (DP == 256 ? 1 : 2) * 1024 <= 233472, "shared memory per SM");
};

// Byte offset of 16-byte unit `unit` of row `row` in a tile of rows of
// `kRowBytes`: units are permuted by the row's low bits, so that the eight
// rows of a matrix load touch all banks.
template <int kRowBytes>
__device__ __forceinline__ uint32_t unit_at(int row, int unit)
{
    return (uint32_t)(row * kRowBytes + ((unit ^ (row & 7)) << 4));
}

template <int DP, int MT, bool kF16>
__global__ void __launch_bounds__(kThreads, DP == 256 ? 1 : 2) paged_rows_kernel(const PagedParams p)
{
    using Lay = RowsLayout<DP, MT>;
    constexpr int S = Lay::kStages, RM = Lay::kRows, RB = Lay::kRowBytes, KS = Lay::kStepKeys;
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : 0xffffu;
    constexpr int NT = DP / 8;                      // 8-column tiles of O
    constexpr int KT = DP / 16;                     // 16-column steps of a score
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t s_base = ptx::smem_u32(smem);
    float *s_m = reinterpret_cast<float *>(smem + Lay::kStatOff);
    float *s_l = s_m + kWarps * RM;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + Lay::kMaskOff);
    int *s_scan = reinterpret_cast<int *>(smem + Lay::kScanOff);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!p.second) ptx::wait_for_primary();
    ptx::launch_dependents();
    const Line<Lay::kChunk> line(p);
    LineCursor at;
    int g0, steps, per;
    line.template share<kThreads>(s_scan, at, g0, steps, per);
    if (steps == 0) {
        if (p.second) ptx::wait_for_primary();
        return;
    }
    const int R = line.R;

    // ---- loads -----------------------------------------------------------
    const int kr = lane % KS;                       // the key of the step whose address this lane finds
    LineCursor ld = at;
    int ld_left = steps;
    // Where a step's key is.  Its page number is fetched at least one step
    // before its use.
    struct Place {
        int page, slot, h;
    };
    auto look_up = [&]() -> Place {
        Place x{-1, 0, ld.h};
        if (ld_left <= 0) return x;
        const int key = ld.c * Lay::kChunk + warp * KS + kr;
        if (key < ld.keys) {
            const int which = p.c.by_page.quotient(key);
            const int b = p.part.tiles == 1 ? ld.g : ld.g / p.part.tiles;
            x.slot = key - which * p.c.page_size;
            x.page = p.c.table[(int64_t)b * p.c.table_stride + which];
        }
        line.advance(ld);
        --ld_left;
        return x;
    };
    const uint32_t ring = s_base + Lay::kRingOff + warp * S * Lay::kStageBytes;
    auto load = [&](int stage, const Place &x) {
        const bool ok = x.page >= 0 && x.page < p.c.num_pages;
        const int64_t off = ok ? (int64_t)x.page * p.c.s_page + (int64_t)x.h * p.c.s_head + (int64_t)x.slot * p.c.s_slot : 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAll;
        if (lane == 0) s_mask[warp * S + stage] = mask;
        constexpr int kLanes = DP / 8 < 32 ? DP / 8 : 32;      // lanes per row
        constexpr int kRowsPer = 32 / kLanes;
        const int unit = lane % kLanes;
        const uint32_t dst = ring + stage * Lay::kStageBytes;
#pragma unroll
        for (int i = 0; i < KS / kRowsPer; ++i) {
            const int row = i * kRowsPer + lane / kLanes;
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            const uint32_t bytes = ((mask >> row) & 1u) && unit * 8 < p.c.D ? 16u : 0u;
            const int64_t src = bytes ? o + unit * 8 : 0;
            const uint32_t to = dst + unit_at<RB>(row, unit);
            ptx::cp_async16(to, p.c.k + src, bytes);
            ptx::cp_async16(to + Lay::kTileBytes, p.c.v + src, bytes);
        }
        ptx::cp_async_commit();
    };
    Place next;
    {
        Place x[S];
#pragma unroll
        for (int s = 0; s < S; ++s) x[s] = look_up();
        next = look_up();
#pragma unroll
        for (int s = 0; s < S; ++s) load(s, x[s]);  // steps past the share load zeros
    }
    auto load_next = [&](int stage) {
        const Place x = next;
        next = look_up();
        load(stage, x);
    };

    // ---- the share, tile by tile ------------------------------------------
    const int qr = lane >> 2, qc = lane & 3;        // this lane's rows (qr, qr + 8) and columns (2 qc, +1) of a tile
    const uint32_t q_smem = s_base + Lay::kQOff;
    // Q of a tile: this thread's 16-byte units, loaded before the tile before
    // is joined where there are registers for them.
    constexpr int kQUnits = RM * (DP / 8) / kThreads;
    constexpr bool kQEarly = MT == 1;
    uint4 q_next[kQUnits];
    auto load_q = [&](const LineCursor &u, int i) -> uint4 {
        const int e = tid + i * kThreads, unit = e % (DP / 8);
        const int b = p.part.tiles == 1 ? u.g : u.g / p.part.tiles;
        const int row = (u.g - b * p.part.tiles) * RM + e / (DP / 8);
        if (row >= R || unit * 8 >= p.c.D) return make_uint4(0u, 0u, 0u, 0u);   // rows past R, columns past D
        const RowPlace r = row_place(p, b, u.h, row);
        return *reinterpret_cast<const uint4 *>(p.q + r.b * p.q_s[0] + r.hq * p.q_s[1] + r.t * p.q_s[2] + unit * 8);
    };
    if constexpr (kQEarly) {
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) q_next[i] = load_q(at, i);
    }
    int stage = 0, done = 0;
    while (done < steps) {
        const int count = min(at.n - at.c, steps - done);      // chunks of this tile in the share
        const int b = p.part.tiles == 1 ? at.g : at.g / p.part.tiles;
        const int row0 = (at.g - b * p.part.tiles) * RM, h = at.h;
        const int tile = at.g * p.c.Hkv + h;
        const bool whole = count == at.n;
        if (at.c == 0 && tid == 0) line.record(at, g0 + done, per);
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            const int e = tid + i * kThreads;
            const uint4 w = kQEarly ? q_next[i] : load_q(at, i);
            ptx::st_shared_v4(q_smem + unit_at<RB>(e / (DP / 8), e % (DP / 8)), w.x, w.y, w.z, w.w);
        }
        int lim[2 * MT];                            // keys that this lane's rows see
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int t = p.by_g.quotient(row0 + i * 8 + qr);
            lim[i] = line.masked ? at.len - p.T + t + 1 : at.len;
        }
        const int lim_all = line.masked ? at.len - p.T + p.by_g.quotient(row0) + 1 : at.len;   // seen by every row
        __syncthreads();

        float o[MT][NT][4], m[2 * MT], l[2 * MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) { m[i] = -INFINITY; l[i] = 0.f; }

        int last_stage = stage;
        for (int step = 0; step < count; ++step) {
            ptx::cp_async_wait<S - 1>();
            __syncwarp();
            const uint32_t kt = ring + stage * Lay::kStageBytes, vt = kt + Lay::kTileBytes;
            const uint32_t mask = s_mask[warp * S + stage];
            const int key0 = (at.c + step) * Lay::kChunk + warp * KS;
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
                    for (int i = 0; i < MT; ++i)
                        ptx::ldmatrix4(qa[i], q_smem + unit_at<RB>(i * 16 + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                    for (int j = 0; j < KS / 16; ++j) {
                        // K rows 16j .. +7 and +8 .. +15, columns 16k .. +7 and +8 .. +15
                        uint32_t kb[4];
                        ptx::ldmatrix4(kb, kt + unit_at<RB>(16 * j + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            ptx::mma_16816<kF16>(s[i][2 * j], qa[i], kb[0], kb[1]);
                            ptx::mma_16816<kF16>(s[i][2 * j + 1], qa[i], kb[2], kb[3]);
                        }
                    }
                }
                if (mask != kAll || key0 + KS > lim_all) {
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
                        const float m_new = fmaxf(mr, mx * p.scale_log2);
                        const float ref = m_new == -INFINITY ? 0.f : m_new;
                        if (__any_sync(0xffffffffu, m_new != mr)) {
                            const float alpha = ptx::ex2_approx(mr - ref);
                            lr *= alpha;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[i][n][2 * r] *= alpha;
                                o[i][n][2 * r + 1] *= alpha;
                            }
                        }
                        mr = m_new;
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
                        ptx::ldmatrix4_trans(vb, vt + unit_at<RB>(16 * j + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            ptx::mma_16816<kF16>(o[i][2 * n], hi[i][j], vb[0], vb[1]);
                            ptx::mma_16816<kF16>(o[i][2 * n + 1], hi[i][j], vb[2], vb[3]);
                            ptx::mma_16816<kF16>(o[i][2 * n], lo[i][j], vb[0], vb[1]);
                            ptx::mma_16816<kF16>(o[i][2 * n + 1], lo[i][j], vb[2], vb[3]);
                        }
                    }
            }
            __syncwarp();
            last_stage = stage;
            stage = stage + 1 == S ? 0 : stage + 1;
            // the tile's last stage is refilled after the warps' states are joined
            if (step + 1 < count) load_next(last_stage);
        }

        at.c += count - 1;
        line.advance(at);
        done += count;
        if constexpr (kQEarly) {
            if (done < steps) {
#pragma unroll
                for (int i = 0; i < kQUnits; ++i) q_next[i] = load_q(at, i);
            }
        }

        // ---- join the warps' states -----------------------------------------
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (qc == 0) {
                s_m[warp * RM + i * 8 + qr] = m[i];
                s_l[warp * RM + i * 8 + qr] = l[i];
            }
        }
        const bool direct = whole && !p.joined;
        const int64_t slot = (int64_t)blockIdx.x + tile;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            // each warp puts a 16 x DP tile of O over its last stage, with the
            // columns permuted by the row so that the stores spread over the banks
            const uint32_t mine = ring + last_stage * Lay::kStageBytes;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = qr + 8 * r, col = (n * 8 + 2 * qc) ^ ((row & 7) << 3);
                    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(mine + (uint32_t)(row * DP + col) * 4u),
                                 "f"(o[i][n][2 * r]), "f"(o[i][n][2 * r + 1]) : "memory");
                }
            __syncthreads();
            for (int e = tid; e < 16 * DP / 4; e += kThreads) {
                // along the columns for rows of O, along the rows for a slot
                const int row = direct ? e / (DP / 4) : e % 16, col = (direct ? e % (DP / 4) : e / 16) * 4;
                const int tr = i * 16 + row;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * RM + tr]);
                const float ref = top == -INFINITY ? 0.f : top;
                float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ptx::ex2_approx(s_m[w * RM + tr] - ref);
                    sum = fmaf(f, s_l[w * RM + tr], sum);
                    const float4 v = *reinterpret_cast<const float4 *>(
                        smem + Lay::kRingOff + (w * S + last_stage) * Lay::kStageBytes +
                        (size_t)(row * DP + (col ^ ((row & 7) << 3))) * 4);
                    acc[0] = fmaf(f, v.x, acc[0]);
                    acc[1] = fmaf(f, v.y, acc[1]);
                    acc[2] = fmaf(f, v.z, acc[2]);
                    acc[3] = fmaf(f, v.w, acc[3]);
                }
                // a NaN among the scores reaches the output
                const bool empty = sum == 0.f;
                const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = empty ? 0.f : acc[c] * inv;
                const int idx = row0 + tr;
                if (idx >= R) continue;
                const float lse2 = empty ? -INFINITY : top + log2f(sum);
                if (direct) {
                    const RowPlace r = row_place(p, b, h, idx);
                    if (col < p.c.D)
                        *reinterpret_cast<uint2 *>(p.o + r.b * p.o_s[0] + r.hq * p.o_s[1] + r.t * p.o_s[2] + col) =
                            make_uint2(ptx::pack16x2<kF16>(acc[0], acc[1]), ptx::pack16x2<kF16>(acc[2], acc[3]));
                    if (p.lse && col == 0) p.lse[((int64_t)r.b * p.Hq + r.hq) * p.T + r.t] = lse2 * kLn2;
                } else {
                    if (col < p.c.D)
                        reinterpret_cast<float4 *>(p.part.o)[(slot * (p.c.D / 4) + col / 4) * RM + tr] =
                            make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (col == 0) p.part.lse[slot * RM + tr] = lse2;
                }
            }
            __syncthreads();
        }
        load_next(last_stage);
    }
    ptx::cp_async_wait<0>();
    // the merge starts when this kernel has ended, and needs the one before too
    if (p.second) ptx::wait_for_primary();
}

template <int DP, int MT, bool kF16>
cudaError_t launch_rows(const PagedParams &p, int ctas, cudaStream_t stream)
{
    static SharedMemory allowed;
    const cudaError_t e = allowed.allow(paged_rows_kernel<DP, MT, kF16>, RowsLayout<DP, MT>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_behind(paged_rows_kernel<DP, MT, kF16>, dim3((unsigned)ctas), kThreads, RowsLayout<DP, MT>::kSmemBytes,
                         stream, p);
}

template <int DP, int MT>
cudaError_t launch_rows_f(const PagedParams &p, int ctas, cudaStream_t stream)
{
    return p.f16 ? launch_rows<DP, MT, true>(p, ctas, stream) : launch_rows<DP, MT, false>(p, ctas, stream);
}

// ---------------------------------------------------------------- merge
// The sum of a row's partial outputs, weighted by their LSEs against the
// largest.  A CTA has kRows rows of one (sequence, key head), kCols threads for
// four columns each, and kZ threads for each of those, which take every kZ-th
// state and are joined in order: a launch of few rows with many states each
// (one sequence of 131072 keys: 38) waited 10 us for one thread's chain of
// loads.  The lanes of a load are neighbours in the slots.
constexpr int kMergeThreads = 256;

template <int kCols, int kZ, bool kF16>
__global__ void __launch_bounds__(kMergeThreads, 4) paged_merge_kernel(const MergeParams p, const int groups)
{
    constexpr int kRows = kMergeThreads / (kCols * kZ);
    const int row = threadIdx.x % kRows, col4 = threadIdx.x / kRows % kCols, z = threadIdx.x / (kRows * kCols);
    const int b = blockIdx.x / (unsigned)groups;
    const int R = p.G * p.T, Hkv = p.Hq / p.G, h = blockIdx.y;
    const int idx = (blockIdx.x - b * groups) * kRows + row;
    const bool real = idx < R;
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

    TileSlots x[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) x[s] = keys[s] > 0 ? p.src[s].tile[tile[s]] : TileSlots{0, 0};
    // not a row, or one CTA had the whole tile and wrote the row itself
    const bool skip = !real || (!p.joined && x[0].count == 1);
    if constexpr (kZ == 1)
        if (skip) return;

    // A batch of states at a time, their LSEs and outputs loaded together; the
    // sums follow the largest LSE so far.
    constexpr int kBatch = 4;
    for (int c = col4; c < (p.D / 4 + kCols - 1) / kCols * kCols; c += kCols) {
        float top = -INFINITY, sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!skip && c < p.D / 4) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Partials &src = p.src[s];
                const float *lse = src.lse + (int64_t)x[s].first * src.rows + at[s];
                const int64_t step = (int64_t)(p.D / 4) * src.rows;
                const float4 *o = reinterpret_cast<const float4 *>(src.o) + x[s].first * step + (int64_t)c * src.rows + at[s];
                for (int i = z; i < x[s].count; i += kBatch * kZ) {
                    float y[kBatch];
                    float4 v[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        y[j] = -INFINITY;
                        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i + j * kZ < x[s].count) {
                            y[j] = lse[(int64_t)(i + j * kZ) * src.rows];
                            v[j] = o[(i + j * kZ) * step];
                        }
                    }
                    float next = top;
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) next = fmaxf(next, y[j]);
                    const float ref = next == -INFINITY ? 0.f : next;
                    const float f = ptx::ex2_approx(top - ref);
                    top = next;
                    sum *= f;
                    acc.x *= f;
                    acc.y *= f;
                    acc.z *= f;
                    acc.w *= f;
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const float w = ptx::ex2_approx(y[j] - ref);
                        sum += w;
                        acc.x = fmaf(w, v[j].x, acc.x);
                        acc.y = fmaf(w, v[j].y, acc.y);
                        acc.z = fmaf(w, v[j].z, acc.z);
                        acc.w = fmaf(w, v[j].w, acc.w);
                    }
                }
            }
        }
        if constexpr (kZ > 1) {
            __shared__ float2 s_stat[kMergeThreads];
            __shared__ float4 s_acc[kMergeThreads];
            s_stat[threadIdx.x] = make_float2(top, sum);
            s_acc[threadIdx.x] = acc;
            __syncthreads();
            if (z == 0) {
#pragma unroll
                for (int j = 1; j < kZ; ++j) {
                    const float2 st = s_stat[threadIdx.x + j * kRows * kCols];
                    const float4 v = s_acc[threadIdx.x + j * kRows * kCols];
                    const float next = fmaxf(top, st.x), ref = next == -INFINITY ? 0.f : next;
                    const float f = ptx::ex2_approx(top - ref), w = ptx::ex2_approx(st.x - ref);
                    top = next;
                    sum = sum * f + w * st.y;
                    acc.x = acc.x * f + w * v.x;
                    acc.y = acc.y * f + w * v.y;
                    acc.z = acc.z * f + w * v.z;
                    acc.w = acc.w * f + w * v.w;
                }
            }
            __syncthreads();
        }
        if (z != 0 || skip || c >= p.D / 4) continue;
        const bool empty = sum == 0.f;
        const float inv = empty ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(p.o + b * p.o_s[0] + hq * p.o_s[1] + t * p.o_s[2] + 4 * c) =
            empty ? make_uint2(0u, 0u)
                  : make_uint2(ptx::pack16x2<kF16>(acc.x * inv, acc.y * inv), ptx::pack16x2<kF16>(acc.z * inv, acc.w * inv));
        if (p.lse && c == 0) p.lse[((int64_t)b * p.Hq + hq) * p.T + t] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

template <int kCols, int kZ>
cudaError_t launch_merge(const MergeParams &p, cudaStream_t stream)
{
    constexpr int kRows = kMergeThreads / (kCols * kZ);
    const int groups = (p.G * p.T + kRows - 1) / kRows;
    const dim3 grid((unsigned)(p.B * groups), (unsigned)(p.Hq / p.G));
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

// 16 rows where they hold the tile or where D = 256 leaves no registers for
// more, else 32.
int paged_rows_per_tile(int D, int64_t rows) { return rows <= 16 || D > 128 ? 16 : 32; }

int paged_rows_chunk(int D) { return D <= 64 ? RowsLayout<64, 1>::kChunk : D <= 128 ? RowsLayout<128, 1>::kChunk : RowsLayout<256, 1>::kChunk; }

int paged_rows_ctas_per_sm(int D) { return D > 128 ? 1 : 2; }

cudaError_t launch_paged_rows(const PagedParams &p, int ctas, cudaStream_t stream)
{
    if (p.c.D > 128) return launch_rows_f<256, 1>(p, ctas, stream);
    if (p.c.D > 64)
        return p.part.rows == 16 ? launch_rows_f<128, 1>(p, ctas, stream) : launch_rows_f<128, 2>(p, ctas, stream);
    return p.part.rows == 16 ? launch_rows_f<64, 1>(p, ctas, stream) : launch_rows_f<64, 2>(p, ctas, stream);
}

cudaError_t launch_paged_merge(const MergeParams &p, int states, int sms, cudaStream_t stream)
{
    // Threads per column that share a row's states: as many as leave each two
    // or more, while the launch stays within one wave of CTAs.
    const int cols = p.D <= 64 ? 16 : 32;
    int z = 1;
    while (z < 8 && 4 * z <= states) {
        const int rows = kMergeThreads / (cols * 2 * z);
        if ((int64_t)p.B * ((p.G * p.T + rows - 1) / rows) * (p.Hq / p.G) > 4 * sms) break;
        z *= 2;
    }
    return p.D <= 64 ? launch_merge_z<16>(p, z, stream) : launch_merge_z<32>(p, z, stream);
}

}  // namespace fa
