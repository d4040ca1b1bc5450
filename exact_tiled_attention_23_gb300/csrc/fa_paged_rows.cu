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
constexpr int kStepKeys = 16;                      // keys of a warp per step
static_assert(kChunkKeys == kWarps * kStepKeys, "one step of every warp per chunk");
constexpr float kLn2 = 0.69314718055994530942f;

template <int DP, int MT>
struct RowsLayout {
    static constexpr int kRows = 16 * MT;
    static constexpr int kRowBytes = 2 * DP;
    static constexpr int kTileBytes = kStepKeys * kRowBytes;      // K or V of a step
    static constexpr int kStageBytes = 2 * kTileBytes;
    // as many stages as 96 KB hold (two CTAs per SM), three at D = 256 (one CTA)
    static constexpr int kStages = DP == 64 ? 6 : 3;
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = kRows * kRowBytes;
    static constexpr int kStatOff = kRingOff + kWarps * kStages * kStageBytes;
    static constexpr int kStatBytes = 2 * kWarps * kRows * 4;     // m and l of every warp
    static constexpr int kMaskOff = kStatOff + kStatBytes;        // valid keys of every stage
    static constexpr int kScanOff = kMaskOff + kWarps * kStages * 4;
    static constexpr int kSmemBytes = kScanOff + 128;
    static_assert((kWarps + 2) * 8 <= 128, "scratch of the line's share");
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
    constexpr int S = Lay::kStages, RM = Lay::kRows, RB = Lay::kRowBytes;
    constexpr int NT = DP / 8;                      // 8-column tiles of O
    constexpr int KT = DP / 16;                     // 16-column steps of a score
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t s_base = ptx::smem_u32(smem);
    float *s_m = reinterpret_cast<float *>(smem + Lay::kStatOff);
    float *s_l = s_m + kWarps * RM;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + Lay::kMaskOff);
    int64_t *s_scan = reinterpret_cast<int64_t *>(smem + Lay::kScanOff);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Line<kChunkKeys> line(p);
    LineCursor at;
    int64_t g0;
    int steps;
    line.share<kThreads>(s_scan, at, g0, steps);
    if (steps == 0) return;
    const int R = line.R;

    // ---- loads -----------------------------------------------------------
    const int kr = lane & 15;                       // the key of the step whose address this lane finds
    LineCursor ld = at;
    int ld_left = steps;
    // The page number of a step's key is fetched one step before its use.
    int pg = -1, pg_slot = 0, pg_head = 0;
    auto look_up = [&] {
        pg = -1;
        if (ld_left <= 0) return;
        const int key = ld.c * kChunkKeys + warp * kStepKeys + kr;
        pg_head = ld.h;
        if (key < ld.keys) {
            const uint32_t which = (uint32_t)key / (uint32_t)p.c.page_size;
            pg_slot = key - (int)which * p.c.page_size;
            pg = p.c.table[(int64_t)(ld.g / p.part.tiles) * p.c.table_stride + which];
        }
        line.advance(ld);
        --ld_left;
    };
    const uint32_t ring = s_base + Lay::kRingOff + warp * S * Lay::kStageBytes;
    auto load = [&](int stage) {
        const bool ok = pg >= 0 && pg < p.c.num_pages;
        const int64_t off = ok ? (int64_t)pg * p.c.s_page + (int64_t)pg_head * p.c.s_head + (int64_t)pg_slot * p.c.s_slot : 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
        if (lane == 0) s_mask[warp * S + stage] = mask;
        look_up();
        constexpr int kLanes = DP / 8 < 32 ? DP / 8 : 32;      // lanes per row
        constexpr int kRowsPer = 32 / kLanes;
        const int unit = lane % kLanes;
        const uint32_t dst = ring + stage * Lay::kStageBytes;
#pragma unroll
        for (int i = 0; i < kStepKeys / kRowsPer; ++i) {
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
    look_up();
#pragma unroll
    for (int s = 0; s < S; ++s) load(s);            // steps past the share load zeros

    // ---- the share, tile by tile ------------------------------------------
    const int qr = lane >> 2, qc = lane & 3;        // this lane's rows (qr, qr + 8) and columns (2 qc, +1) of a tile
    const uint32_t q_smem = s_base + Lay::kQOff;
    int stage = 0, done = 0;
    while (done < steps) {
        const int count = min(at.n - at.c, steps - done);      // chunks of this tile in the share
        const int b = at.g / p.part.tiles, row0 = (at.g - b * p.part.tiles) * RM, h = at.h;
        const int64_t tile = (int64_t)at.g * p.c.Hkv + h;
        const bool whole = count == at.n;
        if (at.c == 0 && tid == 0) p.part.first_chunk[tile] = g0 + done;
        // Q rows of the tile; rows past R and columns past D are zero
        for (int e = tid; e < RM * (DP / 8); e += kThreads) {
            const int row = e / (DP / 8), unit = e % (DP / 8);
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (row0 + row < R && unit * 8 < p.c.D) {
                const RowPlace r = row_place(p, b, h, row0 + row);
                w = *reinterpret_cast<const uint4 *>(p.q + r.b * p.q_s[0] + r.hq * p.q_s[1] + r.t * p.q_s[2] + unit * 8);
            }
            ptx::st_shared_v4(q_smem + unit_at<RB>(row, unit), w.x, w.y, w.z, w.w);
        }
        int lim[2 * MT];                            // keys that this lane's rows see
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int t = (row0 + i * 8 + qr) / p.G;
            lim[i] = line.masked ? at.len - p.T + t + 1 : at.len;
        }
        const int lim_all = line.masked ? at.len - p.T + row0 / p.G + 1 : at.len;   // seen by every row
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
            const int key0 = (at.c + step) * kChunkKeys + warp * kStepKeys;
            if (mask) {
                float s[MT][2][4];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < KT; ++k) {
                    // K rows 0-7 and 8-15, columns 16k .. +7 and +8 .. +15
                    uint32_t kb[4];
                    ptx::ldmatrix4(kb, kt + unit_at<RB>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t qa[4];
                        ptx::ldmatrix4(qa, q_smem + unit_at<RB>(i * 16 + (lane & 15), 2 * k + (lane >> 4)));
                        ptx::mma_16816<kF16>(s[i][0], qa, kb[0], kb[1]);
                        ptx::mma_16816<kF16>(s[i][1], qa, kb[2], kb[3]);
                    }
                }
                if (mask != 0xffffu || key0 + kStepKeys > lim_all) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int key = n * 8 + 2 * qc + (e & 1);
                                if (!((mask >> key) & 1u) || key0 + key >= lim[2 * i + (e >> 1)]) s[i][n][e] = -INFINITY;
                            }
                }
                uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float &mr = m[2 * i + r], &lr = l[2 * i + r];
                        float mx = fmaxf(fmaxf(s[i][0][2 * r], s[i][0][2 * r + 1]), fmaxf(s[i][1][2 * r], s[i][1][2 * r + 1]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float m_new = fmaxf(mr, mx * p.scale_log2);
                        const float ref = m_new == -INFINITY ? 0.f : m_new;
                        const float alpha = ptx::ex2_approx(mr - ref);
                        if (__any_sync(0xffffffffu, m_new != mr)) {
                            lr *= alpha;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[i][n][2 * r] *= alpha;
                                o[i][n][2 * r + 1] *= alpha;
                            }
                        }
                        mr = m_new;
                        float pv[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pv[e] = ptx::ex2_approx(fmaf(s[i][e >> 1][2 * r + (e & 1)], p.scale_log2, -ref));
                            lr += pv[e];
                        }
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const uint32_t w = ptx::pack16x2<kF16>(pv[2 * n], pv[2 * n + 1]);
                            float r0, r1;
                            ptx::unpack2(ptx::widen16x2<kF16>(w), r0, r1);
                            hi[i][2 * n + r] = w;
                            lo[i][2 * n + r] = ptx::pack16x2<kF16>(pv[2 * n] - r0, pv[2 * n + 1] - r1);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < KT; ++n) {
                    // V rows 0-7 and 8-15 (the product's k), columns 16n .. +7 and +8 .. +15
                    uint32_t vb[4];
                    ptx::ldmatrix4_trans(vb, vt + unit_at<RB>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        ptx::mma_16816<kF16>(o[i][2 * n], hi[i], vb[0], vb[1]);
                        ptx::mma_16816<kF16>(o[i][2 * n + 1], hi[i], vb[2], vb[3]);
                        ptx::mma_16816<kF16>(o[i][2 * n], lo[i], vb[0], vb[1]);
                        ptx::mma_16816<kF16>(o[i][2 * n + 1], lo[i], vb[2], vb[3]);
                    }
                }
            }
            __syncwarp();
            last_stage = stage;
            stage = stage + 1 == S ? 0 : stage + 1;
            // the tile's last stage is refilled after the warps' states are joined
            if (step + 1 < count) load(last_stage);
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
                const int row = e / (DP / 4), col = (e % (DP / 4)) * 4;
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
                        *reinterpret_cast<float4 *>(p.part.o + (slot * RM + tr) * p.c.D + col) =
                            make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (col == 0) p.part.lse[slot * RM + tr] = lse2;
                }
            }
            __syncthreads();
        }
        load(last_stage);
        at.c += count - 1;
        line.advance(at);
        done += count;
    }
    ptx::cp_async_wait<0>();
}

template <int DP, int MT, bool kF16>
cudaError_t launch_rows(const PagedParams &p, int ctas, cudaStream_t stream)
{
    // per call: the attribute belongs to the current device
    const cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<DP, MT, kF16>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               RowsLayout<DP, MT>::kSmemBytes);
    if (e != cudaSuccess) return e;
    paged_rows_kernel<DP, MT, kF16><<<ctas, kThreads, RowsLayout<DP, MT>::kSmemBytes, stream>>>(p);
    return cudaGetLastError();
}

template <int DP, int MT>
cudaError_t launch_rows_f(const PagedParams &p, int ctas, cudaStream_t stream)
{
    return p.f16 ? launch_rows<DP, MT, true>(p, ctas, stream) : launch_rows<DP, MT, false>(p, ctas, stream);
}

// ---------------------------------------------------------------- merge
// One warp per query row: the largest LSE of the row's partial states, their
// weights, and the weighted sum of their outputs, in the order of the slots.
// Lane i holds columns 4 i .. 4 i + 3 (and 128 + 4 i .. at D = 256).
template <bool kF16>
__global__ void __launch_bounds__(128) paged_merge_kernel(const MergeParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)p.B * p.Hq * p.T) return;
    const int t = (int)(row % p.T);
    const int hq = (int)(row / p.T % p.Hq);
    const int b = (int)(row / ((int64_t)p.T * p.Hq));
    const int h = hq / p.G;
    int len = p.seq_len[b];
    len = len < 0 ? 0 : (len > p.max_len ? p.max_len : len);
    const bool padding = p.causal && len - p.T + t < 0;        // no token here

    int64_t slot0[2];
    int count[2], tr[2];
    for (int s = 0; s < 2; ++s) {
        slot0[s] = 0;
        count[s] = tr[s] = 0;
        if (s >= p.n_src || padding) continue;
        const Partials &src = p.src[s];
        const int idx = t * p.G + hq % p.G + (src.stacked ? b * p.G * p.T : 0);
        const int rt = idx / src.rows;
        tr[s] = idx - rt * src.rows;
        const int64_t tile = ((int64_t)(src.stacked ? 0 : b) * src.tiles + rt) * (p.Hq / p.G) + h;
        const int chunks = chunks_of(
            keys_of_tile(src.stacked ? src.fixed_len : len, rt, src.rows, p.G * p.T, p.G, p.T, p.causal && !src.stacked),
            src.chunk);
        if (chunks == 0) continue;
        const int64_t per = *src.per_cta, c0 = src.first_chunk[tile];
        const int64_t k0 = c0 / per, k1 = (c0 + chunks - 1) / per;
        slot0[s] = k0 + tile;
        count[s] = (int)(k1 - k0 + 1);
    }
    // one CTA had the whole tile and wrote the row itself
    if (!p.joined && count[0] == 1) return;

    float top = -INFINITY;
    for (int s = 0; s < p.n_src; ++s)
        for (int i = lane; i < count[s]; i += 32)
            top = fmaxf(top, p.src[s].lse[(slot0[s] + i) * p.src[s].rows + tr[s]]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float ref = top == -INFINITY ? 0.f : top;

    float sum = 0.f, acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int s = 0; s < p.n_src; ++s) {
        const Partials &src = p.src[s];
        for (int i = 0; i < count[s]; ++i) {
            const int64_t at = (slot0[s] + i) * src.rows + tr[s];
            const float w = ptx::ex2_approx(src.lse[at] - ref);
            sum += w;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = c * 128 + lane * 4;
                if (col >= p.D) continue;
                const float4 v = *reinterpret_cast<const float4 *>(src.o + at * p.D + col);
                acc[c][0] = fmaf(w, v.x, acc[c][0]);
                acc[c][1] = fmaf(w, v.y, acc[c][1]);
                acc[c][2] = fmaf(w, v.z, acc[c][2]);
                acc[c][3] = fmaf(w, v.w, acc[c][3]);
            }
        }
    }
    const bool empty = sum == 0.f;
    const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int col = c * 128 + lane * 4;
        if (col >= p.D) continue;
        *reinterpret_cast<uint2 *>(p.o + b * p.o_s[0] + hq * p.o_s[1] + t * p.o_s[2] + col) =
            empty ? make_uint2(0u, 0u)
                  : make_uint2(ptx::pack16x2<kF16>(acc[c][0] * inv, acc[c][1] * inv),
                               ptx::pack16x2<kF16>(acc[c][2] * inv, acc[c][3] * inv));
    }
    if (p.lse && lane == 0) p.lse[row] = empty ? -INFINITY : (top + log2f(sum)) * kLn2;
}

}  // namespace

// 16 rows where they hold the tile or where D = 256 leaves no registers for
// more, else 32.
int paged_rows_per_tile(int D, int64_t rows) { return rows <= 16 || D > 128 ? 16 : 32; }

int paged_rows_ctas_per_sm(int D) { return D > 128 ? 1 : 2; }

cudaError_t launch_paged_rows(const PagedParams &p, int ctas, cudaStream_t stream)
{
    if (p.c.D > 128) return launch_rows_f<256, 1>(p, ctas, stream);
    if (p.c.D > 64)
        return p.part.rows == 16 ? launch_rows_f<128, 1>(p, ctas, stream) : launch_rows_f<128, 2>(p, ctas, stream);
    return p.part.rows == 16 ? launch_rows_f<64, 1>(p, ctas, stream) : launch_rows_f<64, 2>(p, ctas, stream);
}

cudaError_t launch_paged_merge(const MergeParams &p, cudaStream_t stream)
{
    const int64_t rows = (int64_t)p.B * p.Hq * p.T;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (p.f16)
        paged_merge_kernel<true><<<grid, 128, 0, stream>>>(p);
    else
        paged_merge_kernel<false><<<grid, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
