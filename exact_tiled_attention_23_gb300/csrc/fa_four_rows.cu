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
#include "fa_four.cuh"
#include "fa_four_rows.h"
#include "fa_paged_line.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr float kLn2 = 0.69314718055994530942f;

// Weights are p = 2^(s - m); m is raised where a score lies 2^(kLift + kRise) above
// it, to 2^kLift below the largest one then: halves are multiples of 2^-24, so that a
// weight is off by 2^-37 of the row's largest at most, where not by half a step.
constexpr float kLift = 12.f, kRise = 3.f;

template <int DP, int J>
struct FourLayout {
    static constexpr int kWarps = kRowsWarps;
    static constexpr int kRows = 8 * J;
    static constexpr int kChunk = DP == 256 ? 16 : 32;            // keys of a step
    static constexpr int kRowBytes = DP / 2, kScaleBytes = DP / 16;
    static constexpr int kTileBytes = kChunk * kRowBytes;         // K or V of a step
    static constexpr int kScales = 2 * kTileBytes;                // where the scales are
    static constexpr int kStageBytes = 2 * kTileBytes + 2 * kChunk * kScaleBytes;
    static constexpr int kStages = DP == 64 ? 4 : 3;
    // what registers and shared memory hold
    static constexpr int kCtas = DP == 128 && J == 2 ? 4 : DP == 256 || J == 2 ? 5 : 8;
    static constexpr int kMaskOff = kWarps * kStages * kStageBytes;
    static constexpr int kSmemBytes = kMaskOff + kWarps * kStages * 4;
    static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory per SM");
    static_assert(kStageBytes % 16 == 0 && kTileBytes % 16 == 0, "alignment");
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

__device__ __forceinline__ uint32_t shared32(uint32_t at)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t shared16(uint32_t at)
{
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t shared8(uint32_t at)
{
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
    return r;
}
template <int kWords>
__device__ __forceinline__ void shared_words(uint32_t at, uint32_t *w)
{
    if constexpr (kWords == 1)
        w[0] = shared32(at);
    else if constexpr (kWords == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t scale)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&scale));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// A chunk's rows are in this order as the products' rows, by eights, so that a
// matrix load's lanes find their banks free: 0 5 1 4 2 7 3 6.
__device__ __forceinline__ int key_of_row(int r) { return r & 1 ? 4 + ((r >> 1) ^ 1) : r >> 1; }

template <int DP, int J, bool kF16, bool kOnePage>
__global__ void __launch_bounds__((32 * FourLayout<DP, J>::kWarps), (FourLayout<DP, J>::kCtas))
four_rows_kernel(const FourParams f)
{
    using Lay = FourLayout<DP, J>;
    constexpr int S = Lay::kStages, KS = Lay::kChunk, RM = Lay::kRows, KJ = KS / 16;
    constexpr bool kTwo = kF16;                     // weights of two halves
    constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : 0xffffu;
    constexpr int kUnits = DP == 256 ? 2 : 1;       // of a lane's elements of a key
    constexpr int kWords = DP == 64 ? 2 : 4;        // of a unit
    constexpr int KT = DP / 16;                     // 16-column steps of a score, tiles of O
    constexpr int kVWords = DP / 64;                // of a lane's elements of a value
    extern __shared__ __align__(16) uint8_t smem[];
    const PagedParams &p = f.p;
    const PagedCache4 &c = f.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = ptx::smem_u32(smem) + warp * S * Lay::kStageBytes;
    uint32_t *s_mask = reinterpret_cast<uint32_t *>(smem + Lay::kMaskOff) + warp * S;
    ptx::wait_for_primary();
    ptx::launch_dependents();
    Line<KS, kRowsTile> line(p);
    const int piece = (int)blockIdx.x * Lay::kWarps + warp;
    LineCursor at;
    int units, used, per;       // of the piece, those in front of `at`, a full piece's
    line.share(piece, (int)gridDim.x * Lay::kWarps, at, used, units, per);
    units += used;
    const int R = line.R;

    // ---- loads -----------------------------------------------------------
    LineCursor ld = at;
    int ld_left = units - used;
    // Where this lane's key of a step is (lane % KS).  Its page number is fetched at
    // least one step before its use.
    struct Place {
        int page, slot, h;      // page < 0: not a key that the tile sees; h < 0: past the piece
    };
    auto look_up = [&]() -> Place {
        if (ld_left <= 0) return Place{-1, 0, -1};
        Place x{-1, 0, ld.h};
        const int key = ld.c * KS + lane % KS;
        if (key < ld.keys) {
            const int which = p.c.by_page.quotient(key);
            const int b = p.part.tiles == 1 ? ld.g : ld.g / p.part.tiles;
            x.slot = key - which * p.c.page_size;
            x.page = p.c.table[(int64_t)b * p.c.table_stride + which];
        }
        ld_left -= ld.c ? 1 : 1 + line.weight;
        line.advance(ld);
        return x;
    };
    auto load = [&](int stage, const Place &x) {
        const bool ok = x.page >= 0 && x.page < p.c.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAll;
        if (lane == 0) s_mask[stage] = mask;
        const uint32_t dst = ring + stage * Lay::kStageBytes;
        constexpr int kLanes = Lay::kRowBytes / 16, kPer = 32 / kLanes;     // lanes per row, rows at a time
        const int unit = lane % kLanes;
        if (x.h < 0) {
            ptx::cp_async_commit();
            return;
        }
        int64_t off = 0, scale = 0;
        if (ok) {
            off = x.page * c.s_page + x.h * c.s_head + x.slot * c.s_slot;
            scale = x.page * c.t_page + x.h * c.t_head + x.slot * c.t_slot;
        }
        int64_t first = 0;
        if constexpr (kOnePage) first = __shfl_sync(0xffffffffu, off, 0);
#pragma unroll
        for (int i = 0; i < KS / kPer; ++i) {
            const int row = i * kPer + lane / kLanes;
            const bool on = (mask >> row) & 1u;
            int64_t o;
            if constexpr (kOnePage)
                o = first + row * c.s_slot;
            else
                o = __shfl_sync(0xffffffffu, off, row);
            o = on ? o + unit * 16 : 0;
            const uint32_t to = dst + row * Lay::kRowBytes + unit * 16;
            copy_async<16>(to, c.k + o, on);
            copy_async<16>(to + Lay::kTileBytes, c.v + o, on);
        }
        if (lane < KS) {
            const uint32_t to = dst + Lay::kScales + lane * Lay::kScaleBytes;
            copy_async<Lay::kScaleBytes>(to, c.ks + scale, ok);
            copy_async<Lay::kScaleBytes>(to + KS * Lay::kScaleBytes, c.vs + scale, ok);
        }
        ptx::cp_async_commit();
    };
    Place next = look_up();
#pragma unroll 1
    for (int s = 0; s < S; ++s) {
        const Place x = next;
        next = look_up();
        load(s, x);
    }

    // ---- the piece, tile by tile -------------------------------------------
    const int qr = lane >> 2, qc = lane & 3;        // this lane's row (and + 8) and columns (2 qc, + 1) of a product
    const int k_row = key_of_row(qr), v_first = key_of_row(2 * qc), v_second = key_of_row(2 * qc + 1);
    int stage = 0;
#pragma unroll 1
    while (used < units) {
        const int rest = units - used;
        const int count = min(at.n - at.c, line.chunks_within(at.c, rest));
        const int b = p.part.tiles == 1 ? at.g : at.g / p.part.tiles;
        const int row0 = (at.g - b * p.part.tiles) * RM, h = at.h;
        const int tile = at.g * p.c.Hkv + h;
        if (at.c == 0 && lane == 0) line.record(at, piece, used, per);
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
                int up = 127 + 14 - (int)(__float_as_uint(largest) >> 23);
                up = largest == 0.f ? 0 : max(-112, min(up, 100));
                const float by = __uint_as_float((uint32_t)(127 + up) << 23);
                mine = __uint_as_float((uint32_t)(127 - up) << 23);
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

#pragma unroll 1
        for (int step = 0; step < count; ++step) {
            ptx::cp_async_wait<S - 1>();
            __syncwarp();
            const uint32_t mask = s_mask[stage];
            const uint32_t kt = ring + stage * Lay::kStageBytes, ks = kt + Lay::kScales;
            const uint32_t vt = kt + Lay::kTileBytes, vs = ks + KS * Lay::kScaleBytes;
            const int key0 = (at.c + step) * KS;
            if (mask) {
                // scores of keys 16 j + k_row (and + 8) and the rows 2 qc, + 1
                float s[J][KJ][4];
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
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
                            shared_words<kWords>(kt + row * Lay::kRowBytes + u * 64 + qc * (4 * kWords), w[e]);
                            if constexpr (DP == 64) {
                                sc[e][0] = shared8(ks + row * Lay::kScaleBytes + qc) * 0x800080u;
                            } else {
                                const uint32_t two = shared16(ks + row * Lay::kScaleBytes + u * 8 + 2 * qc);
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
                }
                if (mask != kAll || key0 + KS > lim_all) {
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
                uint32_t hi[J][KJ][2], lo[J][KJ][2];
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
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    // keys 16 j + v_first, + v_second, and 8 further
                    uint32_t w[2][2][kVWords], sc[2][2];
#pragma unroll
                    for (int a = 0; a < 2; ++a)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 16 * j + 8 * a + (e ? v_second : v_first);
                            shared_words<kVWords>(vt + row * Lay::kRowBytes + qr * (4 * kVWords), w[a][e]);
                            if constexpr (DP == 256)
                                sc[a][e] = shared16(vs + row * Lay::kScaleBytes + 2 * qr);
                            else
                                sc[a][e] = shared8(vs + row * Lay::kScaleBytes + (DP == 64 ? qr / 2 : qr));
                        }
#pragma unroll
                    for (int i = 0; i < kVWords; ++i) {
                        uint32_t x[2][2][4];        // [keys][even and odd columns]
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            uint32_t both = 0;      // the two keys' scales
                            if constexpr (DP == 256)
                                both = i < 2 ? ((sc[a][0] & 0xffu) | (sc[a][1] & 0xffu) << 16) << 7
                                             : ((sc[a][0] >> 8) | (sc[a][1] >> 8) << 16) << 7;
                            else
                                both = (sc[a][0] | sc[a][1] << 16) << 7;
                            const uint32_t even = (w[a][0][i] & 0x0f0f0f0fu) | ((w[a][1][i] << 4) & 0xf0f0f0f0u);
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
                }
            }
            __syncwarp();
            const Place x = next;
            next = look_up();
            load(stage, x);
            if (++stage == S) stage = 0;
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
    ptx::cp_async_wait<0>();
}

template <int DP, int J, bool kF16, bool kOnePage>
cudaError_t launch_one(const FourParams &f, int ctas, cudaStream_t stream)
{
    using Lay = FourLayout<DP, J>;
    static SharedMemory allowed;
    const cudaError_t e = allowed.allow(four_rows_kernel<DP, J, kF16, kOnePage>, Lay::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_behind(four_rows_kernel<DP, J, kF16, kOnePage>, dim3((unsigned)ctas), 32 * Lay::kWarps, Lay::kSmemBytes, stream, f);
}

template <int DP, int J>
cudaError_t launch_rows(const FourParams &f, int ctas, cudaStream_t stream)
{
    // a chunk within one page: its rows' addresses are a step apart
    if (f.p.c.page_size % FourLayout<DP, J>::kChunk == 0)
        return f.p.f16 ? launch_one<DP, J, true, true>(f, ctas, stream) : launch_one<DP, J, false, true>(f, ctas, stream);
    return f.p.f16 ? launch_one<DP, J, true, false>(f, ctas, stream) : launch_one<DP, J, false, false>(f, ctas, stream);
}

}  // namespace

int four_rows_per_tile(int D, int64_t rows) { return rows <= 8 || D > 128 ? 8 : 16; }

int four_rows_chunk(int D) { return D > 128 ? FourLayout<256, 1>::kChunk : FourLayout<128, 1>::kChunk; }

int four_rows_ctas_per_sm(int D, int rows)
{
    return D > 128 ? FourLayout<256, 1>::kCtas : rows == 8 ? FourLayout<128, 1>::kCtas : FourLayout<128, 2>::kCtas;
}

cudaError_t launch_four_rows(const FourParams &f, int ctas, cudaStream_t stream)
{
    if (f.p.c.D > 128) return launch_rows<256, 1>(f, ctas, stream);
    if (f.p.c.D > 64) return f.p.part.rows == 8 ? launch_rows<128, 1>(f, ctas, stream) : launch_rows<128, 2>(f, ctas, stream);
    return f.p.part.rows == 8 ? launch_rows<64, 1>(f, ctas, stream) : launch_rows<64, 2>(f, ctas, stream);
}

// ------------------------------------------------- whole pages as 16-bit rows
namespace {

constexpr int kWideThreads = 256;

// Pages of the sequences of a call as 16-bit pages of their own, page j of sequence
// b as page b * width + j, and the tables and lengths that go with them.  A CTA per
// page; a thread takes 8 elements of a key and of a value.
template <bool kF16>
__global__ void __launch_bounds__(kWideThreads) widen_pages_kernel(const WidenParams p)
{
    ptx::wait_for_primary();
    const PagedCache4 &c = p.c;
    const int b = blockIdx.x / (unsigned)c.table_width, j = blockIdx.x - b * c.table_width;
    const int64_t cap = (int64_t)c.table_width * c.page_size;
    const int n = c.seq_len[b] < 0 ? 0 : (int)min((int64_t)c.seq_len[b], cap);
    if (j == 0 && threadIdx.x == 0) p.seq_len[b] = n;
    const int slots = min(c.page_size, n - j * c.page_size);
    if (slots <= 0) return;                                 // (its entry is not read)
    const int page = c.table[b * c.table_stride + j];
    const bool there = page >= 0 && page < c.num_pages;
    if (threadIdx.x == 0) p.table[blockIdx.x] = there ? (int)blockIdx.x : -1;
    if (!there) return;
    const int units = c.D / 8;
    const int64_t to = (int64_t)blockIdx.x * c.Hkv * c.page_size * c.D;
    for (int e = threadIdx.x; e < c.Hkv * slots * units; e += kWideThreads) {
        const int row = e / units, u = e - row * units, head = row / slots, slot = row - head * slots;
        const int64_t from = page * c.s_page + head * c.s_head + slot * c.s_slot + 4 * u;
        const int64_t scale = page * c.t_page + head * c.t_head + slot * c.t_slot + u / 2;
        const int64_t dst = to + ((int64_t)head * c.page_size + slot) * c.D + 8 * u;
        *reinterpret_cast<uint4 *>(p.k + dst) = rows_from_four<kF16>(*reinterpret_cast<const uint32_t *>(c.k + from), c.ks[scale]);
        *reinterpret_cast<uint4 *>(p.v + dst) = rows_from_four<kF16>(*reinterpret_cast<const uint32_t *>(c.v + from), c.vs[scale]);
    }
}

}  // namespace

cudaError_t launch_widen_pages(const WidenParams &p, int64_t pages, cudaStream_t stream)
{
    return p.f16 ? launch_behind(widen_pages_kernel<true>, dim3((unsigned)pages), kWideThreads, 0, stream, p)
                 : launch_behind(widen_pages_kernel<false>, dim3((unsigned)pages), kWideThreads, 0, stream, p);
}

}  // namespace fa
