// fa_append.cu -- keys and values of new tokens into a paged cache, with the
// position rotation of keys and queries applied on the way.
//
// Token t of sequence b has the index i = seq_len[b] - T + t and the position
// n = offset + i.  Pair p of its key (and query) head, (x, y), turns by the
// angle a = n * inv_freq[p]:
//     x' = x cos a - y sin a,    y' = y cos a + x sin a,
// and the key and value go to slot i % page_size of page table[b][i / page_size].
//
// A far position times a frequency loses its angle in fp32 (a product of 10^5
// is good to 2^-7 radians), so the angle is kept as a fraction of a turn in 64
// bits: inv_freq[p] / 2pi as a fixed-point number F of 2^-64 turns, and n * F
// modulo 2^64 drops whole turns exactly.  F comes from 128 bits of 1 / 2pi, so it
// is off by less than its last bit for every frequency up to 2^16, and the angle
// by n 2^-64 turns: 2^-33 at n = 2^31, where the fp32 form's 2^-26 decides, and
// 2^-24 at the farthest position, 2^40 + 2^31.
//
// Bound by memory: every value is read once and written once, whole 16-byte units
// at a time.  One CTA per token, so that a token's angles are computed once for all
// heads.  Two prompts of 8192 tokens, 32 query and 8 key heads, D = 128: 403 MB in
// 62 us, 6.5 TB/s (a copy: 6.8).  One token: 3 us, a launch and four waits in turn
// (length, page, values, stores).
#include "fa_paged.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;

// 2^128 / (2 pi): the bits of 1 / (2 pi) after the binary point.
constexpr uint64_t kInvTwoPiHi = 0x28be60db9391054aull, kInvTwoPiLo = 0x7f09d5f47d4d3770ull;

// cos and sin of n * f radians, for |f| <= 65536.
__device__ __forceinline__ float2 turn(int64_t n, float f)
{
    const float a = fabsf(f);
    if (!(a <= 65536.f)) return make_float2(NAN, NAN);
    const uint32_t bits = __float_as_uint(a);
    const int e = (int)(bits >> 23);                       // a = m * 2^(e - 150)
    const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : 0u;
    const int shift = 150 - e;                             // >= 6 for a <= 2^16
    // bits 64 .. 191 of m * (2^128 / 2 pi)
    const uint64_t part = m * kInvTwoPiHi, lo = part + __umul64hi(m, kInvTwoPiLo);
    const uint64_t hi = __umul64hi(m, kInvTwoPiHi) + (lo < part ? 1 : 0);
    const uint64_t F = shift < 64 ? (lo >> shift) | (hi << (64 - shift)) : shift < 128 ? hi >> (shift - 64) : 0ull;
    const uint64_t frac = (uint64_t)n * F;                 // modulo one turn
    // to [-1/2, 1/2) turns; sincospif takes half turns
    const float half_turns = __ll2float_rn((int64_t)frac) * 1.0842021724855044e-19f;   // 2^-63
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c, f < 0.f ? -s : s);
}

template <bool kF16>
__device__ __forceinline__ void widen8(const uint4 &w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::unpack2(ptx::widen16x2<kF16>(u[i]), x[2 * i], x[2 * i + 1]);
}

template <bool kF16>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8])
{
    return make_uint4(ptx::pack16x2<kF16>(x[0], x[1]), ptx::pack16x2<kF16>(x[2], x[3]),
                      ptx::pack16x2<kF16>(x[4], x[5]), ptx::pack16x2<kF16>(x[6], x[7]));
}

template <bool kF16>
__device__ __forceinline__ float widen1(uint16_t w)
{
    float lo, hi;
    ptx::unpack2(ptx::widen16x2<kF16>(w), lo, hi);
    return lo;
}

// How the pairs of a head lie: neighbours (2p, 2p+1), also used without a
// rotation; (p, p + rot/2) with rot a multiple of 16, so that 8 pairs are two
// 16-byte units; the same with any even rot.
enum PairMode { kNeighbours = 0, kHalves = 1, kHalvesOdd = 2 };

// One CTA per token: its cosines and sines are computed once for all heads,
// then each thread moves 16-byte units of q, k and v.
template <bool kF16, int kMode>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    extern __shared__ float2 cs[];                          // [rot / 2]
    ptx::wait_for_primary();
    const int64_t b = blockIdx.x / p.T;
    const int t = (int)(blockIdx.x % p.T);
    const int i = max(p.c.seq_len[b], -1) - p.T + t;        // (-1 - T at least: no overflow)
    const int half = p.rot / 2, D = p.c.D, Hkv = p.c.Hkv;
    const int units = D / 8;

    if (i < 0) {                                            // no token here: its query is zero
        if (p.q)
            for (int e = threadIdx.x; e < p.Hq * units; e += kThreads)
                *reinterpret_cast<uint4 *>(p.q_out + b * p.qo_s[0] + (e / units) * p.qo_s[1] + t * p.qo_s[2] +
                                           (e % units) * 8) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const uint32_t at = (uint32_t)i, size = (uint32_t)p.c.page_size;
    int page = -1;
    if (at / size < (uint32_t)p.c.table_width) page = p.c.table[b * p.c.table_stride + at / size];
    const bool stored = page >= 0 && page < p.c.num_pages;   // otherwise the key and value are dropped
    const int64_t row = stored ? page * p.c.s_page + (int64_t)(at % size) * p.c.s_slot : 0;
    for (int j = threadIdx.x; j < half; j += kThreads) cs[j] = turn(p.offset + i, p.inv_freq[j]);
    __syncthreads();

    // heads 0 .. Hkv-1: keys; Hkv .. Hkv+Hq-1: queries; then values
    const int q_heads = p.q ? p.Hq : 0;
    const int k_heads = stored ? Hkv : 0;
    const auto source = [&](int head) -> const uint16_t * {
        if (head < k_heads) return p.k + b * p.k_s[0] + head * p.k_s[1] + t * p.k_s[2];
        return p.q + b * p.q_s[0] + (head - k_heads) * p.q_s[1] + t * p.q_s[2];
    };
    const auto target = [&](int head) -> uint16_t * {
        if (head < k_heads) return p.c.k + row + head * p.c.s_head;
        return p.q_out + b * p.qo_s[0] + (head - k_heads) * p.qo_s[1] + t * p.qo_s[2];
    };

    if (stored)
        for (int e = threadIdx.x; e < Hkv * units; e += kThreads) {
            const int head = e / units, u = e % units;
            *reinterpret_cast<uint4 *>(p.c.v + row + head * p.c.s_head + u * 8) =
                *reinterpret_cast<const uint4 *>(p.v + b * p.v_s[0] + head * p.v_s[1] + t * p.v_s[2] + u * 8);
        }
    if constexpr (kMode == kHalves) {
        // a task is 8 pairs (two units), or one unit past the rotated part
        const int pairs = half / 8, tasks = pairs + (D - p.rot) / 8;
        for (int e = threadIdx.x; e < (k_heads + q_heads) * tasks; e += kThreads) {
            const int head = e / tasks, u = e % tasks;
            const uint16_t *src = source(head);
            uint16_t *dst = target(head);
            if (u < pairs) {
                const uint4 wx = *reinterpret_cast<const uint4 *>(src + u * 8);
                const uint4 wy = *reinterpret_cast<const uint4 *>(src + half + u * 8);
                float x[8], y[8], x2[8], y2[8];
                widen8<kF16>(wx, x);
                widen8<kF16>(wy, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 a = cs[u * 8 + j];
                    x2[j] = x[j] * a.x - y[j] * a.y;
                    y2[j] = y[j] * a.x + x[j] * a.y;
                }
                *reinterpret_cast<uint4 *>(dst + u * 8) = narrow8<kF16>(x2);
                *reinterpret_cast<uint4 *>(dst + half + u * 8) = narrow8<kF16>(y2);
            } else {
                const int d = p.rot + (u - pairs) * 8;
                *reinterpret_cast<uint4 *>(dst + d) = *reinterpret_cast<const uint4 *>(src + d);
            }
        }
    } else if constexpr (kMode == kNeighbours) {
        for (int e = threadIdx.x; e < (k_heads + q_heads) * units; e += kThreads) {
            const int head = e / units, u = e % units;
            const uint4 w = *reinterpret_cast<const uint4 *>(source(head) + u * 8);
            uint4 out = w;
            if (u * 8 < p.rot) {
                float x[8], r[8];
                widen8<kF16>(w, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = u * 8 + 2 * j < p.rot;
                    const float2 a = in ? cs[u * 4 + j] : make_float2(1.f, 0.f);
                    r[2 * j] = in ? x[2 * j] * a.x - x[2 * j + 1] * a.y : x[2 * j];
                    r[2 * j + 1] = in ? x[2 * j + 1] * a.x + x[2 * j] * a.y : x[2 * j + 1];
                }
                out = narrow8<kF16>(r);
            }
            *reinterpret_cast<uint4 *>(target(head) + u * 8) = out;
        }
    } else {
        // The halves of a pair are other threads' elements, which q_out = q
        // overwrites: whole heads at a time, all read before any is written.
        const int per = kThreads / units, mine = threadIdx.x / units, u = threadIdx.x % units;
        for (int first = 0; first < k_heads + q_heads; first += per) {
            const int head = first + mine;
            const bool on = mine < per && head < k_heads + q_heads;
            uint4 out = make_uint4(0u, 0u, 0u, 0u);
            if (on) {
                const uint16_t *src = source(head);
                out = *reinterpret_cast<const uint4 *>(src + u * 8);
                if (u * 8 < p.rot) {
                    float r[8];
                    widen8<kF16>(out, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int d = u * 8 + j;
                        if (d < half) {
                            const float y = widen1<kF16>(src[d + half]);
                            r[j] = r[j] * cs[d].x - y * cs[d].y;
                        } else if (d < p.rot) {
                            const float y = widen1<kF16>(src[d - half]);
                            r[j] = r[j] * cs[d - half].x + y * cs[d - half].y;
                        }
                    }
                    out = narrow8<kF16>(r);
                }
            }
            __syncthreads();
            if (on) *reinterpret_cast<uint4 *>(target(head) + u * 8) = out;
        }
    }
}

template <bool kF16>
cudaError_t launch(const AppendParams &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.B * p.T));
    const size_t smem = (size_t)(p.rot / 2) * sizeof(float2);
    if (p.interleaved || p.rot == 0)
        return launch_behind(append_kernel<kF16, kNeighbours>, grid, kThreads, smem, stream, p);
    if (p.rot % 16 == 0) return launch_behind(append_kernel<kF16, kHalves>, grid, kThreads, smem, stream, p);
    return launch_behind(append_kernel<kF16, kHalvesOdd>, grid, kThreads, smem, stream, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream)
{
    return p.f16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace fa
