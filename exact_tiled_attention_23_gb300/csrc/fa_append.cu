// fa_append.cu -- keys and values of new tokens into a paged cache, of 16 or of 4 bits
// (fa_four.cuh), with the position rotation of keys and queries applied on the way;
// and the rotation alone.
//
// Token t of sequence b has the index i = seq_len[b] - T + t; it turns by the position
// n = offset + i, or by positions that the caller gives, and its key and value go to
// slot i % page_size of page table[b][i / page_size].
//
// Pair p of a head, (x, y), turns by the angle a = n * inv_freq[p], n the token's
// position (on the pair's axis, where there are several):
//     x' = x cos a - y sin a,    y' = y cos a + x sin a.
// A far position times a frequency loses its angle in fp32 (a product of 10^5
// is good to 2^-7 radians), so the angle is kept as a fraction of a turn in 64
// bits: inv_freq[p] / 2pi as a fixed-point number F of 2^-64 turns, and n * F
// modulo 2^64 drops whole turns exactly.  F comes from 128 bits of 1 / 2pi, so it
// is off by less than its last bit for every frequency up to 2^16, and the angle
// by n 2^-64 turns: 2^-33 at n = 2^31, where the fp32 form's 2^-26 decides, and
// 2^-24 at the farthest position, 2^40 + 2^31.
//
// Bound by memory: every value is read once and written once, whole 16-byte units
// at a time.  One CTA per token (where tokens have little, a warp), so that a token's
// angles are computed once for all heads.  Two prompts of 8192 tokens, 32 query and 8
// key heads, D = 128: 403 MB in 62 us, 6.5 TB/s (a copy: 6.8).  One token: 3 us, a
// launch and four waits in turn (length, page, values, stores).
#include "fa_four.cuh"

#include <type_traits>

namespace fa {

namespace {

// Threads of a CTA, and of those the ones that have a token: all, or where tokens are
// many and have little, a warp each (kGroup below).
constexpr int kThreads = 128;

template <int kGroup>
__device__ __forceinline__ int group_thread()
{
    return kGroup == kThreads ? (int)threadIdx.x : (int)threadIdx.x % kGroup;
}

template <int kGroup>
__device__ __forceinline__ void group_sync()
{
    if constexpr (kGroup == 32)
        __syncwarp();
    else
        __syncthreads();
}

// The token of a thread's group; false past the last.  (kFast: where the CTA's sequence
// is on the way to its first read.  Without, a division of the grid's index, which every
// thread has in the same register, leaves more to the rest: 32 registers, not 36, in the
// kernel without a cache, 84.5 and not 91.4 us in the case below.)
template <int kGroup, bool kFast = false>
__device__ __forceinline__ bool group_token(int64_t tokens, FastDiv by_t, int64_t &b, int &t)
{
    const int token = kGroup == kThreads ? (int)blockIdx.x : (int)blockIdx.x * (kThreads / kGroup) + (int)threadIdx.x / kGroup;
    if constexpr (kGroup == kThreads && !kFast) {
        b = blockIdx.x / (int)by_t.by;
        t = (int)(blockIdx.x % (int)by_t.by);
    } else {
        const int at = by_t.quotient(token);
        b = at;
        t = token - at * (int)by_t.by;
    }
    return kGroup == kThreads || token < tokens;
}

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

// The cosines and sines of token t of sequence b, `at` its place in the sequence,
// into cs[rot / 2].
template <int kGroup>
__device__ __forceinline__ void turns_of(const TurnParams &p, int64_t b, int t, int64_t at, float2 *cs)
{
    for (int j = group_thread<kGroup>(); j < p.rot / 2; j += kGroup) {
        int64_t n = at;
        float f = p.inv_freq[j];
        if (p.pos) {
            const int axis = p.pair_axis ? p.pair_axis[j] : 0;
            const bool on = axis >= 0 && axis < p.axes;    // a pair of no axis does not turn
            n = on ? p.pos[axis * p.pos_s[0] + b * p.pos_s[1] + t * p.pos_s[2]] : 0;
            if (!on) f = 0.f;
        }
        float2 x = turn(p.offset + n, f);
        if (p.inverse) x.y = -x.y;
        cs[j] = x;
    }
}

// Turns `heads` heads of D elements by cs, from source(head) to target(head), which
// may be one place; all threads of the group call it.
template <bool kF16, int kMode, int kGroup, typename Source, typename Target>
__device__ __forceinline__ void turn_heads(int heads, int D, int rot, const float2 *cs, const Source &source,
                                           const Target &target)
{
    const int half = rot / 2, units = D / 8;
    if constexpr (kMode == kHalves) {
        // a task is 8 pairs (two units), or one unit past the rotated part
        const int pairs = half / 8, tasks = pairs + (D - rot) / 8;
        for (int e = group_thread<kGroup>(); e < heads * tasks; e += kGroup) {
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
                const int d = rot + (u - pairs) * 8;
                *reinterpret_cast<uint4 *>(dst + d) = *reinterpret_cast<const uint4 *>(src + d);
            }
        }
    } else if constexpr (kMode == kNeighbours) {
        for (int e = group_thread<kGroup>(); e < heads * units; e += kGroup) {
            const int head = e / units, u = e % units;
            const uint4 w = *reinterpret_cast<const uint4 *>(source(head) + u * 8);
            uint4 out = w;
            if (u * 8 < rot) {
                float x[8], r[8];
                widen8<kF16>(w, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = u * 8 + 2 * j < rot;
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
        const int per = kGroup / units, mine = group_thread<kGroup>() / units, u = group_thread<kGroup>() % units;
        for (int first = 0; first < heads; first += per) {
            const int head = first + mine;
            const bool on = mine < per && head < heads;
            uint4 out = make_uint4(0u, 0u, 0u, 0u);
            if (on) {
                const uint16_t *src = source(head);
                out = *reinterpret_cast<const uint4 *>(src + u * 8);
                if (u * 8 < rot) {
                    float r[8];
                    widen8<kF16>(out, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int d = u * 8 + j;
                        if (d < half) {
                            const float y = widen1<kF16>(src[d + half]);
                            r[j] = r[j] * cs[d].x - y * cs[d].y;
                        } else if (d < rot) {
                            const float y = widen1<kF16>(src[d - half]);
                            r[j] = r[j] * cs[d - half].x + y * cs[d - half].y;
                        }
                    }
                    out = narrow8<kF16>(r);
                }
            }
            group_sync<kGroup>();
            if (on) *reinterpret_cast<uint4 *>(target(head) + u * 8) = out;
        }
    }
}

// A token's cosines and sines are computed once for all heads, then each thread of
// its group moves 16-byte units of q, k and v.
template <bool kF16, int kMode, int kGroup>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    extern __shared__ float2 all_cs[];                      // [groups][rot / 2]
    float2 *const cs = kGroup == kThreads ? all_cs : all_cs + (int)threadIdx.x / kGroup * (p.turn.rot / 2);
    ptx::wait_for_primary();
    int64_t b;
    int t;
    if (!group_token<kGroup>((int64_t)p.B * p.T, p.by_t, b, t)) return;
    const int i = max(p.c.seq_len[b], -1) - p.T + t;        // (-1 - T at least: no overflow)
    const int D = p.c.D, Hkv = p.c.Hkv;
    const int units = D / 8;

    if (i < 0) {                                            // no token here: its query is zero
        if (p.q)
            for (int e = group_thread<kGroup>(); e < p.Hq * units; e += kGroup)
                *reinterpret_cast<uint4 *>(p.q_out + b * p.qo_s[0] + (e / units) * p.qo_s[1] + t * p.qo_s[2] +
                                           (e % units) * 8) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const uint32_t at = (uint32_t)i, size = (uint32_t)p.c.page_size;
    int page = -1;
    if (at / size < (uint32_t)p.c.table_width) page = p.c.table[b * p.c.table_stride + at / size];
    const bool stored = page >= 0 && page < p.c.num_pages;   // otherwise the key and value are dropped
    const int64_t row = stored ? page * p.c.s_page + (int64_t)(at % size) * p.c.s_slot : 0;
    turns_of<kGroup>(p.turn, b, t, i, cs);
    group_sync<kGroup>();

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
        for (int e = group_thread<kGroup>(); e < Hkv * units; e += kGroup) {
            const int head = e / units, u = e % units;
            *reinterpret_cast<uint4 *>(p.c.v + row + head * p.c.s_head + u * 8) =
                *reinterpret_cast<const uint4 *>(p.v + b * p.v_s[0] + head * p.v_s[1] + t * p.v_s[2] + u * 8);
        }
    turn_heads<kF16, kMode, kGroup>(k_heads + q_heads, D, p.turn.rot, cs, source, target);
}

// Whether a warp per token serves: where tokens have little and are many, the more the
// more they have.  A CTA and a warp per token, us, into 16 bits, into 4, and without a
// cache (`units`: 16-byte units of a token, of q, k and v in the first two, of q and k
// in the third):
//   tokens   units         into 16        into 4         without
//   500      64, 64, 48    3.3 and 3.3    3.3 and 3.3    2.5 and 2.5
//   2000     15, 15, 10    4.1 and 3.3    5.8 and 4.2    3.3 and 2.9
//   2000     64, 64, 48    4.1 and 3.7    5.8 and 4.2    3.3 and 2.9
//   2000     192, 192, 160 5.0 and 5.4    6.3 and 5.4    3.8 and 4.6
//   5000     192, 192, 160 8.7 and 7.8    11.1 and 8.3   6.6 and 7.0
//   50000    64, 64, 48    48 and 31      62 and 41      28 and 20
//   50000    192, 192, 160 69 and 60      78 and 56      48 and 47
//   16384    768, 768, -   62 and 68      65 and 69
//   32760    -, -, 512                                   84.5 and 87.5
bool warp_per_token(int64_t tokens, int64_t units)
{
    return units <= 192 && tokens > (units <= 64 ? 8 : 64) * (int64_t)sm_count_of(current_device()) &&
           tokens < (int64_t)1 << 30;
}

// kernel(mode, group) with a token per CTA, or per warp.
template <typename P, typename Launch>
cudaError_t launch_tokens(const P &p, int64_t units, const Launch &launch)
{
    const int64_t tokens = (int64_t)p.B * p.T;
    const bool warps = warp_per_token(tokens, units);
    const int per = warps ? kThreads / 32 : 1;
    const dim3 grid((unsigned)((tokens + per - 1) / per));
    const size_t smem = (size_t)per * (p.turn.rot / 2) * sizeof(float2);
    const int mode = p.turn.interleaved || p.turn.rot == 0 ? kNeighbours : p.turn.rot % 16 == 0 ? kHalves : kHalvesOdd;
    using std::integral_constant;
    const auto with_group = [&](auto m) {
        return warps ? launch(m, integral_constant<int, 32>{}, grid, smem)
                     : launch(m, integral_constant<int, kThreads>{}, grid, smem);
    };
    switch (mode) {
    case kNeighbours: return with_group(integral_constant<int, kNeighbours>{});
    case kHalves: return with_group(integral_constant<int, kHalves>{});
    default: return with_group(integral_constant<int, kHalvesOdd>{});
    }
}

template <bool kF16>
cudaError_t launch(const AppendParams &p, cudaStream_t stream)
{
    return launch_tokens(p, (p.Hq + (int64_t)2 * p.c.Hkv) * (p.c.D / 8), [&](auto mode, auto group, dim3 grid, size_t smem) {
        return launch_behind(append_kernel<kF16, decltype(mode)::value, decltype(group)::value>, grid, kThreads, smem, stream, p);
    });
}

// ---------------------------------------------------------------- 4 bits
// A key's pairs turn in fp32 and the result is rounded once, to 4 bits.  A thread
// takes a group of 16 elements of a key or value, so that no thread needs another's
// largest value (a key's partner elements are read a second time, from the L1).  Two
// prompts of 8192 tokens as above: 354 MB in 65 us, 5.4 TB/s (8 instead of 10 CTAs an
// SM 67; with a division per element 74).  One token of 256 sequences: 3.5 us.

// Elements 8 u .. 8 u + 7 of a turned head, which are `w` before.
template <bool kF16, int kMode>
__device__ __forceinline__ void turned8(const uint16_t *src, int u, uint4 w, int rot, const float2 *cs, float (&x)[8])
{
    widen8<kF16>(w, x);
    if (u * 8 >= rot) return;
    const int half = rot / 2;
    if constexpr (kMode == kHalves) {
        const bool first = u * 8 < half;
        const int from = first ? u * 8 : u * 8 - half;
        float y[8];
        widen8<kF16>(*reinterpret_cast<const uint4 *>(src + (first ? from + half : from)), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 a = cs[from + j];
            x[j] = first ? x[j] * a.x - y[j] * a.y : x[j] * a.x + y[j] * a.y;
        }
    } else if constexpr (kMode == kNeighbours) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (u * 8 + 2 * j >= rot) continue;
            const float2 a = cs[u * 4 + j];
            const float r = x[2 * j] * a.x - x[2 * j + 1] * a.y;
            x[2 * j + 1] = x[2 * j + 1] * a.x + x[2 * j] * a.y;
            x[2 * j] = r;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = u * 8 + j;
            if (d < half)
                x[j] = x[j] * cs[d].x - widen1<kF16>(src[d + half]) * cs[d].y;
            else if (d < rot)
                x[j] = x[j] * cs[d - half].x + widen1<kF16>(src[d - half]) * cs[d - half].y;
        }
    }
}

// (A thread's first group is read before it is known where it goes: two waits less.)
template <bool kF16, int kMode, int kGroup>
__global__ void __launch_bounds__(kThreads, 10) append4_kernel(const Append4Params p)
{
    extern __shared__ float2 all_cs[];                      // [groups][rot / 2]
    float2 *const cs = kGroup == kThreads ? all_cs : all_cs + (int)threadIdx.x / kGroup * (p.turn.rot / 2);
    const int thread = group_thread<kGroup>();
    ptx::wait_for_primary();
    int64_t b;
    int t;
    if (!group_token<kGroup, true>((int64_t)p.B * p.T, p.by_t, b, t)) return;
    const int D = p.c.D, Hkv = p.c.Hkv, units = D / 8;
    // keys, then values; groups of a head
    const int groups = D <= 64 ? 2 : D <= 128 ? 3 : 4;      // (the logarithm of how many a row has)
    const auto source = [&](int which) {
        return which < Hkv ? p.k + b * p.k_s[0] + which * p.k_s[1] + t * p.k_s[2]
                           : p.v + b * p.v_s[0] + (which - Hkv) * p.v_s[1] + t * p.v_s[2];
    };
    uint4 w[2];
    const auto fetch = [&](int e) {
        const uint16_t *src = source(e >> groups);
        const int u = 2 * (e & ((1 << groups) - 1));
#pragma unroll
        for (int h = 0; h < 2; ++h)                          // past the head: padding
            w[h] = u + h < units ? *reinterpret_cast<const uint4 *>(src + (u + h) * 8) : make_uint4(0u, 0u, 0u, 0u);
    };
    if (thread < (2 * Hkv) << groups) fetch(thread);
    const int i = max(p.c.seq_len[b], -1) - p.T + t;        // (-1 - T at least: no overflow)

    if (i < 0) {                                            // no token here: its query is zero
        if (p.q)
            for (int e = thread; e < p.Hq * units; e += kGroup)
                *reinterpret_cast<uint4 *>(p.q_out + b * p.qo_s[0] + (e / units) * p.qo_s[1] + t * p.qo_s[2] +
                                           (e % units) * 8) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int entry = p.c.by_page.quotient(i);
    int page = -1;
    if (entry < p.c.table_width) page = p.c.table[b * p.c.table_stride + entry];
    turns_of<kGroup>(p.turn, b, t, i, cs);
    group_sync<kGroup>();

    if (page >= 0 && page < p.c.num_pages) {                // otherwise the key and value are dropped
        const int64_t slot = i - entry * p.c.page_size;
        const int64_t row = page * p.c.s_page + slot * p.c.s_slot, scales = page * p.c.t_page + slot * p.c.t_slot;
        for (int e = thread; e < (2 * Hkv) << groups; e += kGroup) {
            if (e != thread) fetch(e);
            const int which = e >> groups, g = e & ((1 << groups) - 1), head = which < Hkv ? which : which - Hkv;
            float x[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float y[8];
                if (which < Hkv && 2 * g + h < units)
                    turned8<kF16, kMode>(source(which), 2 * g + h, w[h], p.turn.rot, cs, y);
                else
                    widen8<kF16>(w[h], y);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[8 * h + j] = y[j];
            }
            uint32_t code;
            const uint2 four = to_four(x, code);
            *reinterpret_cast<uint2 *>((which < Hkv ? p.c.k : p.c.v) + row + head * p.c.s_head + g * 8) = four;
            ((which < Hkv ? p.c.ks : p.c.vs) + scales + head * p.c.t_head)[g] = (uint8_t)code;
        }
    }
    const auto from = [&](int head) -> const uint16_t * { return p.q + b * p.q_s[0] + head * p.q_s[1] + t * p.q_s[2]; };
    const auto target = [&](int head) -> uint16_t * { return p.q_out + b * p.qo_s[0] + head * p.qo_s[1] + t * p.qo_s[2]; };
    turn_heads<kF16, kMode, kGroup>(p.q ? p.Hq : 0, D, p.turn.rot, cs, from, target);
}

template <bool kF16>
cudaError_t launch4(const Append4Params &p, cudaStream_t stream)
{
    return launch_tokens(p, (p.Hq + (int64_t)2 * p.c.Hkv) * (p.c.D / 8), [&](auto mode, auto group, dim3 grid, size_t smem) {
        return launch_behind(append4_kernel<kF16, decltype(mode)::value, decltype(group)::value>, grid, kThreads, smem, stream, p);
    });
}

// ---------------------------------------------------------------- no cache
// 32760 tokens, 16 query and 16 key heads, D = 128, three axes: 537 MB in 84 us, 6.4
// TB/s; turned back the same.
template <bool kF16, int kMode, int kGroup>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p)
{
    extern __shared__ float2 all_cs[];                      // [groups][rot / 2]
    float2 *const cs = kGroup == kThreads ? all_cs : all_cs + (int)threadIdx.x / kGroup * (p.turn.rot / 2);
    ptx::wait_for_primary();
    int64_t b;
    int t;
    if (!group_token<kGroup>((int64_t)p.B * p.T, p.by_t, b, t)) return;
    turns_of<kGroup>(p.turn, b, t, t, cs);
    group_sync<kGroup>();
    const auto source = [&](int head) -> const uint16_t * {
        const int i = head < p.H[0] ? 0 : 1;
        return p.x[i] + b * p.x_s[i][0] + (head - i * p.H[0]) * p.x_s[i][1] + t * p.x_s[i][2];
    };
    const auto target = [&](int head) -> uint16_t * {
        const int i = head < p.H[0] ? 0 : 1;
        return p.y[i] + b * p.y_s[i][0] + (head - i * p.H[0]) * p.y_s[i][1] + t * p.y_s[i][2];
    };
    turn_heads<kF16, kMode, kGroup>(p.H[0] + p.H[1], p.D, p.turn.rot, cs, source, target);
}

template <bool kF16>
cudaError_t launch_turn(const RotaryParams &p, cudaStream_t stream)
{
    return launch_tokens(p, (int64_t)(p.H[0] + p.H[1]) * (p.D / 8), [&](auto mode, auto group, dim3 grid, size_t smem) {
        return launch_behind(rotary_kernel<kF16, decltype(mode)::value, decltype(group)::value>, grid, kThreads, smem, stream, p);
    });
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream)
{
    return p.f16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

cudaError_t launch_append4(const Append4Params &p, cudaStream_t stream)
{
    return p.f16 ? launch4<true>(p, stream) : launch4<false>(p, stream);
}

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream)
{
    return p.f16 ? launch_turn<true>(p, stream) : launch_turn<false>(p, stream);
}

}  // namespace fa
