// fa_paged_team.cuh -- a team (a cluster of CTAs) joins the states that its warps have
// of one tile, for the row kernels.
#pragma once

#include "fa_paged.h"
#include "sm103_ptx.cuh"

#include <cmath>

namespace fa {

constexpr float kLn2 = 0.69314718055994530942f;

// A state of a row and four of its columns: m, l and O, not yet divided by l.
struct Four {
    float top, sum;
    float4 acc;
};

// The join of `kMany` of them.
template <int kMany>
__device__ __forceinline__ Four join(const float2 (&stat)[kMany], const float4 (&o)[kMany])
{
    Four x{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < kMany; ++i) x.top = fmaxf(x.top, stat[i].x);
    const float ref = x.top == -INFINITY ? 0.f : x.top;
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        const float f = ptx::ex2_approx(stat[i].x - ref);
        x.sum = fmaf(f, stat[i].y, x.sum);
        x.acc.x = fmaf(f, o[i].x, x.acc.x);
        x.acc.y = fmaf(f, o[i].y, x.acc.y);
        x.acc.z = fmaf(f, o[i].z, x.acc.z);
        x.acc.w = fmaf(f, o[i].w, x.acc.w);
    }
    return x;
}

// The join of a team's tile, after the warps have left their states: O `pitch`
// bytes apart from `ring` on, (m, l) from `stat` on.  A thread joins the CTA's
// states of a row and four columns and sends the result to the CTA that finishes
// them, every p.team-th four columns; `mail` has a place for each of the team.
// (Reading all warps' states across the cluster instead: 2.5 us more.)
template <int DP, bool kF16>
__device__ __forceinline__ void join_team(const PagedParams &p, const uint8_t *ring, int pitch, const float2 *stat,
                                          float4 *mail, int b, int h, int len)
{
    constexpr int RM = 8, kUnits = RM * DP / 4;
    static_assert(kUnits <= 32 * kTeamWarps, "a thread per row and four columns");
    float2 *mail_stat = reinterpret_cast<float2 *>(mail + kUnits);
    const int rank = (int)blockIdx.x % p.team, unit = threadIdx.x, units = RM * p.c.D / 4;
    __syncthreads();
    Four x{};
    if (unit < units) {
        float2 st[kTeamWarps];
        float4 o[kTeamWarps];
#pragma unroll
        for (int w = 0; w < kTeamWarps; ++w) {
            st[w] = stat[w * RM + unit % RM];
            o[w] = *reinterpret_cast<const float4 *>(ring + w * pitch + unit * 16);
        }
        x = join<kTeamWarps>(st, o);
    }
    __syncwarp();
    ptx::cluster_wait();                            // the team's CTAs have all started
    if (unit < units) {
        const int c4 = unit / RM, to = c4 % p.team;
        const int place = (c4 / p.team * p.team + rank) * RM + unit % RM;
        ptx::st_cluster4(ptx::cluster_address(ptx::smem_u32(mail + place), to), x.acc);
        ptx::st_cluster2(ptx::cluster_address(ptx::smem_u32(mail_stat + place), to), make_float2(x.top, x.sum));
    }
    __syncwarp();
    ptx::cluster_arrive();
    ptx::cluster_wait();
    const int row = unit % RM, mine = unit / RM, c4 = mine * p.team + rank;
    if (c4 >= p.c.D / 4 || row >= p.G * p.T) return;
    float2 st[kMostTeam];
    float4 o[kMostTeam];
#pragma unroll
    for (int i = 0; i < kMostTeam; ++i) {
        st[i] = make_float2(-INFINITY, 0.f);
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < p.team) {
            const int place = (mine * p.team + i) * RM + row;
            st[i] = mail_stat[place];
            o[i] = mail[place];
        }
    }
    x = join<kMostTeam>(st, o);
    const int t = p.by_g.quotient(row), hq = h * p.G + row - t * p.G;
    // (a row without a token sees nothing, not even a prefix)
    const bool empty = x.sum == 0.f || (p.causal && len - p.T + t < 0);
    const float inv = empty ? 0.f : 1.f / x.sum;
    *reinterpret_cast<uint2 *>(p.o + b * p.o_s[0] + hq * p.o_s[1] + t * p.o_s[2] + 4 * c4) =
        empty ? make_uint2(0u, 0u)
              : make_uint2(ptx::pack16x2<kF16>(x.acc.x * inv, x.acc.y * inv),
                           ptx::pack16x2<kF16>(x.acc.z * inv, x.acc.w * inv));
    if (p.lse && c4 == 0) p.lse[((int64_t)b * p.Hq + hq) * p.T + t] = empty ? -INFINITY : (x.top + log2f(x.sum)) * kLn2;
}

}  // namespace fa
