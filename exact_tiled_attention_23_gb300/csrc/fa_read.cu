// fa_read.cu -- the last tokens of a cache read back as 16-bit rows, decoded where it
// has 4 bits (fa_four.cuh).  Bound by memory: every value is read once and written
// once (two prompts of 8192 tokens, 8 key heads, D = 128, from 4 bits: 86 MB in 17 us,
// 5.1 TB/s).
#include "fa_four.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;

// A CTA has kTokens tokens; a thread takes 16 elements of a key or value of each, all
// read before any is written.
template <bool kFour, bool kF16, int kTokens>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p)
{
    ptx::wait_for_primary();
    const int parts = (p.T + kTokens - 1) / kTokens;
    const int64_t b = blockIdx.x / (unsigned)parts;
    const int t0 = (int)(blockIdx.x - b * parts) * kTokens;
    const int32_t *seq_len = kFour ? p.c4.seq_len : p.c.seq_len, *table = kFour ? p.c4.table : p.c.table;
    const uint32_t size = (uint32_t)(kFour ? p.c4.page_size : p.c.page_size);
    const int n = max(seq_len[b], -1) - p.T;
    int page[kTokens], slot[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int i = n + t0 + k;
        const uint32_t at = (uint32_t)max(i, 0);
        page[k] = -1;
        slot[k] = (int)(at % size);
        if (t0 + k < p.T && i >= 0 && at / size < (uint32_t)(kFour ? p.c4.table_width : p.c.table_width))
            page[k] = table[b * (kFour ? p.c4.table_stride : p.c.table_stride) + at / size];
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k)
        if (page[k] >= (kFour ? p.c4.num_pages : p.c.num_pages)) page[k] = -1;
    const int D = kFour ? p.c4.D : p.c.D, Hkv = kFour ? p.c4.Hkv : p.c.Hkv;
    for (int e = threadIdx.x; e < 2 * Hkv * (int)p.by_groups.by; e += kThreads) {
        const int which = p.by_groups.quotient(e), g = e - which * (int)p.by_groups.by, head = which < Hkv ? which : which - Hkv;
        const bool both = 16 * g + 8 < D;           // (a last group may have 8)
        uint4 w[kTokens][2];
        uint2 four[kTokens];
        uint32_t scale[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            w[k][0] = w[k][1] = make_uint4(0u, 0u, 0u, 0u);
            four[k] = make_uint2(0u, 0u);
            scale[k] = 0;
            if (page[k] < 0) continue;
            if constexpr (kFour) {
                const PagedCache4 &c = p.c4;
                four[k] = *reinterpret_cast<const uint2 *>((which < Hkv ? c.k : c.v) + page[k] * c.s_page + slot[k] * c.s_slot +
                                                           head * c.s_head + 8 * g);
                scale[k] = ((which < Hkv ? c.ks : c.vs) + page[k] * c.t_page + slot[k] * c.t_slot + head * c.t_head)[g];
            } else {
                const PagedCache &c = p.c;
                const uint4 *row = reinterpret_cast<const uint4 *>((which < Hkv ? c.k : c.v) + page[k] * c.s_page +
                                                                   slot[k] * c.s_slot + head * c.s_head + 16 * g);
                w[k][0] = row[0];
                if (both) w[k][1] = row[1];
            }
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int t = t0 + k;
            if (t >= p.T) continue;
            if constexpr (kFour) {
                w[k][0] = rows_from_four<kF16>(four[k].x, scale[k]);
                w[k][1] = rows_from_four<kF16>(four[k].y, scale[k]);
            }
            uint4 *dst = reinterpret_cast<uint4 *>((which < Hkv ? p.k + b * p.k_s[0] + head * p.k_s[1] + t * p.k_s[2]
                                                                : p.v + b * p.v_s[0] + head * p.v_s[1] + t * p.v_s[2]) + 16 * g);
            dst[0] = w[k][0];
            if (both) dst[1] = w[k][1];
        }
    }
}

template <int kTokens>
cudaError_t launch(const ReadParams &p, bool four, cudaStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.B * ((p.T + kTokens - 1) / kTokens)));
    if (!four) return launch_behind(read_kernel<false, false, kTokens>, grid, kThreads, 0, stream, p);
    return p.f16 ? launch_behind(read_kernel<true, true, kTokens>, grid, kThreads, 0, stream, p)
                 : launch_behind(read_kernel<true, false, kTokens>, grid, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, bool four, cudaStream_t stream)
{
    // Few tokens: a CTA each, the shortest way (64 tokens of 8 heads 1.9 us, four to a
    // CTA 3.1; 8192 9.8 and 10.5); many: four, whose reads wait together (16384: 18.7
    // and 15.9).
    const bool many = p.T >= 4 && (int64_t)p.B * p.T > 4 * 16 * (int64_t)sm_count_of(current_device());
    return many ? launch<4>(p, four, stream) : launch<1>(p, four, stream);
}

}  // namespace fa
