// fa_read.cu -- the last tokens of a cache read back as 16-bit rows, decoded where it
// has 4 bits (fa_four.cuh).  Bound by memory: every value is read once and written
// once.
#include "fa_four.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;

// A CTA per token; a thread takes 16 elements of a key or value.
template <bool kFour, bool kF16>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p)
{
    ptx::wait_for_primary();
    const int64_t b = blockIdx.x / (unsigned)p.T;
    const int t = (int)(blockIdx.x - b * p.T);
    const int32_t *seq_len = kFour ? p.c4.seq_len : p.c.seq_len, *table = kFour ? p.c4.table : p.c.table;
    const int i = max(seq_len[b], -1) - p.T + t;
    const uint32_t at = (uint32_t)max(i, 0), size = (uint32_t)(kFour ? p.c4.page_size : p.c.page_size);
    int page = -1;
    if (i >= 0 && at / size < (uint32_t)(kFour ? p.c4.table_width : p.c.table_width))
        page = table[b * (kFour ? p.c4.table_stride : p.c.table_stride) + at / size];
    const bool there = page >= 0 && page < (kFour ? p.c4.num_pages : p.c.num_pages);
    const int64_t slot = there ? at % size : 0;
    if (!there) page = 0;
    const int D = kFour ? p.c4.D : p.c.D, Hkv = kFour ? p.c4.Hkv : p.c.Hkv;
    for (int e = threadIdx.x; e < 2 * Hkv * (int)p.by_groups.by; e += kThreads) {
        const int which = p.by_groups.quotient(e), g = e - which * (int)p.by_groups.by, head = which < Hkv ? which : which - Hkv;
        const bool both = 16 * g + 8 < D;           // (a last group may have 8)
        uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (there) {
            if constexpr (kFour) {
                const PagedCache4 &c = p.c4;
                const uint8_t *row = (which < Hkv ? c.k : c.v) + page * c.s_page + slot * c.s_slot + head * c.s_head;
                const uint8_t *scales = (which < Hkv ? c.ks : c.vs) + page * c.t_page + slot * c.t_slot + head * c.t_head;
                const uint2 x = *reinterpret_cast<const uint2 *>(row + 8 * g);
                const uint32_t scale = scales[g];
                w[0] = rows_from_four<kF16>(x.x, scale);
                w[1] = rows_from_four<kF16>(x.y, scale);
            } else {
                const PagedCache &c = p.c;
                const uint4 *row = reinterpret_cast<const uint4 *>((which < Hkv ? c.k : c.v) + page * c.s_page + slot * c.s_slot +
                                                                   head * c.s_head + 16 * g);
                w[0] = row[0];
                if (both) w[1] = row[1];
            }
        }
        uint4 *dst = reinterpret_cast<uint4 *>((which < Hkv ? p.k + b * p.k_s[0] + head * p.k_s[1] + t * p.k_s[2]
                                                            : p.v + b * p.v_s[0] + head * p.v_s[1] + t * p.v_s[2]) + 16 * g);
        dst[0] = w[0];
        if (both) dst[1] = w[1];
    }
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, bool four, cudaStream_t stream)
{
    const dim3 grid((unsigned)((int64_t)p.B * p.T));
    if (!four) return launch_behind(read_kernel<false, false>, grid, kThreads, 0, stream, p);
    return p.f16 ? launch_behind(read_kernel<true, true>, grid, kThreads, 0, stream, p)
                 : launch_behind(read_kernel<true, false>, grid, kThreads, 0, stream, p);
}

}  // namespace fa
