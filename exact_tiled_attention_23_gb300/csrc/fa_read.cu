// fa_read.cu -- the last tokens of a cache read back as 16-bit rows, decoded where it
// has 4 bits (fa_four.cuh).  Bound by memory: every value is read once and written
// once.
#include "fa_four.cuh"

namespace fa {

namespace {

constexpr int kThreads = 128;

// A CTA per token; a thread takes 8 elements of a key or value.
template <bool kFour, bool kF16>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p)
{
    ptx::wait_for_primary();
    const int64_t b = blockIdx.x / p.T;
    const int t = (int)(blockIdx.x % p.T);
    const int32_t *seq_len = kFour ? p.c4.seq_len : p.c.seq_len, *table = kFour ? p.c4.table : p.c.table;
    const int i = max(seq_len[b], -1) - p.T + t;
    const uint32_t at = (uint32_t)max(i, 0), size = (uint32_t)(kFour ? p.c4.page_size : p.c.page_size);
    int page = -1;
    if (i >= 0 && at / size < (uint32_t)(kFour ? p.c4.table_width : p.c.table_width))
        page = table[b * (kFour ? p.c4.table_stride : p.c.table_stride) + at / size];
    const bool there = page >= 0 && page < (kFour ? p.c4.num_pages : p.c.num_pages);
    const int64_t slot = there ? at % size : 0;
    if (!there) page = 0;
    const int D = kFour ? p.c4.D : p.c.D, Hkv = kFour ? p.c4.Hkv : p.c.Hkv, units = D / 8;
    for (int e = threadIdx.x; e < 2 * Hkv * units; e += kThreads) {
        const int which = e / units, u = e % units, head = which < Hkv ? which : which - Hkv;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (there) {
            if constexpr (kFour) {
                const PagedCache4 &c = p.c4;
                const uint8_t *row = (which < Hkv ? c.k : c.v) + page * c.s_page + slot * c.s_slot + head * c.s_head;
                const uint8_t *scales = (which < Hkv ? c.ks : c.vs) + page * c.t_page + slot * c.t_slot + head * c.t_head;
                w = rows_from_four<kF16>(*reinterpret_cast<const uint32_t *>(row + 4 * u), scales[u / 2]);
            } else {
                const PagedCache &c = p.c;
                w = *reinterpret_cast<const uint4 *>((which < Hkv ? c.k : c.v) + page * c.s_page + slot * c.s_slot +
                                                     head * c.s_head + u * 8);
            }
        }
        uint16_t *dst = which < Hkv ? p.k + b * p.k_s[0] + head * p.k_s[1] + t * p.k_s[2]
                                    : p.v + b * p.v_s[0] + head * p.v_s[1] + t * p.v_s[2];
        *reinterpret_cast<uint4 *>(dst + u * 8) = w;
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
