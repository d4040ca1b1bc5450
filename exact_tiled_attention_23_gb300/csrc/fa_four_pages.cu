// fa_four_pages.cu -- the pages of a 4-bit cache as pages of halves in a workspace, for
// calls whose many row tiles would each decode them again (fa_paged_tc.cu).
//
// Bound by memory: 144 bytes read and 512 written per key and head at D = 128 (a
// sequence of 16384 keys, 8 heads: 86 MB, 23 us with cold caches; with one group of a
// thread in flight instead of four, and a CTA for all heads of a page, 45).
#include "fa_four.cuh"
#include "fa_four_rows.h"

namespace fa {

namespace {

constexpr int kWideThreads = 256;
constexpr int kWideTasks = 1024;       // groups of 16 elements of a CTA at least, where a page has them

// Pages of the sequences of a call as 16-bit pages of their own, page j of sequence
// b as page b * width + j, and the tables and lengths that go with them.  A CTA per
// page and p.heads of its heads; a thread takes groups of 16 elements, four at a time.
template <bool kF16>
__global__ void __launch_bounds__(kWideThreads) widen_pages_kernel(const WidenParams p)
{
    ptx::wait_for_primary();
    const PagedCache4 &c = p.c;
    const int at = blockIdx.x / (unsigned)p.parts, head0 = (blockIdx.x - at * p.parts) * p.heads;
    const int b = at / c.table_width, j = at - b * c.table_width;
    const int64_t cap = (int64_t)c.table_width * c.page_size;
    const int n = c.seq_len[b] < 0 ? 0 : (int)min((int64_t)c.seq_len[b], cap);
    const int slots = min(c.page_size, n - j * c.page_size);
    if (head0 == 0 && threadIdx.x == 0 && j == 0) p.seq_len[b] = n;
    if (slots <= 0) return;                                 // (its entry is not read)
    const int page = c.table[b * c.table_stride + j];
    const bool there = page >= 0 && page < c.num_pages;
    if (head0 == 0 && threadIdx.x == 0) p.table[at] = there ? at : -1;
    if (!there) return;
    const int groups = (int)p.by_groups.by, tasks = 2 * min(p.heads, c.Hkv - head0) * slots * groups;
    const int64_t to = (int64_t)at * c.Hkv * c.page_size * c.D;
    constexpr int kMany = 4;
    for (int first = threadIdx.x; first < tasks; first += kWideThreads * kMany) {
        uint2 w[kMany];
        uint32_t scale[kMany];
        uint16_t *dst[kMany];
        bool both[kMany];
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            const int e = first + i * kWideThreads;
            dst[i] = nullptr;
            if (e >= tasks) continue;
            // keys and values of a head after another's, rows of it, groups of a row
            const int row = p.by_groups.quotient(e), g = e - row * groups, which = row / slots, slot = row - which * slots;
            const int head = head0 + which / 2;
            const int64_t data = page * c.s_page + head * c.s_head + slot * c.s_slot + 8 * g;
            const int64_t scales = page * c.t_page + head * c.t_head + slot * c.t_slot + g;
            w[i] = *reinterpret_cast<const uint2 *>((which & 1 ? c.v : c.k) + data);
            scale[i] = (which & 1 ? c.vs : c.ks)[scales];
            dst[i] = (which & 1 ? p.v : p.k) + to + ((int64_t)head * c.page_size + slot) * c.D + 16 * g;
            both[i] = 16 * g + 8 < c.D;
        }
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            if (!dst[i]) continue;
            reinterpret_cast<uint4 *>(dst[i])[0] = rows_from_four<kF16>(w[i].x, scale[i]);
            if (both[i]) reinterpret_cast<uint4 *>(dst[i])[1] = rows_from_four<kF16>(w[i].y, scale[i]);
        }
    }
}

}  // namespace

cudaError_t launch_widen_pages(WidenParams p, int64_t pages, cudaStream_t stream)
{
    const int64_t groups = (p.c.D + kFourGroup - 1) / kFourGroup, head = 2 * p.c.page_size * groups;
    p.by_groups = make_fast_div((uint32_t)groups);
    p.heads = (int)(head >= kWideTasks ? 1 : kWideTasks / head < p.c.Hkv ? kWideTasks / head : p.c.Hkv);
    p.parts = (p.c.Hkv + p.heads - 1) / p.heads;
    const dim3 grid((unsigned)(pages * p.parts));
    return p.f16 ? launch_behind(widen_pages_kernel<true>, grid, kWideThreads, 0, stream, p)
                 : launch_behind(widen_pages_kernel<false>, grid, kWideThreads, 0, stream, p);
}

}  // namespace fa
