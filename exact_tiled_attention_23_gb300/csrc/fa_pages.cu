// fa_pages.cu -- the pages of a cache: taken by sequences that grow, shared and
// copied by sequences that fork, given up, moved together, and copied.
//
// refs[p] counts the uses of page p; a page with no use is free.  Whatever takes
// pages takes the lowest free ones, in order, so that results depend on nothing
// but the inputs.  What decides who gets which page is a prefix sum, over sequences
// and over pages: one CTA has it for pools up to kOneList pages, until it has found as
// many as are needed, and for more the pages are counted and listed in segments, one
// CTA each.
//
// Bound by latency but for the pages' data: a copy reads and writes every byte once
// (441 MB 68 us, 6.5 TB/s).  Eight of 256 sequences end and eight others take about
// 1000 pages, 34000 pages in the pool: 10.5 us.  64 forks with a copied page of 256 KB
// each: 15 us, of which 5.5 are the copies.
#include "fa_pages.h"
#include "sm103_ptx.cuh"

namespace fa {

namespace {

constexpr int kThreads = 1024;         // of a CTA that sums
constexpr int kWarps = kThreads / 32;
// Pages that one CTA lists by itself, and of a CTA's segment beyond that at least.  64
// sequences take a page each of 65536, half of them free, or one in a hundred: one CTA
// 8.9 and 18.4 us, four 10.1 and 10.2, with two launches (6 us of the host) more.
constexpr int kOneList = 65536, kSegment = 16384;
// Where all pages are looked at, not only as many as are needed: compactions of 8192,
// 16384, 65536 and 262144 pages in segments of 4096 15.0, 17.8, 28 and 69 us, of 16384
// 16.6, 26.8, 38 and 75, in one 16.4, 26.4, 81 and 299.
constexpr int kAllSegment = 4096;

// The sums of x over the threads in front of each, after `base`, which the sum of all
// is added to.  `sums` has two rows that take turns, so that one barrier is enough.
template <typename N>
__device__ __forceinline__ N scan(N x, N &base, N (*sums)[kWarps], int &turn)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    N up = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += y;
    }
    if (lane == 31) sums[turn][warp] = up;
    __syncthreads();
    N all = sums[turn][lane];
    turn ^= 1;
    const N mine = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const N y = __shfl_up_sync(0xffffffffu, all, d);
        if (lane >= d) all += y;
    }
    const N before = __shfl_sync(0xffffffffu, all - mine, warp);
    const N result = base + before + up - x;
    base += __shfl_sync(0xffffffffu, all, 31);
    return result;
}

// Live pages of [first, last), summed over the CTA.
__device__ int count_live(const int32_t *refs, int first, int last)
{
    constexpr int kWide = 8;               // loads together
    __shared__ int total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    int n = 0;
    for (int64_t at = first + (int64_t)threadIdx.x; at < last; at += kThreads * kWide) {
        bool live[kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) live[i] = at + i * kThreads < last && refs[at + i * kThreads] > 0;
#pragma unroll
        for (int i = 0; i < kWide; ++i) n += live[i];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x % 32 == 0 && n) atomicAdd(&total, n);
    __syncthreads();
    const int result = total;
    __syncthreads();
    return result;
}

// each(p, live, live pages of [first, last) in front of p) for every page of
// [first, last), `before` added, until `enough` pages were free.  Returns how many
// pages were live, `before` added, and `last` or how far it came.
template <typename Each>
__device__ __forceinline__ int walk(const int32_t *refs, int first, int &last, int before, int64_t enough, int (*sums)[kWarps],
                                    int &turn, const Each &each)
{
    constexpr int kWide = 8;           // pages of a thread, loaded together
    const int from = first - before;
    for (int64_t at = first; at < last; at += kThreads * kWide) {
        if (at - before - from >= enough) {
            last = (int)at;
            break;
        }
        const int64_t p = at + (int64_t)threadIdx.x * kWide;
        bool live[kWide];
        int n = 0;
#pragma unroll
        for (int i = 0; i < kWide; ++i) live[i] = p + i < last && refs[p + i] > 0;
#pragma unroll
        for (int i = 0; i < kWide; ++i) n += live[i];
        int front = scan(n, before, sums, turn);
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
            if (p + i < last) each((int)(p + i), live[i], front);
            front += live[i];
        }
    }
    return before;
}

__device__ __forceinline__ int segment_first(const PagesParams &p, int s) { return (int)min((int64_t)s * p.segment, (int64_t)p.num_pages); }

// Live pages in front of this CTA's segment, and in all.
__device__ __forceinline__ int live_before(const PagesParams &p, int &all)
{
    int before = 0;
    all = 0;
    for (int s = 0; s < p.segments; ++s) {
        if (s == (int)blockIdx.x) before = all;
        all += p.counts[s];
    }
    return before;
}

__global__ void __launch_bounds__(kThreads) count_kernel(const PagesParams p)
{
    ptx::wait_for_primary();
    const int n = count_live(p.refs, segment_first(p, blockIdx.x), segment_first(p, blockIdx.x + 1));
    if (threadIdx.x == 0) p.counts[blockIdx.x] = n;
}

// The free pages of [first, last) in order, after `before` live pages in front, until
// there are `enough`.  Returns how many were listed.
__device__ __forceinline__ int list_free(const PagesParams &p, int first, int last, int before, int64_t enough)
{
    __shared__ int sums[2][kWarps];
    int turn = 0;
    const int live = walk(p.refs, first, last, before, enough, sums, turn, [&](int page, bool is, int front) {
        if (!is) p.list[page - front] = page;
    });
    return last - first - (live - before);
}

__global__ void __launch_bounds__(kThreads) list_kernel(const PagesParams p)
{
    ptx::wait_for_primary();
    int all;
    const int before = live_before(p, all);
    list_free(p, segment_first(p, blockIdx.x), segment_first(p, blockIdx.x + 1), before, INT32_MAX);
}

// How many free pages p.list has, `enough` or all; lists them where no kernel before
// did.
__device__ __forceinline__ int free_pages(const PagesParams &p, int64_t enough)
{
    if (p.segments > 1) {
        int all;
        live_before(p, all);
        return p.num_pages - all;
    }
    return list_free(p, 0, p.num_pages, 0, enough);
}

__device__ __forceinline__ int64_t capacity(const PagesParams &p) { return (int64_t)p.width * p.page_size; }

__device__ __forceinline__ int64_t length_of(const PagesParams &p, int b)
{
    const int n = p.seq_len[b];
    return n < 0 ? 0 : min((int64_t)n, capacity(p));
}

__device__ __forceinline__ int64_t pages_of(const PagesParams &p, int64_t n) { return (n + p.page_size - 1) / p.page_size; }

// What sequence b has, what it needs to grow (none where its row is too short), and
// whether that is so.
struct Growth {
    int64_t n, then, have, need;
    bool room;
};

__device__ __forceinline__ Growth growth_of(const PagesParams &p, int64_t b)
{
    Growth g{0, 0, 0, 0, false};
    if (b >= p.B) return g;
    g.n = length_of(p, (int)b);
    g.then = g.n + max(p.tokens[b], 0);
    g.room = g.then <= capacity(p);
    g.have = pages_of(p, g.n);
    if (g.room) g.need = pages_of(p, g.then) - g.have;
    return g;
}

// Sequences grow: who gets which free pages is the prefix sum of what they need.  A
// thread has a sequence, and takes one page itself; the pages of those that need more
// are all warps' work, 32 at a time.
__global__ void __launch_bounds__(kThreads) grow_kernel(const PagesParams p)
{
    __shared__ int64_t sums[2][kWarps];
    struct Many {
        int sequence, have, need, first;
    };
    __shared__ Many many[kThreads];
    __shared__ int queued;
    int turn = 0;
    int64_t total = 0;
    if (threadIdx.x == 0) queued = 0;
    ptx::wait_for_primary();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    Growth g{};
    int64_t first = 0;
    for (int64_t at = 0; at < p.B; at += kThreads) {
        g = growth_of(p, at + threadIdx.x);
        first = scan(g.need, total, sums, turn);
        if (p.B > kThreads && at + threadIdx.x < p.B) p.first[at + threadIdx.x] = first;
    }
    __syncthreads();
    const int found = free_pages(p, total);
    __syncthreads();
    for (int64_t at = 0; at < p.B; at += kThreads) {
        const int64_t b = at + threadIdx.x;
        if (p.B > kThreads) {
            g = growth_of(p, b);
            first = b < p.B ? p.first[b] : 0;
        }
        const bool fits = g.room && (g.need == 0 || first + g.need <= found);
        if (b < p.B) {
            if (fits && g.need == 1) {
                const int page = p.list[first];
                p.table[b * p.table_stride + g.have] = page;
                p.refs[page] = 1;
            }
            if (fits && g.then > g.n) p.seq_len[b] = (int)g.then;
            p.taken[b] = fits ? (int)g.need : kRefused;
        }
        if (fits && g.need > 1) many[atomicAdd(&queued, 1)] = Many{(int)b, (int)g.have, (int)g.need, (int)first};
        __syncthreads();
        const int items = queued;
        for (int i = 0; i < items; ++i) {
            const Many x = many[i];
            // (another warp begins each, so that short ones are spread, too)
            for (int64_t j = (int64_t)((warp - i) & (kWarps - 1)) * 32 + lane; j < x.need; j += kThreads) {
                const int page = p.list[x.first + j];
                p.table[x.sequence * p.table_stride + x.have + j] = page;
                p.refs[page] = 1;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) queued = 0;
        __syncthreads();
    }
}

// A row gives up its pages: a CTA each.
__global__ void __launch_bounds__(256) free_kernel(const PagesParams p)
{
    ptx::wait_for_primary();
    const int row = p.rows[blockIdx.x];
    bool again = row < 0 || row >= p.B;
    for (int j = threadIdx.x; j < (int)blockIdx.x; j += 256) again |= p.rows[j] == row;
    if (__syncthreads_or(again)) return;
    const int64_t have = pages_of(p, length_of(p, row));
    for (int64_t e = threadIdx.x; e < p.width; e += 256) {
        int32_t *entry = p.table + row * p.table_stride + e;
        if (e < have) {
            const int page = *entry;
            // (a count that is 0 already stays 0)
            if (page >= 0 && page < p.num_pages && atomicSub(p.refs + page, 1) <= 0) atomicAdd(p.refs + page, 1);
        }
        *entry = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.seq_len[row] = 0;
}

// Forks: which are valid, and which pages the part-full pages are copied to.
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const PagesParams p)
{
    __shared__ int sums[2][kWarps];
    int turn = 0, base = 0;
    ptx::wait_for_primary();
    // a child has its first fork's number, all other rows none: what a second fork of a
    // child, or a fork of a child, gives would depend on the order
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const int x = p.parent[i], y = p.rows[i];
        if (x >= 0 && x < p.B) p.mark[x] = INT32_MAX;
        if (y >= 0 && y < p.B) p.mark[y] = INT32_MAX;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kThreads) {
        const int y = p.rows[i];
        if (y >= 0 && y < p.B) atomicMin(p.mark + y, i);
    }
    __syncthreads();
    const int found = free_pages(p, p.n);
    __syncthreads();
    for (int at = 0; at < p.n; at += kThreads) {
        const int i = at + threadIdx.x;
        bool ok = false;
        int src = -1;
        if (i < p.n) {
            const int x = p.parent[i], y = p.rows[i];
            // (atomics went to the L2: read there)
            ok = x >= 0 && x < p.B && y >= 0 && y < p.B && __ldcg(p.mark + y) == i && __ldcg(p.mark + x) == INT32_MAX &&
                 p.seq_len[y] <= 0;
            if (ok) {
                const int64_t n = length_of(p, x);
                if (n % p.page_size != 0) src = p.table[x * p.table_stride + n / p.page_size];
                if (src < 0 || src >= p.num_pages) src = -1;
            }
        }
        const int rank = scan(src >= 0 ? 1 : 0, base, sums, turn);
        if (i < p.n) {
            int dst = ok ? -1 : kRefused;
            if (src >= 0) dst = rank < found ? p.list[rank] : kRefused;
            if (src >= 0 && dst >= 0) p.refs[dst] = 1;
            p.src[i] = dst >= 0 ? src : -1;
            p.taken[i] = dst;
        }
    }
}

// The rows of the forks that are valid: a CTA each.
__global__ void __launch_bounds__(256) fork_rows_kernel(const PagesParams p)
{
    ptx::wait_for_primary();
    const int copied = p.taken[blockIdx.x];
    if (copied == kRefused) return;
    const int x = p.parent[blockIdx.x], y = p.rows[blockIdx.x];
    const int64_t n = length_of(p, x), have = pages_of(p, n);
    for (int64_t e = threadIdx.x; e < p.width; e += 256) {
        int page = -1;
        if (e < have) {
            page = p.table[x * p.table_stride + e];
            if (copied >= 0 && e == have - 1)
                page = copied;
            else if (page >= 0 && page < p.num_pages)
                atomicAdd(p.refs + page, 1);
        }
        p.table[y * p.table_stride + e] = page;
    }
    if (threadIdx.x == 0) p.seq_len[y] = (int)n;
}

// With L live pages, the live pages from L on move into the holes in front of L, both
// in order: p.src and p.list.  p.taken has a page's new number, or kMove less its place
// in the lists until finish_kernel has been there.
constexpr int kMove = -3;

__global__ void __launch_bounds__(kThreads) compact_kernel(const PagesParams p)
{
    __shared__ int sums[2][kWarps];
    int turn = 0;
    ptx::wait_for_primary();
    const bool alone = p.segments == 1;
    int live, before = 0;
    if (alone)
        live = count_live(p.refs, 0, p.num_pages);
    else
        before = live_before(p, live);
    // live pages in front of L: those of whole segments, and of L's own
    int kept = 0, first = 0;
    if (!alone)
        for (int s = 0; segment_first(p, s + 1) <= live && s < p.segments; ++s) {
            kept += p.counts[s];
            first = segment_first(p, s + 1);
        }
    kept += count_live(p.refs, first, live);
    int last = segment_first(p, blockIdx.x + 1);
    walk(p.refs, segment_first(p, blockIdx.x), last, before, INT32_MAX, sums, turn, [&](int page, bool is, int front) {
        p.taken[page] = !is ? -1 : page < live ? page : kMove - (front - kept);
        if (!is && page < live) p.list[page - front] = page;
        if (is && page >= live) p.src[front - kept] = page;
    });
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = live - kept;
}

// Numbers and counts of the pages that move (the first CTAs), and the tables (the
// rest: one per row and kRemap entries).  An entry's page has its new number in
// p.taken, or still its place in the list.
constexpr int kRemap = 2048;

__global__ void __launch_bounds__(256) finish_kernel(const PagesParams p, const int movers)
{
    ptx::wait_for_primary();
    if ((int)blockIdx.x < movers) {
        for (int64_t j = blockIdx.x * 256ll + threadIdx.x; j < *p.count; j += movers * 256ll) {
            const int src = p.src[j], dst = p.list[j];
            p.taken[src] = dst;
            p.refs[dst] = p.refs[src];
            p.refs[src] = 0;
        }
        return;
    }
    const int block = (int)blockIdx.x - movers;
    const int parts = (p.width + kRemap - 1) / kRemap, b = block / parts, part = block % parts;
    const int64_t have = pages_of(p, length_of(p, b)), first = (int64_t)part * kRemap;
    for (int64_t e = first + threadIdx.x; e < min(have, first + kRemap); e += 256) {
        int32_t *entry = p.table + b * p.table_stride + e;
        const int page = *entry;
        if (page < 0 || page >= p.num_pages) continue;
        const int t = __ldcg(p.taken + page);               // (other CTAs write it)
        const int to = t <= kMove ? p.list[kMove - t] : t;
        if (to >= 0 && to != page) *entry = to;             // (a page that nobody counted stays)
    }
}

// ------------------------------------------------------------------ the data
// A warp takes kPart bytes of a page of one array at a time.
constexpr int kPart = 4096;

template <typename Unit>
__device__ __forceinline__ void copy_part(const PageArray &a, const uint8_t *src, uint8_t *dst, int64_t from, int lane)
{
    constexpr int kSize = sizeof(Unit), kMany = 8;
    const int64_t end = min(from + kPart, a.bytes);
    for (int64_t at = from + lane * kSize; at < end; at += 32 * kSize * kMany) {
        Unit x[kMany];
        int64_t off[kMany];
#pragma unroll
        for (int i = 0; i < kMany; ++i) {
            const int64_t o = at + i * 32 * kSize;
            off[i] = -1;
            if (o < end) {
                off[i] = o;
                if (!a.dense) {
                    const int64_t row = o / a.row_bytes, head = row / a.slots;
                    off[i] = head * a.s_head + (row - head * a.slots) * a.s_slot + (o - row * a.row_bytes);
                }
                x[i] = *reinterpret_cast<const Unit *>(src + off[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kMany; ++i)
            if (off[i] >= 0) *reinterpret_cast<Unit *>(dst + off[i]) = x[i];
    }
}

__global__ void __launch_bounds__(256) copy_kernel(const CopyParams p)
{
    ptx::wait_for_primary();
    const int lane = threadIdx.x % 32;
    const int64_t n = p.count ? min((int64_t)*p.count, p.n) : p.n;
    const int64_t warps = (int64_t)gridDim.x * 8;
    for (int64_t item = blockIdx.x * 8ll + threadIdx.x / 32; item < n * p.parts; item += warps) {
        const int64_t j = item / p.parts;
        int64_t part = item - j * p.parts;
        const int from = p.src[j], to = p.dst[j];
        if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages || from == to) continue;
        int which = 0;
        while (part >= p.a[which].parts) part -= p.a[which++].parts;
        const PageArray &a = p.a[which];
        const uint8_t *src = a.base + from * a.s_page;
        uint8_t *dst = a.base + to * a.s_page;
        if (a.unit == 16)
            copy_part<uint4>(a, src, dst, part * kPart, lane);
        else
            copy_part<uint32_t>(a, src, dst, part * kPart, lane);
    }
}

// Segments of the pool, and counts of them where there is more than one.
cudaError_t count_segments(const PagesParams &p, cudaStream_t stream)
{
    if (p.segments == 1) return cudaSuccess;
    return launch_behind(count_kernel, dim3((unsigned)p.segments), kThreads, 0, stream, p);
}

cudaError_t list_segments(const PagesParams &p, cudaStream_t stream)
{
    const cudaError_t e = count_segments(p, stream);
    if (e != cudaSuccess || p.segments == 1) return e;
    return launch_behind(list_kernel, dim3((unsigned)p.segments), kThreads, 0, stream, p);
}

}  // namespace

int page_segments(int num_pages, bool all)
{
    const int size = all ? kAllSegment : kSegment;
    if (num_pages <= (all ? kAllSegment : kOneList)) return 1;
    const int n = (num_pages - 1) / size + 1;
    return n < kMostSegments ? n : kMostSegments;
}

int64_t copy_parts(int64_t bytes) { return (bytes + kPart - 1) / kPart; }

cudaError_t launch_grow(const PagesParams &p, cudaStream_t stream)
{
    const cudaError_t e = list_segments(p, stream);
    return e != cudaSuccess ? e : launch_behind(grow_kernel, dim3(1), kThreads, 0, stream, p);
}

cudaError_t launch_free(const PagesParams &p, cudaStream_t stream)
{
    return launch_behind(free_kernel, dim3((unsigned)p.n), 256, 0, stream, p);
}

cudaError_t launch_fork(const PagesParams &p, cudaStream_t stream)
{
    cudaError_t e = list_segments(p, stream);
    if (e == cudaSuccess) e = launch_behind(fork_plan_kernel, dim3(1), kThreads, 0, stream, p);
    if (e == cudaSuccess) e = launch_behind(fork_rows_kernel, dim3((unsigned)p.n), 256, 0, stream, p);
    return e;
}

cudaError_t launch_compact(const PagesParams &p, cudaStream_t stream)
{
    cudaError_t e = count_segments(p, stream);
    if (e == cudaSuccess) e = launch_behind(compact_kernel, dim3((unsigned)p.segments), kThreads, 0, stream, p);
    const int64_t rows = (int64_t)p.B * ((p.width + kRemap - 1) / kRemap);
    const int movers = p.num_pages / 2048 + 1 < 152 ? p.num_pages / 2048 + 1 : 152;
    if (e == cudaSuccess) e = launch_behind(finish_kernel, dim3((unsigned)(movers + rows)), 256, 0, stream, p, movers);
    return e;
}

cudaError_t launch_copy(const CopyParams &p, int sms, cudaStream_t stream)
{
    const int64_t need = (p.n * p.parts + 7) / 8, most = (int64_t)sms * 8;
    return launch_behind(copy_kernel, dim3((unsigned)(need < most ? need : most)), 256, 0, stream, p);
}

}  // namespace fa
