// fa_pages_api.cu -- the C ABI of what manages a cache's pages: argument checks,
// workspace layout and launches.  Declared in include/fa.h.
//
// Every check that can fail runs before any launch, so a rejected call has no side
// effect.  The library allocates no device memory.
#include "fa_pages.h"
#include "fa_paged_plan.h"

namespace {

using namespace fa::paged;

// (Kernels count pages, rows and forks in 32 bits, a CTA's threads at a time.)
constexpr int kMostEntries = INT32_MAX - 1024;

fa_status check_table(const fa_page_table *t)
{
    if (!t || t->B < 0 || t->table_width < 0 || t->num_pages < 0 || t->page_size <= 0) return FA_ERR_INVALID_ARG;
    if ((t->B > 0 && (!t->seq_len || (t->table_width > 0 && !t->table))) || (t->num_pages > 0 && !t->refs)) return FA_ERR_INVALID_ARG;
    if (!aligned(t->seq_len, 4) || !aligned(t->table, 4) || !aligned(t->refs, 4)) return FA_ERR_INVALID_ARG;
    if (t->B > 1 && t->table_stride < t->table_width) return FA_ERR_INVALID_ARG;
    if ((int64_t)t->table_width * t->page_size > kMostKeys) return FA_ERR_INVALID_ARG;
    const int64_t parts = (t->table_width + 2047ll) / 2048;
    if (parts * t->B > kMostEntries || t->num_pages > kMostEntries) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// The table, and the workspace's parts in order; returns its bytes.
size_t place(fa::PagesParams &p, const fa_page_table &t, int n, void *workspace, bool all = false)
{
    p.table = t.table;
    p.table_stride = t.table_stride;
    p.seq_len = t.seq_len;
    p.refs = t.refs;
    p.width = t.table_width;
    p.B = t.B;
    p.num_pages = t.num_pages;
    p.page_size = t.page_size;
    p.n = n;
    p.segments = fa::page_segments(t.num_pages, all);
    p.segment = (t.num_pages + p.segments - 1) / p.segments;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        void *r = base ? base + at : nullptr;
        at += round_up(bytes);
        return r;
    };
    p.counts = static_cast<int32_t *>(take((size_t)fa::kMostSegments * 4));
    p.count = static_cast<int32_t *>(take(4));
    p.list = static_cast<int32_t *>(take((size_t)t.num_pages * 4));
    p.src = static_cast<int32_t *>(take((size_t)std::max(t.num_pages, n) * 4));
    p.mark = static_cast<int32_t *>(take((size_t)t.B * 4));
    p.first = static_cast<int64_t *>(take((size_t)t.B * 8));
    return at;
}

fa_status with_workspace(fa::PagesParams &p, const fa_page_table &t, int n, void *workspace, size_t bytes, bool all = false)
{
    const size_t need = place(p, t, n, workspace, all);
    return workspace && aligned(workspace, 16) && bytes >= need ? FA_OK : FA_ERR_INVALID_ARG;
}

bool vector_ok(const int32_t *x, int n) { return n == 0 || (n <= kMostEntries && x && aligned(x, 4)); }

fa_status status_of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// One array of a pool.  Strides and row_bytes in bytes.
fa::PageArray array_of(void *base, int64_t s_page, int64_t s_head, int64_t s_slot, int row_bytes, int Hkv, int slots)
{
    fa::PageArray a{};
    a.base = static_cast<uint8_t *>(base);
    a.s_page = s_page;
    a.s_head = s_head;
    a.s_slot = s_slot;
    a.row_bytes = row_bytes;
    a.slots = slots;
    a.bytes = (int64_t)Hkv * slots * row_bytes;
    a.parts = fa::copy_parts(a.bytes);
    const bool slots_in = (slots == 1 || s_slot == row_bytes) && (Hkv == 1 || s_head == (int64_t)slots * row_bytes);
    const bool heads_in = (Hkv == 1 || s_head == row_bytes) && (slots == 1 || s_slot == (int64_t)Hkv * row_bytes);
    a.dense = slots_in || heads_in;
    const bool wide = s_page % 16 == 0 && (a.dense ? a.bytes % 16 == 0 : row_bytes % 16 == 0 && s_head % 16 == 0 && s_slot % 16 == 0);
    a.unit = wide ? 16 : 4;
    return a;
}

fa_status copy(fa::CopyParams &p, int num_pages, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream)
{
    if (n < 0 || !vector_ok(src, n) || !vector_ok(dst, n) || !aligned(count, 4)) return FA_ERR_INVALID_ARG;
    if (n == 0 || num_pages == 0) return FA_OK;
    p.num_pages = num_pages;
    for (int i = 0; i < p.arrays; ++i) p.parts += p.a[i].parts;
    p.n = n;
    p.src = src;
    p.dst = dst;
    p.count = count;
    return status_of(fa::launch_copy(p, fa::sm_count_of(fa::current_device()), static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t fa_pages_workspace_bytes(const fa_page_table *table, int n)
{
    if (check_table(table) != FA_OK || n < 0 || n > kMostEntries) return 0;
    fa::PagesParams p{};
    return place(p, *table, n, nullptr);
}

fa_status fa_kv_grow(const fa_page_table *table, const int32_t *tokens, int32_t *taken, void *workspace, size_t workspace_bytes,
                     void *stream)
{
    fa_status st = check_table(table);
    if (st != FA_OK) return st;
    if (table->B == 0) return FA_OK;
    if (!vector_ok(tokens, table->B) || !vector_ok(taken, table->B)) return FA_ERR_INVALID_ARG;
    fa::PagesParams p{};
    st = with_workspace(p, *table, 0, workspace, workspace_bytes);
    if (st != FA_OK) return st;
    p.tokens = tokens;
    p.taken = taken;
    return status_of(fa::launch_grow(p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_free(const fa_page_table *table, const int32_t *rows, int n, void *stream)
{
    const fa_status st = check_table(table);
    if (st != FA_OK) return st;
    if (n < 0 || !vector_ok(rows, n)) return FA_ERR_INVALID_ARG;
    if (n == 0 || table->B == 0) return FA_OK;
    fa::PagesParams p{};
    place(p, *table, n, nullptr);
    p.rows = rows;
    return status_of(fa::launch_free(p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_fork(const fa_page_table *table, const int32_t *parent, const int32_t *child, int n, int32_t *src, int32_t *dst,
                     void *workspace, size_t workspace_bytes, void *stream)
{
    fa_status st = check_table(table);
    if (st != FA_OK) return st;
    if (n < 0 || !vector_ok(parent, n) || !vector_ok(child, n) || !vector_ok(src, n) || !vector_ok(dst, n)) return FA_ERR_INVALID_ARG;
    if (n == 0) return FA_OK;
    fa::PagesParams p{};
    st = with_workspace(p, *table, n, workspace, workspace_bytes);
    if (st != FA_OK) return st;
    p.parent = parent;
    p.rows = child;
    p.src = src;
    p.taken = dst;
    return status_of(fa::launch_fork(p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_kv_compact(const fa_page_table *table, int32_t *moved, int32_t *src, int32_t *dst, int32_t *count, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    fa_status st = check_table(table);
    if (st != FA_OK) return st;
    if (!vector_ok(moved, table->num_pages) || !vector_ok(src, table->num_pages) || !vector_ok(dst, table->num_pages) || !count ||
        !aligned(count, 4))
        return FA_ERR_INVALID_ARG;
    fa::PagesParams p{};
    st = with_workspace(p, *table, 0, workspace, workspace_bytes, true);
    if (st != FA_OK) return st;
    p.taken = moved;
    p.src = src;
    p.list = dst;
    p.count = count;
    return status_of(fa::launch_compact(p, static_cast<cudaStream_t>(stream)));
}

fa_status fa_copy_pages(const fa_paged_kv *cache, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream)
{
    const fa_status st = check_cache(cache, 0);
    if (st != FA_OK) return st;
    if ((int64_t)cache->Hkv * cache->page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
    fa::CopyParams p{};
    for (void *x : {cache->k, cache->v})
        p.a[p.arrays++] = array_of(x, 2 * cache->stride_page, 2 * cache->stride_head, 2 * cache->stride_slot, 2 * cache->D,
                                   cache->Hkv, cache->page_size);
    return copy(p, cache->num_pages, src, dst, count, n, stream);
}

fa_status fa_copy_pages_q4(const fa_paged_kv4 *cache, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream)
{
    const fa_status st = check_cache4(cache, 0);
    if (st != FA_OK) return st;
    if ((int64_t)cache->Hkv * cache->page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
    const int P = fa::padded4(cache->D);
    fa::CopyParams p{};
    for (void *x : {cache->k, cache->v})
        p.a[p.arrays++] = array_of(x, cache->stride_page, cache->stride_head, cache->stride_slot, P / 2, cache->Hkv, cache->page_size);
    for (void *x : {cache->k_scales, cache->v_scales})
        p.a[p.arrays++] = array_of(x, cache->scale_stride_page, cache->scale_stride_head, cache->scale_stride_slot, P / 16,
                                   cache->Hkv, cache->page_size);
    return copy(p, cache->num_pages, src, dst, count, n, stream);
}

}  // extern "C"
