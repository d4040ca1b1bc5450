// fa_pages.h -- parameters of the kernels that manage a cache's pages, shared by
// their host checks (fa_pages_api.cu) and the kernels (not part of the public C ABI).
#pragma once

#include "fa_paged.h"

namespace fa {

// What is said of a sequence or a fork that could not be served.
constexpr int kRefused = -2;

struct PagesParams {
    int32_t *table;                    // [B, width], rows table_stride entries apart
    int64_t table_stride;
    int32_t *seq_len;                  // [B]
    int32_t *refs;                     // [num_pages]
    int width, B, num_pages, page_size;
    int n;                             // rows, or forks
    const int32_t *rows;               // [n] rows to free; the children of forks
    const int32_t *parent;             // [n]
    const int32_t *tokens;             // [B]
    int32_t *taken;                    // the answer: [B], [n] or [num_pages]
    // workspace
    int segments, segment;             // of the pool, pages of each
    int32_t *counts;                   // [segments] live pages
    int32_t *list;                     // [num_pages] free pages; holes that are filled
    int32_t *src;                      // [n] or [num_pages] pages that are copied
    int32_t *mark;                     // [B]
    int64_t *first;                    // [B]
    int32_t *count;                    // moves
};

// One of the arrays of a pool.
struct PageArray {
    uint8_t *base;
    int64_t s_page, s_head, s_slot;    // bytes
    int64_t bytes, parts;              // of a page; what a warp copies at a time
    int row_bytes, slots, unit, dense; // dense: a page's bytes are one block
};

struct CopyParams {
    PageArray a[4];
    int arrays, num_pages;
    int64_t parts, n;                  // parts of a page in all arrays; pairs
    const int32_t *src, *dst, *count;  // count: how many pairs, if not n
};

// Segments that a pool is listed in (all: to its end, whatever is needed), and parts of
// a page of so many bytes.
constexpr int kMostSegments = 128;
int page_segments(int num_pages, bool all);
int64_t copy_parts(int64_t bytes);

cudaError_t launch_grow(const PagesParams &p, cudaStream_t stream);
cudaError_t launch_free(const PagesParams &p, cudaStream_t stream);
cudaError_t launch_fork(const PagesParams &p, cudaStream_t stream);
cudaError_t launch_compact(const PagesParams &p, cudaStream_t stream);
cudaError_t launch_copy(const CopyParams &p, int sms, cudaStream_t stream);

}  // namespace fa
