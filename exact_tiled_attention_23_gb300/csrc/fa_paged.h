// fa_paged.h -- parameters of the paged-cache kernels, shared by their host
// checks (fa_paged_api.cu) and the kernels (not part of the public C ABI).
#pragma once

#include "fa.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace fa {

// A sequence's keys and values through the page table.  `table` has one row
// of `table_width` page numbers per sequence, `table_stride` entries apart.
struct PagedCache {
    uint16_t *k, *v;
    int64_t s_page, s_head, s_slot;    // strides in elements, the same for k and v
    const int32_t *table;
    int64_t table_stride;
    const int32_t *seq_len;            // null: every sequence has fixed_len keys
    int table_width;
    int num_pages, page_size;
    int fixed_len;
    int Hkv, D;
};

struct AppendParams {
    PagedCache c;
    const uint16_t *k, *v, *q;         // [B, H, T, D] through the strides below; q may be null
    uint16_t *q_out;
    int64_t k_s[3], v_s[3], q_s[3], qo_s[3];   // batch, head, token
    const float *inv_freq;             // [rot / 2]
    int64_t offset;                    // position of a sequence's first key
    int B, T, Hq, rot, interleaved, f16;
};

// Partial softmax states of row tiles, which the merge joins.  A tile is
// `rows` stacked query rows of one (sequence, key head), in the order of
// fa_paged_line.cuh.  Its states are in slots, each `rows` normalised fp32
// outputs of D columns and `rows` base-2 log-sum-exps.
struct Partials {
    float *o;              // [slots][rows][D]
    float *lse;            // [slots][rows]
    int rows;              // stacked query rows per tile
    int tiles;             // row tiles per (sequence, key head)
    int stacked;           // 1: one list of tiles for all sequences (a shared prefix)
    int chunk;             // keys per chunk of the line
    // Tile i has the slots k + i of the CTAs k that had a share of its chunks.
    // They follow from the tile's first chunk and the chunks per CTA.  (Along
    // the line, k and i never fall and one of them grows from share to share,
    // so no two shares have one slot.)
    int64_t *first_chunk;  // [tiles in all]
    int64_t *per_cta;      // [1]
    int fixed_len;         // stacked: keys of the prefix
};

struct PagedParams {
    PagedCache c;
    const uint16_t *q;
    int64_t q_s[3];                    // batch, head, token
    uint16_t *o;
    int64_t o_s[3];
    float *lse;                        // [B, Hq, T] or null
    int B, T, Hq, G;                   // G = Hq / Hkv query heads share a key head
    int causal, f16;
    float scale_log2;
    int joined;                        // 1: every tile leaves its state in a slot for the merge
    Partials part;
    int box_rows;                      // tensor-core kernel: key rows per copied box
    uint64_t wait_limit_ns;
};

struct MergeParams {
    Partials src[2];
    int n_src;
    const int32_t *seq_len;
    int max_len;
    uint16_t *o;
    int64_t o_s[3];
    float *lse;
    int B, T, Hq, G, D, causal, f16;
    int joined;                        // 0: a tile that one CTA finished is written already
};

// Keys per chunk of the line: the row kernel's, and the tensor-core kernel's.
constexpr int kChunkKeys = 64;
constexpr int kBlockKeys = 128;

// Query rows per tile, and CTAs per SM, of the row kernel.
int paged_rows_per_tile(int D, int64_t rows);
int paged_rows_ctas_per_sm(int D);

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
cudaError_t launch_paged_rows(const PagedParams &p, int ctas, cudaStream_t stream);
cudaError_t launch_paged_tc(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                            cudaStream_t stream);
cudaError_t launch_paged_merge(const MergeParams &p, cudaStream_t stream);

}  // namespace fa
