// fa_four_rows.h -- parameters of the attention kernels over a 4-bit cache, shared by
// their host checks (fa_four_api.cu) and the kernels (not part of the public C ABI).
#pragma once

#include "fa_paged.h"

namespace fa {

// p.c has the table, the lengths and the sizes; c the pools.
struct FourParams {
    PagedParams p;
    PagedCache4 c;
};

struct WidenParams {
    PagedCache4 c;
    uint16_t *k, *v;                   // [B * width, Hkv, page_size, D]
    int32_t *table, *seq_len;          // [B, width], [B]
    int f16;
    // set by the launcher: 16 elements, of a row; heads of a CTA, CTAs of a page
    FastDiv by_groups;
    int heads, parts;
};

int four_rows_per_tile(int D, int64_t rows);
int four_rows_chunk(int D);
int four_rows_ctas_per_sm(int D, int rows);
cudaError_t launch_four_rows(const FourParams &f, int ctas, cudaStream_t stream);
// A team of p.team CTAs per tile of 8 rows, and how many teams fit the device together.
cudaError_t launch_four_team(const FourParams &f, int ctas, cudaStream_t stream);
int four_teams_at_once(int device, int team);
// Tiles of 128 rows on the tensor cores (fa_paged_tc.cu), D <= 128.
cudaError_t launch_four_tc(const FourParams &f, int ctas, cudaStream_t stream);
cudaError_t launch_widen_pages(WidenParams p, int64_t pages, cudaStream_t stream);

}  // namespace fa
