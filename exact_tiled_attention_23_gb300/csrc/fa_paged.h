// fa_paged.h -- parameters of the paged-cache kernels, shared by their host
// checks (fa_paged_api.cu) and the kernels (not part of the public C ABI).
#pragma once

#include "fa.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

namespace fa {

// Division of n < 2^31 by a number known on the host: with s = ceil(log2 d)
// and mul = ceil(2^(31+s) / d) < 2^32, mul * d exceeds 2^(31+s) by less than
// 2^s, so floor(n * mul / 2^(31+s)) = floor(n / d).
struct FastDiv {
    uint32_t mul, shift, by;
#ifdef __CUDACC__
    __device__ __forceinline__ int quotient(int n) const
    {
        return (int)(((uint64_t)(uint32_t)n * mul) >> shift);
    }
#endif
};

inline FastDiv make_fast_div(uint32_t d)
{
    uint32_t s = 0;
    while (((uint64_t)1 << s) < d) ++s;
    const uint64_t top = (uint64_t)1 << (31 + s);
    return FastDiv{(uint32_t)((top + d - 1) / d), 31 + s, d};
}

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
    FastDiv by_page;                   // page_size
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

// Where a tile's partial states are: from which slot on, and how many.
struct TileSlots {
    int first, count;
};

// Partial softmax states of row tiles, which the merge joins.  A tile is
// `rows` stacked query rows of one (sequence, key head), in the order of
// fa_paged_line.cuh.  Its states are in slots: normalised fp32 outputs, four
// columns of all rows after four columns of all rows (a warp that holds one row
// per lane stores and the merge loads whole lines), and base-2 log-sum-exps.
// Tile i has the slots k + i of the pieces k that have some of its chunks.
// (Along the line, k and i never fall and one of them grows from share to
// share, so no two shares have one slot.)  Where there are more tiles than
// pieces and a tile within one piece leaves no state, `pairs` is 1 and a piece
// has two slots: 2k for the tile that continues in it, 2k + 1 for the one that
// begins in it and ends in another.  (16 sequences of 4096 tokens, 32 heads of
// 128: 20 MB, where a slot for every tile took 1.09 GB.)
struct Partials {
    int slots;
    int pairs;
    float *o;              // [slots][D / 4][slot_rows][4]
    float *lse;            // [slots][slot_rows]
    TileSlots *tile;       // [tiles in all], of tiles with at least one chunk
    int rows;              // stacked query rows per tile
    int slot_rows;         // rows of a slot: rows, or fewer where the only tile has fewer
    int tiles;             // row tiles per (sequence, key head)
    int stacked;           // 1: one list of tiles for all sequences (a shared prefix)
    int chunk;             // keys per chunk of the line
    int fixed_len;         // stacked: keys of the prefix
#ifdef __CUDACC__
    // What a tile's record says of piece `piece`, its first; the slot of its
    // state from a piece (continued: from a chunk past its first on); and the
    // slot of its state number i.
    __device__ __forceinline__ int first_of(int piece, int at_tile) const { return pairs ? 2 * piece : piece + at_tile; }
    __device__ __forceinline__ int slot_of(int piece, int at_tile, bool continued) const
    {
        return pairs ? 2 * piece + (continued ? 0 : 1) : piece + at_tile;
    }
    __device__ __forceinline__ int slot_at(int first, int i) const
    {
        return pairs ? first + 2 * i + (i == 0 ? 1 : 0) : first + i;
    }
#endif
};

// A shared prefix on the tensor cores beside the sequences' own keys in the
// row kernel: the first is bound by its chain of products and softmax, the
// second by memory, so they run at the same time, each on some of the SMs, in
// proportion to their work.  Both kernels work the split out from seq_len.
struct Beside {
    int on;
    int sms, per_sm;                   // pieces of the row kernel per SM
    int blocks;                        // 128-key blocks of the prefix's tiles
    int chunk, tiles;                  // own keys per chunk; tiles per sequence (row tiles * Hkv)
    const int32_t *seq_len;
    int cap, B;                        // most keys of a sequence; sequences
};

// What a tile costs beside its keys, in chunks of the row kernel (256 sequences of
// 1 to 511 keys: 64 -> 57 us) and in blocks of the tensor-core kernel (geometric
// means in us of ten batches behind prefixes, the shapes at kBlockCost, and of six
// batches of 16 to 1024 tokens over 1000 to 16384 keys: 1 block 48.1 and 112, 3
// blocks 47.4 and 82.0, 5 blocks 46.8 and 79.0, 8 blocks 46.8 and 81.3).
constexpr int kRowsTile = 1, kBlocksTile = 5;

// Own chunks and tiles (a chunk has 8 KB of keys and values at D = 64 and 128)
// that cost an SM as much time as one block, with weights of two numbers.
// Geometric means of ten shapes (32 to 256 sequences of 100 to 4000 keys at most,
// prefixes of 1000 to 30000), in us on two GPUs, caches warm, and cold on one: 10:
// 50.8, 49.6 and 61.2; 13: 47.8, 48.1 and 59.5; 14: 47.7, 48.5 and 59.5; 16: 47.3,
// 49.7 and 60.2; 20: 51.8 and 61.7.  (With one number a weight 10 was best: 47.5,
// 46.6 and 58.7.)
constexpr int kBlockCost = 13;

// SMs for the prefix beside `own` chunks and tiles of the sequences' own keys.
#ifdef __CUDACC__
__device__ __forceinline__ int beside_front(const Beside &s, unsigned own)
{
    const float part = (float)s.blocks * kBlockCost;
    const int front = (int)((float)s.sms * part / (part + (float)own) + 0.5f);
    return front < 1 ? 1 : front < s.sms ? front : s.sms - 1;
}
#endif

struct PagedParams {
    PagedCache c;
    const uint16_t *q;
    int64_t q_s[3];                    // batch, head, token
    uint16_t *o;
    int64_t o_s[3];
    float *lse;                        // [B, Hq, T] or null
    int B, T, Hq, G;                   // G = Hq / Hkv query heads share a key head
    FastDiv by_g, by_gt;               // G, G * T
    int causal, f16;
    float scale_log2;
    int second;                        // 1: may start beside the kernel before, and ends after it
    int joined;                        // 1: every tile leaves its state in a slot for the merge
    int two;                           // tensor-core kernel: weights of two 16-bit numbers
    Partials part;
    Beside beside;
    int team;                          // CTAs that share a tile (teams only: 1, 2, 4 or 8)
    const int32_t *prefix_table;       // teams only: keys before the own ones
    int prefix_len;
    int box_rows;                      // key rows per copied box (row kernel: 0 = 16-byte copies)
    uint64_t wait_limit_ns;
};

struct MergeParams {
    Partials src[2];                   // the sequences' own keys, then the prefix
    int n_src;
    const int32_t *seq_len;
    int max_len;
    uint16_t *o;
    int64_t o_s[3];
    float *lse;
    int B, T, Hq, G, D, causal, f16;
    FastDiv by_g, by_r;                // by G, by G T
    int joined;                        // 0: a tile that one CTA finished is written already
};

// Keys per block of the tensor-core kernel.
constexpr int kBlockKeys = 128;

// The row kernel's query rows per tile, keys per chunk, warps (each with a
// piece of the line) per CTA, and CTAs per SM.
int paged_rows_per_tile(int D, int64_t rows);
int paged_rows_chunk(int D);
constexpr int kRowsWarps = 2;
constexpr int kTeamWarps = 8;             // of a CTA that works in a team
constexpr int kMostTeam = 8;              // CTAs of a team (the largest cluster that any GPU takes)
int paged_rows_ctas_per_sm(int D, int rows);

// The current device's number, and its multiprocessors (148 if unknown).
int current_device();
int sm_count_of(int device);

// Raises a kernel's dynamic shared memory limit once per device.
class SharedMemory {
  public:
    template <typename... P>
    cudaError_t allow(void (*kernel)(P...), int bytes)
    {
        const int dev = current_device();
        const bool known = dev >= 0 && dev < 64;
        if (known && (done_.load(std::memory_order_acquire) >> dev) & 1) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && known) done_.fetch_or((uint64_t)1 << dev, std::memory_order_release);
        return e;
    }

  private:
    std::atomic<uint64_t> done_{0};
};

// Launches `kernel` so that its launch may overlap the end of the kernel before
// it on the stream; the kernel itself waits for that one's end (and its
// writes) before it touches memory that one may write.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), int cluster, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args)
{
    return launch_clusters(kernel, 1, grid, threads, smem, stream, args...);
}

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);
// (tk, tv are read only where p.box_rows > 0)
cudaError_t launch_paged_rows(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                              cudaStream_t stream);
cudaError_t launch_paged_team(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                              cudaStream_t stream);
// Teams of `team` CTAs that fit the device together (a cluster does not cross a
// group of SMs, so that fewer than SMs / team do); 0 if it cannot be known.
int paged_teams_at_once(int device, int team);
cudaError_t launch_paged_tc(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                            cudaStream_t stream);
// states: about how many partial states a row has
cudaError_t launch_paged_merge(const MergeParams &p, int states, int sms, cudaStream_t stream);

}  // namespace fa
