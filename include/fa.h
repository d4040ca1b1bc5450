/*
 * fa.h -- C ABI of the exact tiled attention forward pass for GB300 (sm_103a).
 *
 * The library computes, for every batch b and head h,
 *
 *     O   = softmax(scale * Q K^T + mask) V
 *     LSE = log-sum-exp of each row of (scale * Q K^T + mask), natural log
 *
 * block by block with the online-softmax running max m and running sum l,
 * rescaled by exp(m_old - m_new) whenever a key block raises the max, and
 * without ever writing the N x N score matrix to device memory
 * ("vectorized-flash-attention-kernel", Core algorithm and Key design
 * decisions 1-3; "FlashAttention" module F08, Paper).  The mask hides key j
 * from query i when j >= kv_len[b] (key padding), and, if `causal`, when
 * j > i ("kvRow > qRow -> -inf", Core algorithm step 2).
 *
 * Layout (all arguments): Q, K, V and O are contiguous row-major
 * [B, H, N, D] arrays; LSE is a contiguous [B, H, N] float array; kv_len is
 * an int32 array of B entries.  Every pointer is DEVICE memory owned by the
 * caller unless stated otherwise (fa_fwd_from_host takes host arrays); no
 * call allocates device memory or keeps a pointer after it returns.  The
 * library's own state is: device-side status words (see fa_device_status); a
 * cached driver entry point; the fixed scratch array of
 * fa_fwd_splitkv_noalloc (FA_NOALLOC_SCRATCH_BYTES of device memory, held from
 * the time the library's code is loaded on a device); and, per device that
 * calls fa_fwd_from_host, four streams and a set of events, created by the
 * first such call and kept for the life of the process.
 *
 * Calls are asynchronous: they validate their arguments on the host, enqueue
 * one kernel on `stream` (a cudaStream_t; NULL = the legacy default stream)
 * and return.  Results are ready when the stream reaches that point.  Input
 * and output buffers must not overlap.
 *
 * Numerical contract:
 *   - rows whose mask hides every key (kv_len[b] == 0) get O = +0.0 exactly
 *     and LSE = -inf, never NaN ("js-flash-attention-tiled-online-softmax-
 *     exactness", Root causes 2);
 *   - query rows at or past kv_len[b] are still computed over the keys
 *     j < kv_len[b] (padding hides keys, not queries);
 *   - kv_len entries outside [0, N] are clamped to that range on the device;
 *   - input range: the 16-bit paths keep each key block's weights p against a
 *     reference that moves only when a block's sum of p would pass 2^64
 *     (bf16) or 2^15 (fp16), so the fp32 output accumulator holds up to
 *     N * 2^64 * max|V|; O is finite for bf16 |V| < 2^32 (any N < 2^31) and
 *     for every fp16 V.  Q and K may take any finite values.
 */
#ifndef EXACT_TILED_ATTENTION_FA_H
#define EXACT_TILED_ATTENTION_FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, misalignment, overflow */
    FA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (head dim, device)        */
    FA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed                   */
    FA_ERR_TIMEOUT = 4        /* a bounded device-side wait gave up (fa_device_status) */
} fa_status;

/*
 * fa_fwd -- bf16 attention forward on the tensor cores (tcgen05, TMEM, TMA).
 *
 *   Q, K, V  const bf16 [B,H,N,D] device pointers, 16-byte aligned.
 *   O        bf16 [B,H,N,D] device pointer, 16-byte aligned; each element is
 *            the fp32 result rounded to nearest-even.
 *   LSE      float [B,H,N] device pointer, or NULL to skip it (the saved row
 *            statistic a recomputing backward needs: "vectorized-flash-
 *            attention-kernel", Key design decisions 4).
 *   B, H, N  batch, heads, sequence length; any value >= 0.  B*H*N == 0
 *            returns FA_OK without a launch.
 *   D        head dimension: a multiple of 8 from 8 to 128, or 256 (the
 *            pages run D = 16 in "vectorized-flash-attention-kernel",
 *            Evidence & signatures, and d = 32 in "js-flash-attention-tiled-
 *            online-softmax-exactness", Verification).  Other values give
 *            FA_ERR_UNSUPPORTED.  Below 128 the tensor cores run at D
 *            rounded up to 64 or 128 with zero-filled columns, which leave
 *            every score unchanged; only the D real columns of O are
 *            written.
 *   causal   nonzero: key j is hidden from query i when j > i.
 *   scale    softmax scale; NaN or <= 0 selects the default 1/sqrt(D)
 *            ("vectorized-flash-attention-kernel", Constructor options).
 *   kv_len   const int32 [B] device pointer of key lengths, or NULL (= N).
 *   stream   cudaStream_t to enqueue on.
 *
 * Three kernels serve this call.  One gives every CTA two 128-row query
 * tiles (D <= 128).  One gives it one tile (any D here): D = 256, and D <= 64
 * on grids whose one-tile CTAs (2 * B * H * ceil(N/256)) fit in one wave of
 * the GPU's SMs.  The third gives it one tile and splits each row's keys
 * between two softmax warpgroups, whose partial softmax states it merges at
 * the end (D <= 128): 64 < D <= 128 with N >= 8192 or on such small grids.
 * The environment variable FA_FWD_TILES = "1", "2" or "3", read on every
 * call, forces one of them (D = 256 always runs the one-tile kernel).  The
 * kernels agree to rounding, not bit for bit.
 *
 * Accumulation is fp32 (scores, running sums, O); P is rounded to bf16 for
 * the second product, and O is divided by the sum of those rounded weights
 * (the LSE uses the sum of the unrounded ones), so O is a convex combination
 * of V rows whatever the rounding.  Returns FA_ERR_INVALID_ARG / FA_ERR_UNSUPPORTED from
 * host-side checks before anything is enqueued, FA_ERR_CUDA if the launch
 * fails.
 */
fa_status fa_fwd(const void *Q, const void *K, const void *V, void *O, float *LSE,
                 int B, int H, int N, int D, int causal, float scale,
                 const int32_t *kv_len, void *stream);

/*
 * fa_fwd_f16 -- fp16 attention forward on the tensor cores ("FlashAttention"
 * module F08, Exercises: the backward exercise's "fp16" variant of the same
 * tiles).  Same arguments, layout and limits as fa_fwd with IEEE half Q, K,
 * V and O (O rounded to nearest even); LSE stays fp32.  P is rounded to fp16
 * for the second product; the reference max is raised whenever a key
 * block's sum of p would pass 2^15, so P stays inside the fp16 range.
 */
fa_status fa_fwd_f16(const void *Q, const void *K, const void *V, void *O, float *LSE,
                     int B, int H, int N, int D, int causal, float scale,
                     const int32_t *kv_len, void *stream);

/*
 * fa_fwd_fp32 -- fp32 attention forward (fp32 multiply-add on the CUDA cores,
 * no TF32).  Same argument meaning as fa_fwd with float Q, K, V, O; any head
 * dimension 1 <= D <= 256; pointers need only float alignment.
 */
fa_status fa_fwd_fp32(const float *Q, const float *K, const float *V, float *O, float *LSE,
                      int B, int H, int N, int D, int causal, float scale,
                      const int32_t *kv_len, void *stream);

/* The forward kernel fa_fwd and fa_fwd_f16 run for these sizes on the
 * current device: 1 = one 128-row query tile per CTA, 2 = two tiles per CTA,
 * 3 = one tile with each row's keys split between two softmax warpgroups
 * (FA_FWD_TILES, when set, decides as it does for those calls).  0 for a head
 * dimension the tensor-core kernels do not take.  No device work. */
int fa_fwd_kernel_choice(int B, int H, int N, int D);

/*
 * Split-KV forward ("FlashAttention" module F08, Paper and Math: partial
 * softmax states merge associatively).  Same computation and arguments as
 * fa_fwd, for sequences too short to fill the GPU with query tiles: the key
 * blocks of every (batch, head, 256-query-row) item are divided into
 * `num_splits` contiguous ranges processed by separate CTAs.  Each range
 * writes its normalised fp32 partial output and partial LSE to `workspace`,
 * and a second kernel on the same stream merges them:
 *     m = max_s LSE_s,  w_s = exp(LSE_s - m),
 *     O = sum_s w_s O_s / sum_s w_s,  LSE = m + ln sum_s w_s.
 * Ranges that see no key have LSE_s = -inf and weight 0.
 *
 *   num_splits       1..FA_MAX_SPLITS, or 0 for fa_fwd_splitkv_auto_splits().
 *                    With 1 split (given or chosen) the single-pass kernel
 *                    of fa_fwd runs and the workspace is not touched.
 *   workspace        caller-owned device memory, 16-byte aligned, of at least
 *                    fa_fwd_splitkv_workspace_bytes(B,H,N,D,num_splits)
 *                    bytes; its contents on entry do not matter, it is fully
 *                    rewritten, and it must not be used by another call that
 *                    may run at the same time.
 * D is a multiple of 8 up to 128 (256 gives FA_ERR_UNSUPPORTED here).
 * Returns FA_ERR_INVALID_ARG for a missing, misaligned or too small
 * workspace or a split count out of range; otherwise as fa_fwd.
 */
#define FA_MAX_SPLITS 64

fa_status fa_fwd_splitkv(const void *Q, const void *K, const void *V, void *O, float *LSE,
                         int B, int H, int N, int D, int causal, float scale,
                         const int32_t *kv_len, int num_splits, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_fwd_splitkv needs: num_splits * B*H*N * (D + 1) * 4
 * (0 for invalid sizes); num_splits 0 means the automatic choice. */
size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int N, int D, int num_splits);

/* The split count fa_fwd_splitkv uses for num_splits = 0 on the current
 * device.  1 unless D <= 64, N >= 4096 and fa_fwd's grid (2 * B * H *
 * ceil(N/256) one-tile CTAs) leaves SMs idle: there, as many ranges as fill
 * one wave of CTAs (one per SM), at least two key blocks per range, at most
 * FA_MAX_SPLITS.  (Measured on GB300: elsewhere the split path is not faster
 * than fa_fwd.) */
int fa_fwd_splitkv_auto_splits(int B, int H, int N, int D);

/*
 * fa_fwd_splitkv_noalloc -- fa_fwd_splitkv for callers that cannot allocate
 * device memory.  The paper has no counterpart: this is a library service.
 *
 * Some callers cannot call cudaMalloc or any allocator: code inside a
 * framework's allocation-free region, a plugin that is only handed its input
 * and output buffers, or a real-time loop where an allocation could block.
 * This entry point takes no workspace.  It uses a fixed scratch array of
 * FA_NOALLOC_SCRATCH_BYTES bytes that the library keeps in device memory.
 * A device holds that array from the time the library's code is loaded on
 * it (with CUDA's lazy module loading, the first call of this entry point
 * there at the latest) until the process exits.  The call itself allocates
 * nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 *
 * Arguments are those of fa_fwd_splitkv without the workspace.  The caller
 * still passes the inputs and outputs.
 *
 * Limits and behaviour:
 *   - A problem whose fa_fwd_splitkv_workspace_bytes(B,H,N,D,num_splits)
 *     exceeds FA_NOALLOC_SCRATCH_BYTES is rejected with FA_ERR_UNSUPPORTED
 *     before anything is enqueued.  Fewer splits, or fa_fwd, are the
 *     alternatives.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current, and later calls on
 *     that device reuse it.  Make that first call before any stream capture.
 *     The address is kept for the life of the process: after a
 *     cudaDeviceReset of a device this entry point must not be called on it
 *     again, because the array may then sit at another address.
 *   - All calls share the one array, and it keeps the last call's contents.
 *     Each call rewrites every part it reads, so nothing needs clearing.
 *   - Two calls whose kernels overlap on the GPU (different streams, or
 *     different host threads without ordering) race on the array and give
 *     wrong results.  Order them.
 */
#define FA_NOALLOC_SCRATCH_BYTES (32u << 20)

fa_status fa_fwd_splitkv_noalloc(const void *Q, const void *K, const void *V, void *O, float *LSE,
                                 int B, int H, int N, int D, int causal, float scale,
                                 const int32_t *kv_len, int num_splits, void *stream);

/*
 * fa_fwd_from_host -- fa_fwd (or fa_fwd_f16) over inputs and outputs in host
 * memory, with the host<->device copies overlapped with the computation.  The
 * paper has no counterpart: this is a library service for callers whose data
 * starts and ends on the host.
 *
 * The (batch, head) slices are split into `groups` groups, none spanning two
 * batches.  Group c is copied to the device on a library-owned copy stream,
 * computed on one of two library-owned compute streams (alternating, so that
 * consecutive groups' kernels can share the SMs) while group c+1 is copied
 * in, and copied back on a second copy stream.  On a
 * Grace-Blackwell node the copies of a long-context problem take longer than
 * the attention, so the overlap shortens the whole call.
 *
 *   Q_host, K_host, V_host  const [B,H,N,D] host arrays (bf16, or fp16 if f16
 *                           is nonzero).  Page-locked memory lets the copies
 *                           run asynchronously.
 *   O_host                  [B,H,N,D] host array for O.
 *   LSE_host                float [B,H,N] host array, or NULL to skip LSE.
 *   Q_dev, K_dev, V_dev, O_dev  caller-owned device buffers of the same
 *                           shape, 16-byte aligned.  The inputs are copied
 *                           into them, and O is computed there.
 *   LSE_dev                 float [B,H,N] device buffer; required when
 *                           LSE_host is given, else may be NULL.
 *   B,H,N,D, causal, scale, kv_len  as in fa_fwd (kv_len in device memory).
 *   groups                  1..FA_MAX_HOST_GROUPS, or 0 for
 *                           fa_fwd_from_host_auto_groups(B,H,N,D).
 *   stream                  the caller's stream.  The copies start after the
 *                           work already enqueued on it.  Work enqueued on it
 *                           afterwards starts only once O and LSE are back in
 *                           host memory.
 *
 * Returns as fa_fwd; all argument checks run before any CUDA call.  The first
 * call on a device creates that device's four streams and their events.
 * Calls on one device share them.  Calls from several host threads are safe:
 * each enqueues its whole sequence of copies, launches and event records
 * under a per-device lock, so the calls run one after another on the
 * library's streams.  If a CUDA call fails partway, the caller's stream
 * still waits for everything the call had enqueued before the failure, so
 * the buffers may be freed or reused once that stream reaches this point.
 */
#define FA_MAX_HOST_GROUPS 1024

fa_status fa_fwd_from_host(const void *Q_host, const void *K_host, const void *V_host, void *O_host,
                           float *LSE_host, void *Q_dev, void *K_dev, void *V_dev, void *O_dev,
                           float *LSE_dev, int B, int H, int N, int D, int causal, float scale,
                           const int32_t *kv_len, int f16, int groups, void *stream);

/* The group count fa_fwd_from_host uses for groups = 0 on the current
 * device: min(B*H, 8, 256-row work items / SMs), at least 1.  (Groups never
 * span batches, so a call may run more groups than asked for: at least B.) */
int fa_fwd_from_host_auto_groups(int B, int H, int N, int D);

/*
 * fa_bwd -- backward pass of fa_fwd by recomputation ("FlashAttention"
 * module F08, Math: backward via recomputation and the identity
 * rowsum(dP*P) = rowsum(dO*O); "vectorized-flash-attention-kernel", Key
 * design decisions 4: the saved row statistics rebuild P).  Computes the
 * gradients of sum(O * dO) for O = fa_fwd(Q, K, V, ...):
 *
 *     P = exp(scale*Q K^T + mask - LSE),  dV = P^T dO,  dP = dO V^T,
 *     Delta = rowsum(dO * O),  dS = P * (dP - Delta),
 *     dQ = scale * dS K,  dK = scale * dS^T Q.
 *
 *   Q, K, V, O, dO  const bf16 [B,H,N,D]: the forward's inputs and output
 *                   and the upstream gradient; 16-byte aligned.
 *   LSE             const float [B,H,N]: the LSE fa_fwd returned.
 *   dQ, dK, dV      bf16 [B,H,N,D] outputs (fp32 accumulation, rounded to
 *                   nearest even); keys at or past kv_len get zero dK, dV.
 *   B,H,N,D, causal, scale, kv_len: as in the forward call; D a multiple
 *            of 8 up to 128 (zero-padded to 64 / 128 like the forward; 256
 *            gives FA_ERR_UNSUPPORTED).
 *   workspace       caller-owned device memory, 16-byte aligned, of at least
 *                   fa_bwd_workspace_bytes(B,H,N,D) bytes (an fp32 dQ
 *                   accumulator and Delta); fully rewritten by each call;
 *                   calls that may overlap need separate workspaces.
 * dQ is summed across key tiles by fp32 reduce-adds, so its last bits may
 * differ from run to run; dK and dV are deterministic.  Three kernels are
 * enqueued on `stream`.  Errors as fa_fwd, plus FA_ERR_INVALID_ARG for a
 * missing or too small workspace.
 */
fa_status fa_bwd(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                 const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int N, int D,
                 int causal, float scale, const int32_t *kv_len, void *workspace,
                 size_t workspace_bytes, void *stream);

/*
 * fa_bwd_f16 -- fa_bwd for the fp16 forward (fa_fwd_f16): IEEE half Q, K, V,
 * O, dO and dQ, dK, dV; LSE, the workspace and every accumulation stay fp32,
 * and P and dS are rounded to fp16 for the tensor-core products (P <= 1; dS
 * must stay inside the fp16 range, as in any fp16 training).  Same arguments,
 * limits and errors as fa_bwd.
 */
fa_status fa_bwd_f16(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                     const float *LSE, void *dQ, void *dK, void *dV, int B, int H, int N, int D,
                     int causal, float scale, const int32_t *kv_len, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_bwd needs: B*H*N*(D + 1)*4 (0 for invalid sizes). */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int D);

/*
 * ---------------------------------------------------------------- paged cache
 * The operators below serve generation: keys and values of earlier tokens stay
 * in a cache, new tokens are appended, and few queries attend to many keys.
 * The pages this library follows have no counterpart; the row mathematics is
 * fa_fwd's.
 *
 * The cache is a pool of num_pages pages of page_size slots.  Key row (page,
 * head, slot) is D contiguous 16-bit elements at
 *     k + page * stride_page + head * stride_head + slot * stride_slot
 * (elements; multiples of 8), and v likewise, so both [pages, Hkv, slots, D]
 * and [pages, slots, Hkv, D] pools serve.  Key i of sequence b is slot
 * i % page_size of page table[b * table_stride + i / page_size], for i <
 * seq_len[b].  seq_len entries are clamped to [0, table_width * page_size] on
 * the device.  A page number outside [0, num_pages) (-1, say, for a page that
 * was given up) holds nothing: its keys are hidden and appends to it are
 * dropped.  Slots at or past a sequence's length may hold anything; keys and
 * values before it have to be finite.
 *
 * table and seq_len are device memory that the caller updates between calls;
 * a captured graph reads their contents at replay.
 */
typedef struct fa_paged_kv {
    void *k, *v;                 /* 16-byte aligned */
    int64_t stride_page, stride_head, stride_slot;
    int num_pages, page_size;
    int Hkv, D;                  /* key heads; head dimension: a multiple of 8 up to 128, or 256 */
    const int32_t *table;        /* [B, table_width] page numbers, rows table_stride entries apart */
    int64_t table_stride;
    int table_width;             /* table_width * page_size <= 2^31 - 4096 (with a prefix: the sum) */
    const int32_t *seq_len;      /* [B] keys per sequence, the call's own tokens included
                                  * (seq_len and table may be NULL where B is 0) */
} fa_paged_kv;

/* A [B, H, N, D] array of 16-bit elements whose last dimension is contiguous:
 * row (b, h, n) is at ptr + b * stride_b + h * stride_h + n * stride_n
 * (elements; multiples of 8, >= 0).  ptr is 16-byte aligned.  Inputs may
 * repeat rows through strides of 0; outputs may not. */
typedef struct fa_rows {
    void *ptr;
    int64_t stride_b, stride_h, stride_n;
} fa_rows;

/*
 * fa_kv_append -- keys and values of T new tokens per sequence into a paged
 * cache, with the position rotation of keys and queries.
 *
 * seq_len already counts the new tokens: token t of sequence b is its key i =
 * seq_len[b] - T + t, at position n = position_offset + i.  Tokens with i < 0
 * do not exist (a shorter row of a padded batch is aligned at its end): they
 * are not stored, and their query is set to zero.  Tokens that the table has no
 * room for, i >= table_width * page_size, are not stored either (seq_len is not
 * clamped here, so that no earlier key is overwritten); their query is turned.
 *
 * The first rot_dim elements of a head turn in pairs: pair p, of elements p
 * and p + rot_dim / 2 (2p and 2p + 1 if interleaved), by the angle n *
 * inv_freq[p].  The angle is kept modulo one turn in 64-bit fixed point, good
 * to n 2^-64 turns (2^-24 at the farthest position); its sine and cosine and the
 * products are fp32 until they are rounded once.
 *
 *   K, V             [B, Hkv, T, D] new keys and values.
 *   Q, Q_out         [B, Hq, T, D] queries and where to put them rotated, or
 *                    Q = NULL for none.  Q_out may be Q (same address and
 *                    strides) and may not overlap an input otherwise.
 *   inv_freq         float [rot_dim / 2] device array, each in [-65536, 65536]
 *                    (others give NaN).  NULL with rot_dim = 0: no rotation.
 *   rot_dim          even, 0 <= rot_dim <= D.
 *   position_offset  position of a sequence's first key, 0 .. 2^40: behind a
 *                    shared prefix its length, which seq_len does not count.
 *   f16              elements are IEEE half (else bf16).
 *
 * Two tokens of one call that land on the same slot (tables that share a page
 * there) leave it undefined.  One kernel; errors as fa_fwd.
 */
fa_status fa_kv_append(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                       const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim,
                       int interleaved, int64_t position_offset, int f16, void *stream);

/*
 * fa_fwd_paged -- fa_fwd over a paged cache: T query tokens per sequence, Hq
 * query heads that share Hkv key heads (head h uses key head h / (Hq / Hkv)).
 *
 *   Q, O       [B, Hq, T, D].  O may not overlap Q or the cache.
 *   LSE        float [B, Hq, T], contiguous, or NULL.
 *   causal     nonzero: the queries are the last T tokens of their sequence;
 *              query t sees the keys i <= seq_len[b] - T + t.  Queries before
 *              the sequence's first token see none.  Zero: every query sees
 *              all seq_len[b] keys.
 *   scale      as in fa_fwd.
 *   f16        elements are IEEE half (else bf16).
 *   workspace  caller-owned device memory, 16-byte aligned, of at least
 *              fa_fwd_paged_workspace_bytes bytes; its contents on entry do
 *              not matter, and calls that may overlap need separate ones.
 * Queries that see no key get O = +0.0 and LSE = -inf.  Results do not depend
 * on timing: partial states are joined in a fixed order.
 *
 * V is multiplied by 16-bit weights p.  A weight is the sum of two numbers, good
 * to 2^-16 (fp16: 2^-22), so that O's own rounding decides.  Where more than 32
 * query rows of a sequence share a key (T * Hq / Hkv), D <= 128 and page_size is a
 * multiple of 8, it is one number, as in fa_fwd, and O is divided by the sum of the
 * rounded weights: beside its own rounding O is then off by up to 2^-7 (2^-10) of
 * sum p |v| / sum p.  A caller that needs more of such a call passes at most
 * 32 * Hkv / Hq tokens at a time.  A small fp16 weight is off by 2^-32 of its row's
 * largest instead where that is more.
 *
 * Returns as fa_fwd,
 * and FA_ERR_INVALID_ARG for a missing, misaligned or too small workspace, an
 * Hq that is no multiple of Hkv, or sizes past what 32 bits count: tables that
 * allow up to 2^29 chunks of keys in all (16 keys, 32 at D <= 64, 128 where more
 * than 32 rows share keys; per sequence, key head and tile of rows) are taken.
 */
fa_status fa_fwd_paged(const fa_rows *Q, const fa_paged_kv *cache, const fa_rows *O, float *LSE, int B, int Hq, int T,
                       int causal, float scale, int f16, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_fwd_paged needs on the current device (0 for invalid
 * or empty sizes).  They depend on the sizes, not on seq_len's contents. */
size_t fa_fwd_paged_workspace_bytes(const fa_paged_kv *cache, int B, int Hq, int T);

/*
 * fa_fwd_shared_prefix -- fa_fwd_paged for sequences that begin with the same
 * prefix_len keys.  Key i of the prefix is slot i % page_size of page
 * prefix_table[i / page_size] of the same pool; cache->table and seq_len give
 * the keys that follow, each sequence's own.  The prefix's keys are read once
 * for the whole batch, and every query that has a token sees all of them.
 * prefix_len need not be a multiple of page_size.  Results equal fa_fwd_paged
 * on tables that spell the whole sequence, to rounding.
 *
 *   prefix_table  int32 device array of ceil(prefix_len / page_size) pages.
 *   prefix_len    >= 0, a host value (0: fa_fwd_paged).
 * With causal set a query whose own index seq_len[b] - T + t is below 0 has
 * no token and gets O = +0.0 and LSE = -inf.
 */
fa_status fa_fwd_shared_prefix(const fa_rows *Q, const fa_paged_kv *cache, const int32_t *prefix_table, int prefix_len,
                               const fa_rows *O, float *LSE, int B, int Hq, int T, int causal, float scale, int f16,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_fwd_shared_prefix needs (0 for invalid or empty sizes). */
size_t fa_fwd_shared_prefix_workspace_bytes(const fa_paged_kv *cache, int prefix_len, int B, int Hq, int T);

/*
 * Positions that the caller gives, on one or more axes (time, height and width of a
 * video's patches, say): token t of sequence b is at
 *     n[axis * stride_axis + b * stride_b + t * stride_t]
 * on each axis, plus the call's position_offset (any int32; the axes' entries may
 * repeat through strides of 0).  Pair p of a head turns by its position on axis
 * pair_axis[p] (device memory, rot_dim / 2 entries; a pair whose entry is no axis
 * does not turn).  pair_axis = NULL: axis 0.
 */
typedef struct fa_positions {
    const int32_t *n;                           /* (may be NULL where there are no tokens) */
    int64_t stride_axis, stride_b, stride_t;    /* >= 0 */
    int axes;                                   /* >= 1 */
    const int32_t *pair_axis;
} fa_positions;

/* fa_kv_append with the tokens' positions given (NULL: their places in the
 * sequences, as fa_kv_append). */
fa_status fa_kv_append_at(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                          const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim, int interleaved,
                          const fa_positions *positions, int64_t position_offset, int f16, void *stream);

/*
 * fa_rotary -- the position rotation of fa_kv_append on queries and keys without a
 * cache, for training and for attention over whole sequences (fa_fwd).
 *
 *   Q, Q_out         [B, Hq, T, D], and where to put them turned; Q_out may be Q
 *                    (same address and strides) and may not overlap an input
 *                    otherwise.  Not looked at where Hq is 0.
 *   K, K_out         [B, Hkv, T, D], likewise.
 *   D                a multiple of 8 up to 256.
 *   inv_freq, rot_dim, interleaved, position_offset: as in fa_kv_append.
 *   positions        NULL: token t is at position_offset + t.
 *   inverse          nonzero: turned back, which is the gradient of the rotation.
 * One kernel; sines, cosines and products are fp32 until they are rounded once.
 */
fa_status fa_rotary(const fa_rows *Q, const fa_rows *Q_out, const fa_rows *K, const fa_rows *K_out, int B, int Hq, int Hkv,
                    int T, int D, const float *inv_freq, int rot_dim, int interleaved, const fa_positions *positions,
                    int64_t position_offset, int inverse, int f16, void *stream);

/*
 * ------------------------------------------------------------- 4-bit cache
 * A paged cache (above) whose rows are held in 4 bits: at D = 128 a key and its value
 * take 144 bytes a head, where 16 bits take 512.
 *
 * A row of D elements is padded with zeros to P = 64, 128 or 256 (the least that
 * holds it), in groups of 16.  Element d is u * s: u is nibble d of the row's P / 2
 * bytes (an even d is the lower half of byte d / 2), s its group's scale, byte d / 16
 * of the row's P / 16 bytes of scales.
 *   u  sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   s  5 exponent bits, 3 mantissa bits, no sign: the IEEE half with the bits s << 7.
 *      At most 10240 (byte 226); larger bytes are undefined.
 * u * s is exact as an IEEE half and as bf16.  Appending, s is the group's largest
 * magnitude / 6 and u the element / s, both rounded to nearest (halfway to the even
 * mantissa bit), u at most 6: an element is off by at most 0.18 of its group's largest,
 * by 0.2 where that is below 6 * 2^-14, and by 1/3 below 9 * 2^-17.  A group whose
 * largest is 6 * 2^-18 or less is held as zeros, and magnitudes above 61440 are held as
 * that.  Elements have to be finite (others become some finite value).
 *
 * The pools' rows are
 *     k + page * stride_page + head * stride_head + slot * stride_slot
 *     k_scales + page * scale_stride_page + head * scale_stride_head + slot * scale_stride_slot
 * (bytes; multiples of 16, and of P / 16), and v and v_scales likewise.
 */
typedef struct fa_paged_kv4 {
    void *k, *v;                 /* 16-byte aligned */
    int64_t stride_page, stride_head, stride_slot;
    void *k_scales, *v_scales;   /* 16-byte aligned */
    int64_t scale_stride_page, scale_stride_head, scale_stride_slot;
    int num_pages, page_size;
    int Hkv, D;                  /* as in fa_paged_kv, and so are the following */
    const int32_t *table;
    int64_t table_stride;
    int table_width;
    const int32_t *seq_len;
} fa_paged_kv4;

/* fa_kv_append_at into a 4-bit cache.  A key turns in fp32 and is rounded once, to 4
 * bits; the queries are as in fa_kv_append. */
fa_status fa_kv_append_q4(const fa_paged_kv4 *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                          const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim, int interleaved,
                          const fa_positions *positions, int64_t position_offset, int f16, void *stream);

/*
 * fa_fwd_paged_q4 -- fa_fwd_paged over a 4-bit cache: exact attention over the rows
 * that it holds.  Arguments, workspace rules and errors as fa_fwd_paged.
 *
 * A weight is off by 2^-11 relative, for fp16 queries by 2^-22, or by 2^-37 of its
 * row's largest where that is more.  Where more than 32 query rows of a sequence share
 * a key (T * Hq / Hkv), D <= 128 and page_size is a multiple of 8, it is off by 2^-11
 * in either type, or by 2^-32 of the largest, and O is divided by the sum of the
 * rounded weights.  Beyond 512 such rows the keys are decoded once to 16 bits in the
 * workspace, 256 MB of them at a time (or a sequence, if its row of the table takes up
 * to 1 GB; one with more keys is not decoded first), and the errors are fa_fwd_paged's.
 * So a prompt's answer depends, within these errors, on how it is cut into calls.
 *
 * What is saved is memory, and time where few rows share a key: up to 32 rows a call
 * takes less time than over 16 bits (D = 128, 64 sequences of up to 8191 keys, 4, 16 and
 * 32 rows: 71, 99 and 213 us against 163, 174 and 259).  With more rows it takes more (36,
 * 256 and 1024 rows: 259, 513 and 1580 us against 176, 340 and 1262).  Where pages are no
 * multiple of 8 slots, or D is 256, every 8 or 16 rows decode their keys again (1024
 * tokens of 4 rows over 16384 keys, 8 key heads: 1.2 and 4.3 ms, over 16 bits 1.4 and 4.9;
 * with D = 128 and pages of 64 slots 0.22 and 0.20).  Beyond 512 rows sequences are
 * decoded by what their rows of the table can hold, so that a table much wider than the
 * sequences costs workspace and time.
 */
fa_status fa_fwd_paged_q4(const fa_rows *Q, const fa_paged_kv4 *cache, const fa_rows *O, float *LSE, int B, int Hq, int T,
                          int causal, float scale, int f16, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_fwd_paged_q4 needs on the current device (0 for invalid or
 * empty sizes).  They depend on the sizes, not on seq_len's contents. */
size_t fa_fwd_paged_q4_workspace_bytes(const fa_paged_kv4 *cache, int B, int Hq, int T);

/*
 * fa_kv_read -- the keys and values of the last T tokens of every sequence as rows
 * K, V [B, Hkv, T, D], aligned at their end like an append's tokens.  Tokens that a
 * sequence does not have, or whose page holds nothing, are zero.  fa_kv_read_q4: of a
 * 4-bit cache, decoded (exactly) to IEEE halves (f16) or bf16.  One kernel.
 */
fa_status fa_kv_read(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, int B, int T, void *stream);
fa_status fa_kv_read_q4(const fa_paged_kv4 *cache, const fa_rows *K, const fa_rows *V, int B, int T, int f16, void *stream);

/*
 * ------------------------------------------------------------- pages
 * Which pages sequences have, kept on the device: no call waits for the GPU, and all
 * can be captured into a graph.
 *
 * refs[p] counts the uses of page p: one for each table entry in front of a
 * sequence's length (entry e of row b with e < ceil(seq_len[b] / page_size)), and what
 * the caller adds for uses of its own, a shared prefix say.  A page whose count is 0
 * (or less) is free.  Calls that take pages take the lowest free ones, in order, so
 * that results depend on nothing but the inputs.  Layers with caches of their own
 * share one table: its calls are made once, and the copies that they list are made in
 * every cache with fa_copy_pages.
 */
typedef struct fa_page_table {
    int32_t *table;              /* [B, table_width], rows table_stride entries apart */
    int64_t table_stride;
    int table_width;             /* table_width * page_size <= 2^31 - 4096 */
    int B;
    int32_t *seq_len;            /* [B] */
    int32_t *refs;               /* [num_pages] */
    int num_pages, page_size;    /* num_pages, and the entries of the calls' vectors, <= 2^31 - 1025 */
} fa_page_table;

/* Bytes of workspace (16-byte aligned; its contents do not matter, and calls that may
 * overlap need separate ones) that the calls below need, for n forks. */
size_t fa_pages_workspace_bytes(const fa_page_table *table, int n);

/*
 * fa_kv_grow -- every sequence b grows by tokens[b] (0 or less: not), and gets the
 * pages for them: what an append needs.  taken[b] is how many pages it got, or -2 if
 * it was not grown: the table's row is too short (it asks for no pages then), or it
 * needs pages and the free ones do not suffice for what it and all sequences in front of
 * it ask for.  Pages are given in the order of the sequences.
 */
fa_status fa_kv_grow(const fa_page_table *table, const int32_t *tokens, int32_t *taken, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * fa_kv_free -- rows [n] give up their pages: counts fall by one, the rows' entries
 * become -1 and their lengths 0.  A row that is listed twice, or is none, counts once,
 * or not at all.
 */
fa_status fa_kv_free(const fa_page_table *table, const int32_t *rows, int n, void *stream);

/*
 * fa_kv_fork -- row child[i] becomes what row parent[i] is, for i < n.  Full pages are
 * shared; a last page that is part full is copied to a free one, since both rows will
 * write behind it.  src[i] and dst[i] are that copy, which the caller makes with
 * fa_copy_pages, or -1 for none.  dst[i] = -2: not forked, because no page was free,
 * the child was not empty (seq_len 0), a row is none, the child is an earlier fork's
 * child, or the parent is a fork's child in the same call (whether that one is done or
 * not).
 */
fa_status fa_kv_fork(const fa_page_table *table, const int32_t *parent, const int32_t *child, int n, int32_t *src, int32_t *dst,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * fa_kv_compact -- with L pages in use, those from page L on move to the free ones in
 * front of it, both in order, so that the pool's end is free.  moved[p] is page p's new
 * number (-1 if it is free); counts and the sequences' entries follow, other tables are
 * the caller's to map.  *count copies from src[] to dst[] (num_pages entries each) are
 * the caller's to make with fa_copy_pages.
 */
fa_status fa_kv_compact(const fa_page_table *table, int32_t *moved, int32_t *src, int32_t *dst, int32_t *count, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * fa_copy_pages -- page src[i] of a cache's pools to page dst[i], keys and values of
 * all heads and slots, for i < n (or *count, device memory, where that is less; NULL:
 * n).  Pairs with a number outside the pool are skipped.  No page may be the target of
 * two pairs or of one and the source of another: its contents would be undefined.
 */
fa_status fa_copy_pages(const fa_paged_kv *cache, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream);
fa_status fa_copy_pages_q4(const fa_paged_kv4 *cache, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream);

/* Human-readable name of a status code (static string, never NULL). */
const char *fa_status_string(fa_status s);

/*
 * fa_device_status -- synchronise `stream`, then report and clear the
 * device-side status word.  Returns FA_ERR_TIMEOUT if a kernel of this
 * library gave up a bounded wait since the last call (its output is then
 * undefined), FA_ERR_CUDA if synchronising failed, FA_OK otherwise.
 *
 * Every wait of the tensor-core kernels on another part of the same CTA
 * gives up after a budget: 4 s by default, or the environment variable
 * FA_WAIT_LIMIT_MS (milliseconds, fractions allowed), read once per process.
 * A kernel that gives up still waits, with a budget of at least 1 s, for the
 * copies and MMAs it has in flight before it exits, so the CUDA context stays
 * usable.
 */
fa_status fa_device_status(void *stream);

/*
 * fa_last_error_detail -- the site code of the last device-side give-up that
 * fa_device_status saw (0 if none): a diagnostic for bug reports.
 */
uint32_t fa_last_error_detail(void);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_TILED_ATTENTION_FA_H */
