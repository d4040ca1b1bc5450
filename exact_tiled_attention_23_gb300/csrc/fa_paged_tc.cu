// fa_paged_tc.cu -- attention of many stacked query rows over a paged cache, on
// the tensor cores.
//
// Serves the row tiles that the row kernel (fa_paged_rows.cu) would have to cut
// into many: the rows of a whole batch over a shared prefix, and pieces of a
// prompt.  A tile is 128 stacked query rows of one (sequence, key head); the
// line of 128-key blocks of all tiles is cut into one equal piece per CTA
// (fa_paged_line.cuh), one CTA per SM, and a tile that two or more CTAs had a
// share of is joined by the merge.
//
// Within a block the work is laid out as in the split-row forward kernel
// (fa_fwd_halves.cu): each row's 128 keys are split into halves of 64 with
// separate online-softmax states, warps 4-7 and 8-11, and one thread each issues
// S = Q K^T (warp 3) and O_h += P_h V_h (warp 1).  What is different:
//
//   * the roles run along the CTA's whole piece of the line without stopping
//     at a tile's end: the rings, the score tile and the P tiles go on counting,
//     the softmax warps fetch the next tile's Q once the last scores are done,
//     and only O is handed over (o_final, o_read);
//   * K and V come through the page table: the lanes of warps 0 (K) and 2 (V)
//     each find one box of a block (as many rows as divide a page, 8 to 128).  A box
//     past the tile's last key, or of a page outside the pool, is read past the
//     tensor's end, which fills it with zeros;
//   * a box that the sequence ends in brings whatever the page holds behind the
//     last key, and 0 * NaN is NaN: warp 1 clears those rows of V before its
//     products read them;
//   * keys of pages outside the pool are hidden: a scan of the CTA's pages, done
//     while the first copies fly, decides whether the blocks have to ask.
//
// Measured: 1024 tokens over 16384 keys, 32 query and 8 key heads, D = 128, bf16,
// 2.7e11 operations, 200 us with the merge, 1.33 PFLOP/s (a large matrix product:
// 1.88); ~1680 clk per block, as in the split-row kernel, bound by the softmax and
// the hand-offs around it (tensor pipe 52 % busy).  Short calls pay ~10 us until
// the pipeline runs, most of it instruction fetch.
//
// The tensor cores take 16-bit weights.  For the rows of a generation step over
// a shared prefix a weight is the sum of two numbers, p = hi + lo, with a product
// each, as in the row kernel that reads the sequences' own keys: the answer of a
// sequence is as exact alone as among many (kTwo).  hi and lo take the two P tiles,
// so that a block's weights wait for the products of the block before.  Beside the
// own keys that costs 1 to 3 % (kBlockCost in fa_paged.h).  Pieces of a prompt would
// go from 199 to 271 us: there P is rounded once and O divided by the sum of the
// rounded weights, as in fa_fwd.
//
// Every mbarrier wait is bounded; a wait that runs out records the site in
// this file's status word, raises the CTA's abort flag, and every role drains
// its copies / MMAs, frees TMEM and exits.
#include "fa_fwd_softmax.cuh"
#include "fa_internal.h"
#include "fa_paged.h"
#include "fa_paged_line.cuh"
#include "fa_tc_common.cuh"
#include "sm103_ptx.cuh"

#include <cmath>

namespace fa {

__device__ uint32_t g_status_paged;

namespace {

constexpr int BM = 128;                   // query rows per tile (= TMEM lanes)
constexpr int BN = kBlockKeys;            // keys per block
constexpr int kHalf = 64;                 // keys of a block per softmax warpgroup
constexpr int kThreads = 384;             // warp 0 K copies, 1 PV, 2 V copies, 3 S, 4-11 softmax
constexpr int kSoftmaxWarp0 = 4;
constexpr int kChunkBytes = 128 * 128;    // 128 rows x 64 columns of 16 bits
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // S [0,128)
constexpr uint32_t kColP = 128;           // P tiles [128,192), [192,256)
constexpr uint32_t kColO = 256;           // O_A and O_B, D columns each
constexpr float kLn2 = 0.69314718055994530942f;
// fp16 weights are multiples of 2^-24.  Against a reference 2^7 below the largest
// score a weight is off by 2^-32 of the row's largest (against the largest itself,
// by 2^-25: 8192 keys with 0.5 % of the weight came out 1.3 % off), and 64 weights
// as large as that still stay below the limit of a block's sum.
constexpr int kLiftF16 = 7;

template <int D>
struct TcLayout {
    static constexpr int kChunks = D / 64;                      // 128-byte swizzle atoms per row
    static constexpr int kTileBytes = kChunks * kChunkBytes;    // a Q, K or V tile
    // K slots and V slots: a tile takes ~1500 clk to arrive, and V's products
    // follow the softmax, so V is requested further ahead.
    static constexpr int kRingK = D == 128 ? 3 : 4, kRingV = D == 128 ? 3 : 4;
    static constexpr int kQOff = 0;
    static constexpr int kKOff = kTileBytes;
    static constexpr int kVOff = kKOff + kRingK * kTileBytes;
    static constexpr int kBarOff = kVOff + kRingV * kTileBytes;
    // q_full, k_full/k_empty[RK], v_full/v_empty[RV], s_full, s_read,
    // p_full[2][2], pv_done[2][2], o_final, o_read, mma_drain, mma_drain_s
    static constexpr int kBars = 1 + 2 * (kRingK + kRingV) + 2 + 4 + 4 + 4;
    static constexpr int kSmemBytes = kBarOff + 512 + 1024;    // + alignment slack
    __device__ static constexpr uint32_t col_o(int h) { return kColO + (uint32_t)(h * D); }
    __device__ static constexpr uint32_t col_p(int buf, int h) { return kColP + (uint32_t)(buf * 64 + h * 32); }
    static_assert(D == 64 || D == 128, "head dim");
    static_assert(kColO + 2 * D <= kTmemCols, "TMEM columns");
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    static_assert(kBars * 8 + 16 <= 512, "barrier area");
};

// wait_bounded with everything past its first test out of line.  The loops below
// are bound by the fetch of their instructions; with the tests of the clock at
// every wait inside them, pieces of a prompt ran 6 % slower.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, uint64_t limit_ns, uint32_t site, Abort ab,
                                       bool follow_abort)
{
    return wait_bounded(bar, parity, limit_ns, site, ab, follow_abort);
}

__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, uint64_t limit_ns, uint32_t site, Abort ab,
                                         bool follow_abort = true)
{
    return ptx::mbar_test(bar, parity) || wait_long(bar, parity, limit_ns, site, ab, follow_abort);
}

using BlockLine = Line<BN, kBlocksTile>;

// OnlineRow::exp_pass for weights of two numbers: hi to the columns at t_hi, lo to
// those at t_lo.  The sum of p serves O and the LSE.
template <bool kF16, typename PreStore>
__device__ __forceinline__ void exp_two(const uint32_t (&s)[2][32], float sl2, float m_ref, uint32_t t_hi, uint32_t t_lo,
                                        float &sum, PreStore &pre_store)
{
    const float ref = m_ref == -INFINITY ? 0.f : m_ref;
    const uint64_t scale = ptx::pack2(sl2, sl2), less = ptx::pack2(-ref, -ref), minus = ptx::pack2(-1.f, -1.f);
    uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float y0, y1, r0, r1;
            ptx::unpack2(ptx::fma2(ptx::pack2(u2f(s[c][2 * t]), u2f(s[c][2 * t + 1])), scale, less), y0, y1);
            const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
            const uint64_t both = ptx::pack2(p0, p1);
            acc[t & 3] = ptx::add2(acc[t & 3], both);
            hi[t] = ptx::pack16x2<kF16>(p0, p1);
            ptx::unpack2(ptx::fma2(ptx::widen16x2<kF16>(hi[t]), minus, both), r0, r1);
            lo[t] = ptx::pack16x2<kF16>(r0, r1);
        }
        if (c == 0) pre_store();
        ptx::tmem_st16(t_hi + c * 16, hi);
        ptx::tmem_st16(t_lo + c * 16, lo);
    }
    sum = 0.f;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        float x, y;
        ptx::unpack2(acc[a], x, y);
        sum += x + y;
    }
}

// A role's way along the CTA's piece of the line, tile by tile: what a block
// needs beyond its number is found once per tile, because the issuing threads
// run alone and every instruction between two products counts (a walk that
// asked at every block, with a division, made the kernel 1.7 times slower).
struct Walk {
    LineCursor u;
    int left;          // blocks from here to the end of the piece
    // blocks of this tile in the piece
    __device__ __forceinline__ int count() const { return min(u.n - u.c, left); }
    // past `done` = count() blocks; false at the end of the piece
    __device__ __forceinline__ bool next_tile(const BlockLine &line, int done)
    {
        left -= done;
        if (left == 0) return false;
        u.c += done - 1;
        line.advance(u);
        return true;
    }
};

template <int D, bool kF16, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedParams p)
{
    using Lay = TcLayout<D>;
    constexpr int kChunks = Lay::kChunks, kTileBytes = Lay::kTileBytes, RK = Lay::kRingK, RV = Lay::kRingV;
    constexpr int kQOff = Lay::kQOff, kKOff = Lay::kKOff, kVOff = Lay::kVOff;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff);
    uint64_t *q_full = bars + 0;               // a tile's rows are in place (8 arrivals)
    uint64_t *k_full = bars + 1;               // [RK]
    uint64_t *k_empty = k_full + RK;           // [RK]
    uint64_t *v_full = k_empty + RK;           // [RV]
    uint64_t *v_empty = v_full + RV;           // [RV]
    uint64_t *s_full = v_empty + RV;           // S of a block complete
    uint64_t *s_read = s_full + 1;             // all softmax warps hold it in registers (8 arrivals)
    uint64_t *p_full = s_read + 1;             // [half][P tile]: P_h stored (4 arrivals)
    uint64_t *pv_done = p_full + 4;            // [half][P tile]: O_h += P_h V done
    uint64_t *o_final = pv_done + 4;           // every product of a tile complete
    uint64_t *o_read = o_final + 1;            // the softmax warps hold O (8 arrivals)
    uint64_t *mma_drain = o_read + 1;
    uint64_t *mma_drain_s = mma_drain + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Lay::kBars);
    int *abort_word = reinterpret_cast<int *>(tmem_slot + 1);
    int *hidden_word = abort_word + 1;
    const Abort ab{abort_word, &g_status_paged};
    const uint64_t limit = p.wait_limit_ns;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    // Set-up that reads no memory overlaps the end of the kernel before.
    if (threadIdx.x == 0) {
        for (int i = 0; i < Lay::kBars; ++i) {
            uint32_t count = 1;
            if (&bars[i] == q_full || &bars[i] == s_read || &bars[i] == o_read) count = 8;   // one per softmax warp
            if (&bars[i] >= p_full && &bars[i] < p_full + 4) count = 4;           // the four warps of a half
            ptx::mbar_init(&bars[i], count);
        }
        *abort_word = 0;
        *hidden_word = 0;
        ptx::fence_mbarrier_init();
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
    }
    if (!p.second) ptx::wait_for_primary();
    ptx::launch_dependents();
    BlockLine line(p);
    Walk walk;
    int used, units, per;                      // units of the piece: before `walk`, from there on; a full piece's
    line.share((int)blockIdx.x, (int)gridDim.x, walk.u, used, units, per);
    walk.left = 0;
    {
        LineCursor u = walk.u;
        for (int rest = units; rest > 0;) {
            const int n = min(u.n - u.c, line.chunks_within(u.c, rest));
            walk.left += n;
            rest -= line.start_of(u.c + n) - line.start_of(u.c);
            u.c += n - 1;
            line.advance(u);
            if (u.n == 0) break;
        }
    }
    if (walk.left == 0) {
        if (p.second) ptx::wait_for_primary();
        return;
    }
    const int blocks = walk.left;
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0 || warp == 2) {
        // ================= K copies (warp 0), V copies (warp 2) =================
        // Lane i < boxes finds box i of a block; lane 0 copies them all.  One
        // warp each: a copy costs its issuing thread ~100 clk, and with pages
        // of 16 keys a block takes 32.
        const int box = p.box_rows, boxes = BN / box;
        const CUtensorMap *tm = warp == 0 ? &tm_k : &tm_v;
        uint64_t *full = warp == 0 ? k_full : v_full, *empty = warp == 0 ? k_empty : v_empty;
        const uint32_t slots = ptx::smem_u32(smem + (warp == 0 ? kKOff : kVOff));
        const int ring = warp == 0 ? RK : RV;
        int issued = 0, slot = 0;
        uint32_t phase = 1;                                     // of the slot's last release
        for (int t = 0; t < blocks; ++t) {
            int page = p.c.num_pages, at = 0;                   // past the tensor's end: zeros
            const int64_t key = (int64_t)walk.u.c * BN + lane * box;
            if (lane < boxes && key < walk.u.keys) {
                const int which = p.c.by_page.quotient((int)key);
                const int x = p.c.table[(int64_t)(walk.u.g / p.part.tiles) * p.c.table_stride + which];
                if (x >= 0 && x < p.c.num_pages) page = x;
                at = (int)key - which * p.c.page_size;
            }
            const int h = walk.u.h;
            if (t + 1 < blocks) line.advance(walk.u);
            bool ok = true;
            if (t >= ring && lane == 0) ok = wait_for(&empty[slot], phase, limit, kSiteSlotEmpty, ab);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot], kTileBytes);
#pragma unroll 2
            for (int i = 0; i < boxes; ++i) {
                const int box_page = __shfl_sync(0xffffffffu, page, i), box_at = __shfl_sync(0xffffffffu, at, i);
                if (lane == 0)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        ptx::tma_load_4d(slots + slot * kTileBytes + c * kChunkBytes + i * box * 128, tm, &full[slot], c * 64,
                                         box_at, h, box_page);
            }
            issued = t + 1;
            if (++slot == ring) {
                slot = 0;
                phase ^= 1;
            }
        }
        // Drain: no copy may still be landing in shared memory at exit.
        if (lane == 0)
            for (int t = issued > ring ? issued - ring : 0; t < issued; ++t)
                wait_for(&full[t % ring], (t / ring) & 1, limit, kSiteDrain, ab, false);
        __syncwarp();
    } else if (warp == 3) {
        // ================= S products =================
        // S of block t into the score tile, once the softmax warps hold block
        // t-1's in registers.
        if (lane == 0) {
            constexpr uint32_t idesc = make_idesc(BM, BN, 0, 0, kF16);
            const uint64_t q_desc = make_sdesc(ptx::smem_u32(smem + kQOff), 16, 1024);
            const uint64_t k_desc = make_sdesc(ptx::smem_u32(smem + kKOff), 16, 1024);
            constexpr uint64_t kTileStep = kTileBytes >> 4;
            int t = 0;
            bool ok = true;
            for (int tile = 0;; ++tile) {
                const int count = walk.count(), end = t + count;
                ok = wait_for(q_full, tile & 1, limit, kSiteQFull, ab);
#pragma unroll 1
                for (; ok && t < end; ++t) {
                    ok = wait_for(&k_full[t % RK], (t / RK) & 1, limit, kSiteSlotFull, ab);
                    if (ok && t > 0) ok = wait_for(s_read, (t - 1) & 1, limit, kSiteSFull, ab);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint64_t kd = k_desc + (uint64_t)(t % RK) * kTileStep;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t off = (uint64_t)(((k / 4) * kChunkBytes + (k % 4) * 32) >> 4);
                        ptx::mma_ss(tmem + kColS, q_desc + off, kd + off, idesc, k > 0);
                    }
                    ptx::mma_commit(s_full);
                    ptx::mma_commit(&k_empty[t % RK]);
                }
                if (!ok) break;
                if (!walk.next_tile(line, count)) break;
            }
            ptx::mma_commit(mma_drain_s);
            wait_for(mma_drain_s, 0, limit, kSiteDrain, ab, false);
        }
    } else if (warp == 1) {
        // ================= PV products =================
        // O_h += P_h V[64h ..]: K-steps 4h .. 4h+3 of the block, A from the
        // half's 32 columns of P tile t % 2 (kTwo: of both tiles, hi and lo of
        // one block).  A tile's first products replace O,
        // once the softmax warps hold the tile before.  Lane 0 waits and
        // issues; the warp clears V behind a sequence's end together.
        constexpr uint32_t idesc = make_idesc(BM, D, 0, 1, kF16);
        const uint64_t v_desc = make_sdesc(ptx::smem_u32(smem + kVOff), kChunkBytes, 1024);
        constexpr uint64_t kTileStep = kTileBytes >> 4;
        auto issue = [&](int t, bool first, bool v_ready) -> bool {
            const int buf = t & 1;
            if (!v_ready && !wait_for(&v_full[t % RV], (t / RV) & 1, limit, kSiteSlotFull, ab)) return false;
            const uint64_t vd = v_desc + (uint64_t)(t % RV) * kTileStep;
            for (int h = 0; h < 2; ++h) {
                if (!wait_for(&p_full[h * 2 + buf], (t >> 1) & 1, limit, kSitePFull, ab)) return false;
                ptx::tc_fence_after();
                const uint32_t to = tmem + Lay::col_o(h);
#pragma unroll
                for (int n = 0; n < (kTwo ? 2 : 1); ++n) {
                    const uint32_t tp = tmem + Lay::col_p(kTwo ? n : buf, h);
#pragma unroll
                    for (int k = 0; k < kHalf / 16; ++k)
                        ptx::mma_ts(to, tp + k * 8, vd + (uint64_t)(((4 * h + k) * 2048) >> 4), idesc,
                                    (!first || k > 0 || n > 0) ? 1u : 0u);
                }
                ptx::mma_commit(&pv_done[h * 2 + buf]);
            }
            ptx::mma_commit(&v_empty[t % RV]);
            return true;
        };
        int t = 0;
        for (int tile = 0;; ++tile) {
            const int count = walk.count(), end = t + count;
            // Rows of the last block's V that hold what lies behind the
            // sequence's last key: from there to the end of the box it is in.
            const int from = walk.u.len - (walk.u.c + count - 1) * BN;
            const bool rest = from < BN && (from & (p.box_rows - 1)) != 0;      // (a box has a power of two rows)
            const int to = rest ? (from | (p.box_rows - 1)) + 1 : from;
            bool ok = true;
            if (lane == 0) {
                if (tile > 0) ok = wait_for(o_read, (tile - 1) & 1, limit, kSiteOFinal, ab);
                const int t0 = t;
#pragma unroll 1
                for (; ok && t < end - (rest ? 1 : 0); ++t) ok = issue(t, t == t0, false);
                if (rest) ok = ok && wait_for(&v_full[t % RV], (t / RV) & 1, limit, kSiteSlotFull, ab);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (rest) {
                t = end - 1;
                const uint32_t v = ptx::smem_u32(smem + kVOff + (t % RV) * kTileBytes);
                for (int e = lane; e < (to - from) * kChunks * 8; e += 32) {
                    const int row = from + e / (kChunks * 8), unit = e % (kChunks * 8);
                    ptx::st_shared_v4(v + (unit / 8) * kChunkBytes + row * 128 + ((unit % 8) << 4), 0u, 0u, 0u, 0u);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ok = issue(t, count == 1, true);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
            }
            t = end;
            if (lane == 0) ptx::mma_commit(o_final);
            if (!walk.next_tile(line, count)) break;
        }
        if (lane == 0) {
            ptx::mma_commit(mma_drain);
            wait_for(mma_drain, 0, limit, kSiteDrain, ab, false);
        }
        __syncwarp();
    } else {
        // ================= online softmax of one key half + epilogue =================
        const int h = (warp - kSoftmaxWarp0) / 4;     // key half: columns 64h .. 64h+63 of every block
        const int quarter = warp & 3;                 // TMEM lanes 32*quarter ..
        const int r_local = quarter * 32 + lane;
        const int thread = threadIdx.x - 32 * kSoftmaxWarp0;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + kColS + (uint32_t)(h * kHalf);
        const float sl2 = p.scale_log2;

        // The rows of the walk's tile into the Q buffer, in the 128-byte-swizzled
        // layout; rows past the last and columns past D are zero.  The products
        // that read the buffer before are done.
        auto copy_q = [&] {
            // two threads per row, so that a row's place is found once
            const int b = walk.u.g / p.part.tiles, row = thread >> 1, idx = (walk.u.g - b * p.part.tiles) * BM + row;
            constexpr int kUnits = D / 16;                        // 16-byte units per thread
            const int unit0 = (thread & 1) * kUnits;
            uint4 w[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (idx < line.R) {
                const RowPlace r = row_place(p, b, walk.u.h, idx);
                const uint16_t *src = p.q + r.b * p.q_s[0] + r.hq * p.q_s[1] + r.t * p.q_s[2];
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    if ((unit0 + i) * 8 < p.c.D) w[i] = *reinterpret_cast<const uint4 *>(src + (unit0 + i) * 8);
            }
            const uint32_t dst = ptx::smem_u32(smem + kQOff) + row * 128;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int unit = unit0 + i;
                ptx::st_shared_v4(dst + (unit / 8) * kChunkBytes + (((unit % 8) ^ (row & 7)) << 4), w[i].x, w[i].y, w[i].z, w[i].w);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full);
        };

        // the first tile's Q, and whether any page of this piece is hidden
        copy_q();
        bool hidden = false;
        {
            Walk s = walk;
            int count;
            do {
                count = s.count();
                const int from = p.c.by_page.quotient(s.u.c * BN);
                const int last = p.c.by_page.quotient((int)min((int64_t)s.u.keys, (int64_t)(s.u.c + count) * BN) - 1);
                const int32_t *table = p.c.table + (int64_t)(s.u.g / p.part.tiles) * p.c.table_stride;
                for (int i = from + thread; i <= last; i += 256) {
                    const int page = table[i];
                    hidden = hidden || page < 0 || page >= p.c.num_pages;
                }
            } while (s.next_tile(line, count));
        }
        if (hidden) *hidden_word = 1;
        ptx::bar_sync(1, 256);
        hidden = *hidden_word != 0;

        int t = 0;
        bool ok = true;
        for (int tile = 0;; ++tile) {
            const int count = walk.count();
            const int b = walk.u.g / p.part.tiles, row0 = (walk.u.g - b * p.part.tiles) * BM;
            const int row = row0 + r_local;
            const int lim = min(walk.u.len, line.masked ? walk.u.len - p.T + p.by_g.quotient(row) + 1 : walk.u.len);
            // Blocks from t_mask on have keys that some row of the tile does
            // not see; a tile's first row sees the fewest.
            const int least = min(walk.u.len, line.masked ? walk.u.len - p.T + p.by_g.quotient(row0) + 1 : walk.u.len);
            const int t_mask = t + max(0, least) / BN - walk.u.c;
            OnlineRow<D, kF16, kHalf, kF16 ? kLiftF16 : 0> st;
            for (int j = 0; j < count; ++j, ++t) {
                const int buf = t & 1;
                const uint32_t tP = tmem + lane_off + Lay::col_p(kTwo ? 0 : buf, h);
                const int reader = t - (kTwo ? 1 : 2);            // the last block whose products read it
                const uint32_t tO = tmem + lane_off + Lay::col_o(h);
                const bool got = wait_for(s_full, t & 1, limit, kSiteSFull, ab);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                // whether that reader is done: tested now, waited for below only
                // if it was not
                const bool p_free = reader < 0 || ptx::mbar_test(&pv_done[h * 2 + (reader & 1)], (reader >> 1) & 1);
                ptx::tc_fence_after();
                // Hidden keys become -inf in TMEM, eight at a time and only in
                // blocks that have some: selects on the 64 registers of the row
                // would lie in the middle of the loop, whose instruction
                // fetches cost more than this detour.
                if (t >= t_mask || hidden) {
                    const int key0 = (walk.u.c + j) * BN + h * kHalf;
#pragma unroll 1
                    for (int k = 0; k < kHalf; k += 8) {
                        bool gone = false;                        // (a page holds a multiple of 8 keys)
                        if (hidden && key0 + k < walk.u.keys) {
                            const int page = p.c.table[(int64_t)b * p.c.table_stride + p.c.by_page.quotient(key0 + k)];
                            gone = page < 0 || page >= p.c.num_pages;
                        }
                        const int vis = gone ? 0 : lim - (key0 + k);         // columns i < vis are visible
                        if (!__any_sync(0xffffffffu, vis < 8)) continue;
                        uint32_t x[8];
                        ptx::tmem_ld8(tS + k, x);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i >= vis) x[i] = f2u(-INFINITY);
                        ptx::tmem_st8(tS + k, x);
                    }
                    ptx::tmem_wait_st();
                }
                uint32_t s_raw[2][32];
                ptx::tmem_ld32(tS, s_raw[0]);
                ptx::tmem_ld32(tS + 32, s_raw[1]);
                ptx::tmem_wait_ld();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(s_read);

                bool hook_ok = true;
                auto before_o = [&] {
                    if (j > 0) {
                        hook_ok = wait_for(&pv_done[h * 2 + ((t - 1) & 1)], ((t - 1) >> 1) & 1, limit, kSiteOFinal, ab) &&
                                  hook_ok;
                        ptx::tc_fence_after();
                    }
                };
                auto before_p = [&] {
                    if (!__all_sync(0xffffffffu, p_free)) {
                        hook_ok = wait_for(&pv_done[h * 2 + (reader & 1)], (reader >> 1) & 1, limit, kSiteOFinal, ab) && hook_ok;
                        ptx::tc_fence_after();
                    }
                };
                // OnlineRow::block as a loop of at most two turns: one copy of its code
                float sum, sum_o;
                bool raise = __any_sync(0xffffffffu, st.m_ref == -INFINITY);
#pragma unroll 1
                for (int turn = 0; turn < 2; ++turn) {
                    if (raise) st.raise(s_raw, sl2, j > 0, tO, before_o);
                    if constexpr (kTwo) {
                        exp_two<kF16>(s_raw, sl2, st.m_ref, tP, tmem + lane_off + Lay::col_p(1, h), sum, before_p);
                        sum_o = sum;
                    } else {
                        st.template exp_pass<1>(s_raw, sl2, tP, sum, sum_o, before_p);
                    }
                    raise = __any_sync(0xffffffffu, !(sum <= (kF16 ? kLazyLimitF16 : kLazyLimit)));
                    ptx::tmem_wait_st();      // the first turn's P stores land before new ones
                    if (!raise) break;
                }
                st.l += sum;
                st.l_o += sum_o;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&p_full[h * 2 + buf]);
                if (!__all_sync(0xffffffffu, hook_ok)) {
                    ok = false;
                    break;
                }
            }

            // The scores of the tile are done: the next tile's Q, while the last
            // products run.
            const LineCursor was = walk.u;
            const bool more = walk.next_tile(line, count);
            if (ok && more) copy_q();

            // ---- join the halves: m = max(m_A, m_B), w_h = 2^(m_h - m),
            // O = (w_A O_A + w_B O_B) / (w_A l_oA + w_B l_oB)
            bool have = ok;
            if (have) have = wait_for(o_final, tile & 1, limit, kSiteOFinal, ab);
            // all eight warps agree, so that the named barriers are reached by
            // all of them or by none; the last tile's exchange is read, too
            have = ptx::bar_and(1, 256, have);
            if (!have) break;
            ptx::tc_fence_after();
            // (m, l, l_o) of the other half through the first columns of P tile
            // 0, which no product reads before these warps store the next P.
            uint32_t mine[4] = {f2u(st.m_ref), f2u(st.l), f2u(st.l_o), 0u}, its[4];
            ptx::tmem_st4(tmem + lane_off + kColP + (uint32_t)(h * 4), mine);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::bar_sync(2, 256);
            ptx::tc_fence_after();
            ptx::tmem_ld4(tmem + lane_off + kColP + (uint32_t)((1 - h) * 4), its);
            ptx::tmem_wait_ld();
            float mh[2], lh[2], loh[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mh[e] = u2f(e == h ? mine[0] : its[0]);
                lh[e] = u2f(e == h ? mine[1] : its[1]);
                loh[e] = u2f(e == h ? mine[2] : its[2]);
            }
            // both halves have read before either stores the next tile's P
            ptx::tc_fence_before();
            ptx::bar_sync(2, 256);
            ptx::tc_fence_after();
            const bool on[2] = {lh[0] != 0.f, lh[1] != 0.f};      // a NaN stays on and reaches the output
            const float m = fmaxf(on[0] ? mh[0] : -INFINITY, on[1] ? mh[1] : -INFINITY);
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) w[e] = on[e] ? ptx::ex2_approx(mh[e] - m) : 0.f;
            const float l_all = w[0] * lh[0] + w[1] * lh[1];
            const bool empty = !(on[0] || on[1]);
            const float inv = empty ? 0.f : 1.f / (w[0] * loh[0] + w[1] * loh[1]);
            const float c0 = w[0] * inv, c1 = w[1] * inv;
            const float lse2 = empty ? -INFINITY : m + log2f(l_all);

            // This thread writes columns [h*D/2, (h+1)*D/2) of its row.
            const bool direct = count == was.n && !p.joined;
            const int64_t slot = p.part.slot_of((int)blockIdx.x, was.g * p.c.Hkv + was.h, was.c > 0);
            if (thread == 0 && was.c == 0) line.record(was, (int)blockIdx.x, used, per);
            used += line.start_of(was.c + count) - line.start_of(was.c);
            uint16_t *o_row = nullptr;
            const bool real = row < line.R;
            if (real) {
                const RowPlace r = row_place(p, b, was.h, row);
                o_row = p.o + r.b * p.o_s[0] + r.hq * p.o_s[1] + r.t * p.o_s[2];
                if (h == 0) {
                    if (!direct)
                        p.part.lse[slot * BM + r_local] = lse2;
                    else if (p.lse)
                        p.lse[((int64_t)r.b * p.Hq + r.hq) * p.T + r.t] = lse2 * kLn2;
                }
            }
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
                __syncwarp();
                const int col = h * (D / 2) + c * 32;
                uint32_t oa[32], ob[32];
                ptx::tmem_ld32(tmem + lane_off + Lay::col_o(0) + (uint32_t)col, oa);
                ptx::tmem_ld32(tmem + lane_off + Lay::col_o(1) + (uint32_t)col, ob);
                ptx::tmem_wait_ld();
                if (c + 1 == D / 64) {
                    // O is in registers: the next tile's products may replace it
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(o_read);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (!real || col + 8 * k >= p.c.D) continue;
                    // (a half with no visible key has weight 0 and O_h = 0)
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = empty ? 0.f : fmaf(c0, u2f(oa[8 * k + e]), c1 * u2f(ob[8 * k + e]));
                    if (direct) {
                        *reinterpret_cast<uint4 *>(o_row + col + 8 * k) =
                            make_uint4(ptx::pack16x2<kF16>(x[0], x[1]), ptx::pack16x2<kF16>(x[2], x[3]),
                                       ptx::pack16x2<kF16>(x[4], x[5]), ptx::pack16x2<kF16>(x[6], x[7]));
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(p.part.o) +
                                      (slot * (p.c.D / 4) + (col + 8 * k) / 4) * BM + r_local;
                        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                        dst[BM] = make_float4(x[4], x[5], x[6], x[7]);
                    }
                }
            }
            __syncwarp();
            if (!more) break;
        }
    }
    // ---- teardown ----------------------------------------------------------
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
    // the merge starts when this kernel has ended, and needs the one before too
    if (p.second) ptx::wait_for_primary();
}

template <int D, bool kF16, bool kTwo>
cudaError_t launch(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    static SharedMemory allowed;
    const cudaError_t e = allowed.allow(paged_tc_kernel<D, kF16, kTwo>, TcLayout<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_behind(paged_tc_kernel<D, kF16, kTwo>, dim3((unsigned)ctas), kThreads, TcLayout<D>::kSmemBytes, stream, tk, tv, p);
}

template <int D>
cudaError_t launch_d(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas, cudaStream_t stream)
{
    if (p.two) return p.f16 ? launch<D, true, true>(p, tk, tv, ctas, stream) : launch<D, false, true>(p, tk, tv, ctas, stream);
    return p.f16 ? launch<D, true, false>(p, tk, tv, ctas, stream) : launch<D, false, false>(p, tk, tv, ctas, stream);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams &p, const CUtensorMap &tk, const CUtensorMap &tv, int ctas,
                            cudaStream_t stream)
{
    return p.c.D <= 64 ? launch_d<64>(p, tk, tv, ctas, stream) : launch_d<128>(p, tk, tv, ctas, stream);
}

cudaError_t read_and_clear_status_paged(uint32_t *out)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status_paged, sizeof(v));
    if (e != cudaSuccess) return e;
    if (v) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_status_paged, &zero, sizeof(zero));
        if (e != cudaSuccess) return e;
    }
    *out = v;
    return cudaSuccess;
}

}  // namespace fa
