// fa_four_api.cu -- the C ABI of the 4-bit cache, of positions of several axes and of
// reading a cache back: argument checks, workspace layout and launches.  Declared in
// include/fa.h.
//
// Every check that can fail runs before any launch, so a rejected call has no side
// effect.  The library allocates no device memory.
#include "fa_paged_plan.h"

namespace {

using namespace fa::paged;

// Sequences whose keys are decoded to 16 bits at a time: as many as have kWide bytes of
// them at most, one at least, if that has kMostWide at most.  A sequence counts with all
// keys that its row of the table can hold, since its length is on the device: at D = 128
// and 8 key heads a row for 131072 keys takes 512 MB of workspace, whatever it holds, and
// its sequences are decoded and attended to one after another.  256 tokens of 64
// sequences of 500 keys, with rows for 512, 16384, 131072 and 262144 keys: 382, 717, 2198
// and 3066 us, and for more, where every tile decodes its keys itself, 419; of 8 of 4000
// keys 225 (rows for 4000), 261, 456, 565 and 243.  Tables no wider than the longest
// sequence needs are what this is for.
constexpr int64_t kWide = (int64_t)256 << 20, kMostWide = (int64_t)1 << 30;

// Row tiles of a sequence up to which each decodes its keys itself on the tensor cores;
// more read keys that are decoded once.  1, 2, 3, 4 and 8 tiles, themselves against
// once, in us: 8 sequences of 4000 to 8000 keys 55 and 100, 91 and 120, 126 and 137,
// 163 and 161, 312 and 237; 64 of up to 8000 (4 tiles) 957 and 1017; one of 16384 (2, 4
// and 8) 40 and 53, 64 and 62, 112 and 85.
constexpr int kDirectTiles = 4;

// How a forward over a 4-bit cache is cut, and its workspace.
struct FourPlan {
    bool wide = false;      // decoded first, and then the tensor-core kernel of 16-bit caches
    Plan direct;            // else: the row kernel, or the tensor-core kernel that decodes
    int group = 0;          // sequences at a time
    fa_paged_kv pool{};     // of a group, without its places in the workspace
    size_t pool_bytes = 0, table_bytes = 0, len_bytes = 0, inner = 0, bytes = 0;
    bool ok = true;

    FourPlan(const fa_paged_kv4 &c, int B, int Hq, int T) : direct(B, c, (int64_t)(Hq / c.Hkv) * T, (int64_t)c.table_width * c.page_size)
    {
        const int64_t R = (int64_t)(Hq / c.Hkv) * T;
        const int64_t page = (int64_t)c.Hkv * c.page_size * c.D, each = page * c.table_width * 4;
        wide = direct.tc && direct.part.tiles > kDirectTiles && each > 0 && each <= kMostWide;
        if (!wide) {
            ok = direct.ok;
            bytes = direct.bytes;
            return;
        }
        group = (int)std::max<int64_t>(1, std::min<int64_t>(B, kWide / each));
        const int64_t pages = (int64_t)group * c.table_width;       // (2^30 bytes of rows of 64 at least: fewer than 2^24)
        pool.stride_page = page;
        pool.stride_head = (int64_t)c.page_size * c.D;
        pool.stride_slot = c.D;
        pool.num_pages = (int)pages;
        pool.page_size = c.page_size;
        pool.Hkv = c.Hkv;
        pool.D = c.D;
        pool.table_stride = pool.table_width = c.table_width;
        const Plan p(group, pool, R, (int64_t)c.table_width * c.page_size, false, false);
        ok = p.ok;
        inner = p.bytes;
        pool_bytes = round_up((size_t)pages * page * 2);
        table_bytes = round_up((size_t)pages * 4);
        len_bytes = round_up((size_t)group * 4);
        bytes = 2 * pool_bytes + table_bytes + len_bytes + inner;
    }
};

fa_status check_sizes4(const fa_paged_kv4 *c, int B, int Hq, int T)
{
    if (B < 0 || Hq < 0 || T < 0) return FA_ERR_INVALID_ARG;
    const fa_status st = check_cache4(c, B);
    if (st != FA_OK) return st;
    if (Hq % c->Hkv != 0) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * Hq > INT32_MAX || (int64_t)B * Hq * T > (int64_t)1 << 32) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa_rows from_sequence(const fa_rows &r, int64_t b)
{
    return fa_rows{static_cast<uint16_t *>(r.ptr) + b * r.stride_b, r.stride_b, r.stride_h, r.stride_n};
}

template <typename C>
fa_status read_rows(fa::ReadParams &p, const C *cache, const fa_rows *K, const fa_rows *V, int B, int T, bool four, void *stream)
{
    if ((int64_t)B * T > INT32_MAX) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T == 0) return FA_OK;
    if (!rows_ok(K, B, cache->Hkv, T, cache->D, true) || !rows_ok(V, B, cache->Hkv, T, cache->D, true)) return FA_ERR_INVALID_ARG;
    if (2 * (int64_t)cache->Hkv > INT32_MAX / cache->D) return FA_ERR_INVALID_ARG;
    p.k = static_cast<uint16_t *>(K->ptr);
    strides_of(p.k_s, *K);
    p.v = static_cast<uint16_t *>(V->ptr);
    strides_of(p.v_s, *V);
    p.by_groups = fa::make_fast_div((uint32_t)(cache->D + 15) / 16);
    p.B = B;
    p.T = T;
    return fa::launch_read(p, four, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

fa_status fa_rotary(const fa_rows *Q, const fa_rows *Q_out, const fa_rows *K, const fa_rows *K_out, int B, int Hq, int Hkv,
                    int T, int D, const float *inv_freq, int rot_dim, int interleaved, const fa_positions *positions,
                    int64_t position_offset, int inverse, int f16, void *stream)
{
    if (B < 0 || T < 0 || Hq < 0 || Hkv < 0 || D <= 0) return FA_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256) return FA_ERR_UNSUPPORTED;
    fa::RotaryParams p{};
    const fa_status st = check_turn(p.turn, (int64_t)B * T, D, inv_freq, rot_dim, interleaved, positions, position_offset);
    if (st != FA_OK) return st;
    if ((int64_t)B * T > INT32_MAX || (int64_t)Hq + Hkv > INT32_MAX / D) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T == 0 || Hq + Hkv == 0) return FA_OK;
    const fa_rows *in[2] = {Q, K}, *out[2] = {Q_out, K_out};
    const int H[2] = {Hq, Hkv};
    for (int i = 0; i < 2; ++i) {
        if (H[i] == 0) continue;
        if (!rows_ok(in[i], B, H[i], T, D, false) || !rows_ok(out[i], B, H[i], T, D, true)) return FA_ERR_INVALID_ARG;
        if (out[i]->ptr == in[i]->ptr && !same_rows(*in[i], *out[i], B, H[i], T)) return FA_ERR_INVALID_ARG;
        if (H[1 - i] && out[i]->ptr == in[1 - i]->ptr) return FA_ERR_INVALID_ARG;
        p.x[i] = static_cast<const uint16_t *>(in[i]->ptr);
        strides_of(p.x_s[i], *in[i]);
        p.y[i] = static_cast<uint16_t *>(out[i]->ptr);
        strides_of(p.y_s[i], *out[i]);
        p.H[i] = H[i];
    }
    if (Hq && Hkv && Q_out->ptr == K_out->ptr) return FA_ERR_INVALID_ARG;
    p.turn.inverse = inverse ? 1 : 0;
    p.by_t = fa::make_fast_div((uint32_t)T);
    p.B = B;
    p.T = T;
    p.D = D;
    p.f16 = f16 ? 1 : 0;
    return fa::launch_rotary(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_kv_append_q4(const fa_paged_kv4 *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                          const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim, int interleaved,
                          const fa_positions *positions, int64_t position_offset, int f16, void *stream)
{
    if (B < 0 || T < 0 || Hq < 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache4(cache, B);
    if (st != FA_OK) return st;
    fa::Append4Params p{};
    st = check_turn(p.turn, (int64_t)B * T, cache->D, inv_freq, rot_dim, interleaved, positions, position_offset);
    if (st != FA_OK) return st;
    if ((int64_t)B * T > INT32_MAX) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T == 0) return FA_OK;
    const bool queries = Q && Hq > 0;
    st = check_append(K, V, Q, Q_out, B, queries ? Hq : 0, 2 * (int64_t)cache->Hkv > INT32_MAX / 256 ? INT32_MAX : cache->Hkv, T, cache->D);
    if (st != FA_OK) return st;
    p.c = cache4_of(*cache);
    put_rows(p, K, V, queries ? Q : nullptr, Q_out);
    p.by_t = fa::make_fast_div((uint32_t)T);
    p.B = B;
    p.T = T;
    p.Hq = queries ? Hq : 0;
    p.f16 = f16 ? 1 : 0;
    return fa::launch_append4(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_kv_read(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, int B, int T, void *stream)
{
    if (B < 0 || T < 0) return FA_ERR_INVALID_ARG;
    const fa_status st = check_cache(cache, B);
    if (st != FA_OK) return st;
    fa::ReadParams p{};
    p.c = cache_of(*cache);
    return read_rows(p, cache, K, V, B, T, false, stream);
}

fa_status fa_kv_read_q4(const fa_paged_kv4 *cache, const fa_rows *K, const fa_rows *V, int B, int T, int f16, void *stream)
{
    if (B < 0 || T < 0) return FA_ERR_INVALID_ARG;
    const fa_status st = check_cache4(cache, B);
    if (st != FA_OK) return st;
    fa::ReadParams p{};
    p.c4 = cache4_of(*cache);
    p.f16 = f16 ? 1 : 0;
    return read_rows(p, cache, K, V, B, T, true, stream);
}

size_t fa_fwd_paged_q4_workspace_bytes(const fa_paged_kv4 *cache, int B, int Hq, int T)
{
    if (check_sizes4(cache, B, Hq, T) != FA_OK || (int64_t)B * Hq * T == 0) return 0;
    const FourPlan plan(*cache, B, Hq, T);
    return plan.ok ? plan.bytes : 0;
}

fa_status fa_fwd_paged_q4(const fa_rows *Q, const fa_paged_kv4 *cache, const fa_rows *O, float *LSE, int B, int Hq, int T,
                          int causal, float scale, int f16, void *workspace, size_t workspace_bytes, void *stream)
{
    const fa_status st = check_sizes4(cache, B, Hq, T);
    if (st != FA_OK) return st;
    if ((int64_t)B * Hq * T == 0) return FA_OK;
    const int D = cache->D;
    if (!rows_ok(Q, B, Hq, T, D, false) || !rows_ok(O, B, Hq, T, D, true)) return FA_ERR_INVALID_ARG;
    if (LSE && !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
    const int64_t own_keys = (int64_t)cache->table_width * cache->page_size;
    const int G = Hq / cache->Hkv;
    FourPlan whole(*cache, B, Hq, T);
    if (!whole.ok || !workspace || !aligned(workspace, 16) || workspace_bytes < whole.bytes) return FA_ERR_INVALID_ARG;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);

    if (whole.wide) {
        uint8_t *at = static_cast<uint8_t *>(workspace);
        fa::WidenParams w{};
        w.f16 = f16 ? 1 : 0;
        w.k = reinterpret_cast<uint16_t *>(at);
        w.v = reinterpret_cast<uint16_t *>(at + whole.pool_bytes);
        w.table = reinterpret_cast<int32_t *>(at + 2 * whole.pool_bytes);
        w.seq_len = reinterpret_cast<int32_t *>(at + 2 * whole.pool_bytes + whole.table_bytes);
        uint8_t *inner = at + 2 * whole.pool_bytes + whole.table_bytes + whole.len_bytes;
        fa_paged_kv pool = whole.pool;
        pool.k = w.k;
        pool.v = w.v;
        pool.table = w.table;
        pool.seq_len = w.seq_len;
        for (int b = 0; b < B; b += whole.group) {
            const int n = std::min(whole.group, B - b);
            fa_paged_kv4 part = *cache;
            part.table += (int64_t)b * cache->table_stride;
            part.seq_len += b;
            w.c = cache4_of(part);
            if (fa::launch_widen_pages(w, (int64_t)n * cache->table_width, cs) != cudaSuccess) return FA_ERR_CUDA;
            const fa_rows q = from_sequence(*Q, b), o = from_sequence(*O, b);
            const fa_status s = fa_fwd_paged(&q, &pool, &o, LSE ? LSE + (int64_t)b * Hq * T : nullptr, n, Hq, T, causal, scale,
                                             f16, inner, whole.inner, stream);
            if (s != FA_OK) return s;
        }
        return FA_OK;
    }

    Plan &plan = whole.direct;
    plan.place(static_cast<uint8_t *>(workspace), D);
    fa::FourParams f{};
    f.c = cache4_of(*cache);
    fa::PagedParams &p = f.p;
    p.c.table = cache->table;
    p.c.table_stride = cache->table_stride;
    p.c.seq_len = cache->seq_len;
    p.c.table_width = cache->table_width;
    p.c.num_pages = cache->num_pages;
    p.c.page_size = cache->page_size;
    p.c.by_page = f.c.by_page;
    p.c.Hkv = cache->Hkv;
    p.c.D = D;
    p.q = static_cast<const uint16_t *>(Q->ptr);
    strides_of(p.q_s, *Q);
    p.o = static_cast<uint16_t *>(O->ptr);
    strides_of(p.o_s, *O);
    p.lse = LSE;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.G = G;
    p.by_g = fa::make_fast_div((uint32_t)G);
    p.by_gt = fa::make_fast_div((uint32_t)(G * T));
    p.causal = causal ? 1 : 0;
    p.f16 = f16 ? 1 : 0;
    const bool given = scale > 0.f && !std::isinf(scale);
    p.scale_log2 = (given ? scale : 1.0f / std::sqrt((float)D)) * 1.4426950408889634f;
    p.part = plan.part;
    p.wait_limit_ns = fa::wait_budget_ns();
    // (eight chunks a warp at most here, too: 16 sequences of 2000 keys 13.9 us, with four
    // chunks 17.4; one of 32000 keys 18.1, with 16 chunks 23.8)
    p.team = plan.tc ? 0 : team_size(D, plan, (own_keys + p.part.chunk - 1) / p.part.chunk, fa::four_teams_at_once);
    if (p.team) return fa::launch_four_team(f, (int)plan.items * p.team, cs) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    if ((plan.tc ? fa::launch_four_tc(f, (int)plan.ctas, cs) : fa::launch_four_rows(f, (int)plan.ctas, cs)) != cudaSuccess) return FA_ERR_CUDA;

    fa::MergeParams m{};
    m.src[m.n_src++] = plan.part;
    m.seq_len = cache->seq_len;
    m.max_len = (int)own_keys;
    m.o = p.o;
    strides_of(m.o_s, *O);
    m.lse = LSE;
    m.B = B;
    m.T = T;
    m.Hq = Hq;
    m.G = G;
    m.by_g = p.by_g;
    m.by_r = p.by_gt;
    m.D = D;
    m.causal = p.causal;
    m.f16 = p.f16;
    const int64_t states = plan.pieces / plan.items + 1;
    return fa::launch_paged_merge(m, (int)states, fa::sm_count_of(fa::current_device()), cs) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
