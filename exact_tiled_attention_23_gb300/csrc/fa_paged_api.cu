// fa_paged_api.cu -- the C ABI of the paged-cache operators: argument checks,
// workspace layout and launches.  Declared in include/fa.h.
//
// Every check that can fail runs before any launch, so a rejected call has no
// side effect.  The library allocates no device memory.
#include "fa_paged_plan.h"

namespace {

using namespace fa::paged;

// One part's kernel.
bool launch_part(fa::PagedParams p, const fa_paged_kv &c, const Plan &plan, cudaStream_t stream)
{
    p.part = plan.part;
    CUtensorMap tk{}, tv{};
    p.box_rows = plan.box;
    p.wait_limit_ns = fa::wait_budget_ns();
    if (!plan.box)
        return (p.team ? fa::launch_paged_team(p, tk, tv, (int)plan.items * p.team, stream)
                       : fa::launch_paged_rows(p, tk, tv, (int)plan.ctas, stream)) == cudaSuccess;
    // [D, slot, head, page]; the stride of a dimension of one entry is not followed
    const uint64_t row = (uint64_t)c.D * 2;
    const uint64_t dims[4] = {(uint64_t)c.D, (uint64_t)c.page_size, (uint64_t)c.Hkv, (uint64_t)c.num_pages};
    const uint64_t strides[3] = {(uint64_t)c.stride_slot * 2, c.Hkv > 1 ? (uint64_t)c.stride_head * 2 : row,
                                 c.num_pages > 1 ? (uint64_t)c.stride_page * 2 : row};
    const uint32_t box[4] = {64, (uint32_t)plan.box, 1, 1};
    if (!fa::encode_tiled16(&tk, c.k, 4, dims, strides, box, p.f16 != 0) ||
        !fa::encode_tiled16(&tv, c.v, 4, dims, strides, box, p.f16 != 0))
        return false;
    if (p.team) return fa::launch_paged_team(p, tk, tv, (int)plan.items * p.team, stream) == cudaSuccess;
    return (plan.tc ? fa::launch_paged_tc(p, tk, tv, (int)plan.ctas, stream)
                    : fa::launch_paged_rows(p, tk, tv, (int)plan.ctas, stream)) == cudaSuccess;
}

// Sizes of a paged forward; `keys` is what a table row can hold.
fa_status check_sizes(const fa_paged_kv *c, int B, int Hq, int T)
{
    if (B < 0 || Hq < 0 || T < 0) return FA_ERR_INVALID_ARG;
    const fa_status st = check_cache(c, B);
    if (st != FA_OK) return st;
    if (Hq % c->Hkv != 0) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * Hq > INT32_MAX || (int64_t)B * Hq * T > (int64_t)1 << 32) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa_status run(const fa_rows *Q, const fa_paged_kv *c, const int32_t *prefix_table, int prefix_len, const fa_rows *O,
              float *LSE, int B, int Hq, int T, int causal, float scale, int f16, void *workspace,
              size_t workspace_bytes, void *stream)
{
    fa_status st = check_sizes(c, B, Hq, T);
    if (st != FA_OK) return st;
    if (prefix_len < 0) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * Hq * T == 0) return FA_OK;
    const int D = c->D;
    if (!rows_ok(Q, B, Hq, T, D, false) || !rows_ok(O, B, Hq, T, D, true)) return FA_ERR_INVALID_ARG;
    if (LSE && !aligned(LSE, 4)) return FA_ERR_INVALID_ARG;
    if (prefix_len > 0 && (!prefix_table || !aligned(prefix_table, 4))) return FA_ERR_INVALID_ARG;
    const int64_t own_keys = (int64_t)c->table_width * c->page_size;
    if (own_keys + prefix_len > kMostKeys) return FA_ERR_INVALID_ARG;
    const int G = Hq / c->Hkv;
    Plan own(B, *c, (int64_t)G * T, own_keys, false, prefix_len > 0);
    Plan front(1, *c, (int64_t)G * T * B, prefix_len, true, true);
    if (!own.ok || (prefix_len > 0 && !front.ok)) return FA_ERR_INVALID_ARG;
    const size_t need = own.bytes + (prefix_len > 0 ? front.bytes : 0);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return FA_ERR_INVALID_ARG;
    uint8_t *end = own.place(static_cast<uint8_t *>(workspace), D);
    if (prefix_len > 0) front.place(end, D);

    fa::PagedParams p{};
    p.c = cache_of(*c);
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
    p.joined = prefix_len > 0;

    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int64_t chunk = own.part.chunk;
    p.team = team_size(D, own, (prefix_len + chunk - 1) / chunk + (own_keys + chunk - 1) / chunk, fa::paged_teams_at_once);
    if (p.team) {
        p.prefix_table = prefix_table;
        p.prefix_len = prefix_len;
        return launch_part(p, *c, own, cs) ? FA_OK : FA_ERR_CUDA;
    }
    fa::MergeParams m{};
    m.src[m.n_src++] = own.part;
    if (prefix_len > 0) {
        p.beside.on = front.tc && !own.tc;
        p.beside.sms = fa::sm_count_of(fa::current_device());
        p.beside.per_sm = fa::paged_rows_ctas_per_sm(D, own.part.rows) * fa::kRowsWarps;
        p.beside.blocks = (int)(front.items * ((prefix_len + front.part.chunk - 1) / front.part.chunk));
        p.beside.chunk = own.part.chunk;
        p.beside.tiles = own.part.tiles * c->Hkv;
        p.beside.seq_len = c->seq_len;
        p.beside.cap = (int)own_keys;
        p.beside.B = B;
        fa::PagedParams f = p;
        // (as exact as the row kernel's own keys, whatever the batch stacks up to)
        f.two = (int64_t)G * T <= kMostRows;
        f.c.table = prefix_table;
        f.c.table_width = (int)((prefix_len + (int64_t)c->page_size - 1) / c->page_size);
        f.c.table_stride = 0;
        f.c.seq_len = nullptr;
        f.c.fixed_len = prefix_len;
        if (!launch_part(f, *c, front, cs)) return FA_ERR_CUDA;
        m.src[m.n_src++] = front.part;
        p.second = 1;
    }
    if (!launch_part(p, *c, own, cs)) return FA_ERR_CUDA;
    m.seq_len = c->seq_len;
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
    m.joined = p.joined;
    const int64_t states = own.pieces / own.items + 1 + (prefix_len > 0 ? front.pieces / front.items + 1 : 0);
    return fa::launch_paged_merge(m, (int)states, fa::sm_count_of(fa::current_device()), cs) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

namespace fa {

int current_device()
{
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

int sm_count_of(int device)
{
    static std::atomic<int> known[64];
    if (device < 0) return 148;
    if (device < 64 && known[device].load(std::memory_order_relaxed) > 0) return known[device].load(std::memory_order_relaxed);
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0) return 148;
    if (device < 64) known[device].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace fa

extern "C" {

fa_status fa_kv_append(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                       const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim,
                       int interleaved, int64_t position_offset, int f16, void *stream)
{
    return fa_kv_append_at(cache, K, V, Q, Q_out, B, Hq, T, inv_freq, rot_dim, interleaved, nullptr, position_offset, f16, stream);
}

fa_status fa_kv_append_at(const fa_paged_kv *cache, const fa_rows *K, const fa_rows *V, const fa_rows *Q,
                          const fa_rows *Q_out, int B, int Hq, int T, const float *inv_freq, int rot_dim, int interleaved,
                          const fa_positions *positions, int64_t position_offset, int f16, void *stream)
{
    if (B < 0 || T < 0 || Hq < 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_cache(cache, B);
    if (st != FA_OK) return st;
    fa::AppendParams p{};
    st = check_turn(p.turn, (int64_t)B * T, cache->D, inv_freq, rot_dim, interleaved, positions, position_offset);
    if (st != FA_OK) return st;
    if ((int64_t)B * T > INT32_MAX) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T == 0) return FA_OK;
    const bool queries = Q && Hq > 0;
    st = check_append(K, V, Q, Q_out, B, queries ? Hq : 0, cache->Hkv, T, cache->D);
    if (st != FA_OK) return st;

    p.c = cache_of(*cache);
    put_rows(p, K, V, queries ? Q : nullptr, Q_out);
    p.by_t = fa::make_fast_div((uint32_t)T);
    p.B = B;
    p.T = T;
    p.Hq = queries ? Hq : 0;
    p.f16 = f16 ? 1 : 0;
    return fa::launch_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_paged_workspace_bytes(const fa_paged_kv *cache, int B, int Hq, int T)
{
    return fa_fwd_shared_prefix_workspace_bytes(cache, 0, B, Hq, T);
}

fa_status fa_fwd_paged(const fa_rows *Q, const fa_paged_kv *cache, const fa_rows *O, float *LSE, int B, int Hq, int T,
                       int causal, float scale, int f16, void *workspace, size_t workspace_bytes, void *stream)
{
    return run(Q, cache, nullptr, 0, O, LSE, B, Hq, T, causal, scale, f16, workspace, workspace_bytes, stream);
}

size_t fa_fwd_shared_prefix_workspace_bytes(const fa_paged_kv *cache, int prefix_len, int B, int Hq, int T)
{
    if (check_sizes(cache, B, Hq, T) != FA_OK || prefix_len < 0 || (int64_t)B * Hq * T == 0) return 0;
    const int G = Hq / cache->Hkv;
    const Plan own(B, *cache, (int64_t)G * T, (int64_t)cache->table_width * cache->page_size, false, prefix_len > 0);
    if (!own.ok || (int64_t)cache->table_width * cache->page_size + prefix_len > kMostKeys) return 0;
    if (prefix_len == 0) return own.bytes;
    const Plan front(1, *cache, (int64_t)G * T * B, prefix_len, true, true);
    return front.ok ? own.bytes + front.bytes : 0;
}

fa_status fa_fwd_shared_prefix(const fa_rows *Q, const fa_paged_kv *cache, const int32_t *prefix_table, int prefix_len,
                               const fa_rows *O, float *LSE, int B, int Hq, int T, int causal, float scale, int f16,
                               void *workspace, size_t workspace_bytes, void *stream)
{
    return run(Q, cache, prefix_table, prefix_len, O, LSE, B, Hq, T, causal, scale, f16, workspace, workspace_bytes,
               stream);
}

}  // extern "C"
