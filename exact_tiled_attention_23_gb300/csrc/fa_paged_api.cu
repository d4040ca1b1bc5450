// fa_paged_api.cu -- the C ABI of the paged-cache operators: argument checks,
// workspace layout and launches.  Declared in include/fa.h.
//
// Every check that can fail runs before any launch, so a rejected call has no
// side effect.  The library allocates no device memory.
#include "fa.h"
#include "fa_internal.h"
#include "fa_paged.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides that 16-byte accesses can follow.
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// A [B, H, T, D] view: a pointer that 16-byte accesses can use, and strides.
// Outputs may not have two elements at one address.
bool rows_ok(const fa_rows *r, int B, int H, int T, int D, bool output)
{
    if (!r || !r->ptr || !aligned(r->ptr, 16)) return false;
    if (!stride_ok(r->stride_b) || !stride_ok(r->stride_h) || !stride_ok(r->stride_n)) return false;
    if (!output) return true;
    return (B <= 1 || r->stride_b >= D) && (H <= 1 || r->stride_h >= D) && (T <= 1 || r->stride_n >= D);
}

// Most keys of a sequence: places in it, up to the end of a block past the last
// key, are 32-bit numbers.
constexpr int64_t kMostKeys = INT32_MAX - 4095;

fa_status check_cache(const fa_paged_kv *c, int B)
{
    if (!c) return FA_ERR_INVALID_ARG;
    if (c->D <= 0 || c->Hkv <= 0 || c->num_pages < 0 || c->page_size <= 0 || c->table_width < 0) return FA_ERR_INVALID_ARG;
    if (c->D % 8 != 0 || (c->D > 128 && c->D != 256)) return FA_ERR_UNSUPPORTED;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_INVALID_ARG;
    if (!stride_ok(c->stride_page) || !stride_ok(c->stride_head) || !stride_ok(c->stride_slot)) return FA_ERR_INVALID_ARG;
    if ((c->num_pages > 1 && c->stride_page < c->D) || (c->Hkv > 1 && c->stride_head < c->D) ||
        (c->page_size > 1 && c->stride_slot < c->D))
        return FA_ERR_INVALID_ARG;
    if ((B > 0 && !c->seq_len) || !aligned(c->seq_len, 4)) return FA_ERR_INVALID_ARG;
    if ((B > 0 && c->table_width > 0 && !c->table) || !aligned(c->table, 4)) return FA_ERR_INVALID_ARG;
    if (B > 1 && c->table_stride < c->table_width) return FA_ERR_INVALID_ARG;
    if ((int64_t)c->table_width * c->page_size > kMostKeys) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa::PagedCache cache_of(const fa_paged_kv &c)
{
    fa::PagedCache r{};
    r.k = static_cast<uint16_t *>(c.k);
    r.v = static_cast<uint16_t *>(c.v);
    r.s_page = c.stride_page;
    r.s_head = c.stride_head;
    r.s_slot = c.stride_slot;
    r.table = c.table;
    r.table_stride = c.table_stride;
    r.table_width = c.table_width;
    r.seq_len = c.seq_len;
    r.num_pages = c.num_pages;
    r.page_size = c.page_size;
    r.by_page = fa::make_fast_div((uint32_t)c.page_size);
    r.Hkv = c.Hkv;
    r.D = c.D;
    return r;
}

void strides_of(int64_t (&s)[3], const fa_rows &r)
{
    s[0] = r.stride_b;
    s[1] = r.stride_h;
    s[2] = r.stride_n;
}

// Whether rows of one address are the same rows.
bool same_rows(const fa_rows &x, const fa_rows &y, int B, int H, int T)
{
    return x.ptr == y.ptr && (B == 1 || x.stride_b == y.stride_b) && (H == 1 || x.stride_h == y.stride_h) &&
           (T == 1 || x.stride_n == y.stride_n);
}

size_t round_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Most stacked rows that the row kernel takes where the tensor-core kernel could.
// Row kernel against tensor cores in us, geometric means of seven batches (1 to 64
// sequences of 500 to 65536 keys, 1 or 8 key heads of 4 queries, bf16): D = 64: 16
// rows 18 and 26, 32 rows 26.2 and 26.3, 36 rows 38 and 27; D = 128: 16 rows 32 and
// 30, 20 to 32 rows 50 to 56 and 30 to 31, 36 rows 78 and 32.  At D = 128 and 17 to
// 32 rows it is the weights of two 16-bit numbers that the row kernel is for.
constexpr int64_t kMostRows = 32;

// Key rows per TMA box of this pool: the largest power of two, 8 (the rows of a
// swizzle atom) to 128, that divides a page.  0 where TMA cannot copy it: other
// page sizes, strides past a tensor map's range.
int box_rows_of(const fa_paged_kv &c)
{
    if (c.page_size % 8 != 0 || c.num_pages <= 0) return 0;
    const int64_t far = (int64_t)1 << 38;
    if (c.stride_page >= far || c.stride_head >= far || c.stride_slot >= far) return 0;
    int box = 8;
    while (box < 128 && c.page_size % (2 * box) == 0) box *= 2;
    return box;
}

// How one part of a call (the sequences' own keys, or a shared prefix) is cut
// into tiles, and its piece of the workspace.
struct Plan {
    fa::Partials part{};
    int64_t items = 0;      // tiles in all
    int64_t ctas = 0;
    int64_t pieces = 0;     // of the line: one per CTA, or per warp of the row kernel
    size_t bytes = 0;
    bool ok = true;
    bool tc = false;        // the tensor-core kernel (else the row kernel)
    int box = 0;            // key rows per TMA box, 0: no TMA

    // rows: stacked query rows per (sequence, key head); keys: most keys of a
    // sequence; joined: every tile leaves a state
    Plan(int nseq, const fa_paged_kv &c, int64_t rows, int64_t keys, bool stacked, bool joined)
    {
        const int Hkv = c.Hkv, D = c.D;
        box = box_rows_of(c);
        tc = box > 0 && D <= 128 && rows > kMostRows;    // (TMEM holds two O tiles of 128 columns at most)
        if (!tc) box = std::min(box, fa::paged_rows_chunk(D));
        part.rows = tc ? 128 : fa::paged_rows_per_tile(D, rows);
        part.chunk = tc ? fa::kBlockKeys : fa::paged_rows_chunk(D);
        const int64_t tiles = (rows + part.rows - 1) / part.rows;
        items = (int64_t)nseq * Hkv * tiles;
        if (rows > INT32_MAX / 2 || Hkv > 65535 || (int64_t)Hkv * tiles > INT32_MAX || items > INT32_MAX) {
            ok = false;
            return;
        }
        part.tiles = (int)tiles;
        part.stacked = stacked;
        part.fixed_len = stacked ? (int)keys : 0;
        const int64_t chunks = items * ((keys + part.chunk - 1) / part.chunk);
        // places on the line are 32-bit numbers
        if (chunks + 4096 > (tc ? UINT32_MAX / (1 + fa::kBlocksTile) : UINT32_MAX / (1 + fa::kRowsTile))) {
            ok = false;
            return;
        }
        ctas = (int64_t)fa::sm_count_of(fa::current_device()) * (tc ? 1 : fa::paged_rows_ctas_per_sm(D, part.rows));
        const int each = tc ? 1 : fa::kRowsWarps;
        ctas = std::max<int64_t>(1, std::min(ctas, (chunks + each - 1) / each));
        pieces = ctas * each;
        part.slot_rows = (int)std::min<int64_t>(part.rows, tiles == 1 ? (tc ? 128 : rows) : part.rows);
        part.pairs = !joined && items > pieces;
        const size_t slots = (size_t)(part.pairs ? 2 * pieces : pieces + items);
        if (slots > INT32_MAX) {
            ok = false;
            return;
        }
        part.slots = (int)slots;
        bytes = round_up((size_t)items * sizeof(fa::TileSlots)) + round_up(slots * part.slot_rows * 4) + round_up(slots * part.slot_rows * D * 4);
    }

    // Places the piece at `at`; returns its end.
    uint8_t *place(uint8_t *at, int D)
    {
        const size_t slots = (size_t)part.slots;
        part.tile = reinterpret_cast<fa::TileSlots *>(at);
        at += round_up((size_t)items * sizeof(fa::TileSlots));
        part.lse = reinterpret_cast<float *>(at);
        at += round_up(slots * part.slot_rows * 4);
        part.o = reinterpret_cast<float *>(at);
        return at + round_up(slots * part.slot_rows * D * 4);
    }
};

// CTAs of a team per tile, 0 where teams do not pay.  A team's tile has up to 8
// rows, so that its states fit the stages.  All teams are on the GPU at once
// (16 teams of 8 where 15 fit: 10.1 us, as teams of 4: 6.3), and a warp has at
// most eight chunks of the longest sequence that the table allows.  With 8 of
// 128 tiles of 1024 keys: 12.0 us, cut as a line 18.4, and where one sequence
// alone is that long 11.2 and 10.2, since a line spreads it over the GPU; with 16
// of 2048 keys 24.3 and 29.9, but 18.9 and 13.6.
int team_size(const fa_paged_kv &c, const Plan &own, int prefix_len, int64_t own_keys)
{
    constexpr int kMostChunks = 8;
    if (c.D > 128 || own.part.rows != 8 || own.part.tiles != 1) return 0;
    const int chunk = fa::paged_rows_chunk(c.D), device = fa::current_device();
    if (own.items > fa::sm_count_of(device)) return 0;
    const int64_t chunks = (prefix_len + (int64_t)chunk - 1) / chunk + (own_keys + chunk - 1) / chunk;
    int team = 0;
    for (int t = 1; t <= fa::kMostTeam && own.items <= fa::paged_teams_at_once(device, t); t *= 2) {
        const int64_t each = (chunks + t * fa::kTeamWarps - 1) / (t * fa::kTeamWarps);
        if (each <= kMostChunks) team = t;
        if (each <= 1) break;
    }
    return team;
}

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
    p.team = team_size(*c, own, prefix_len, own_keys);
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
    if (B < 0 || T < 0 || Hq < 0) return FA_ERR_INVALID_ARG;
    const fa_status st = check_cache(cache, B);
    if (st != FA_OK) return st;
    if (rot_dim < 0 || rot_dim > cache->D || rot_dim % 2 != 0) return FA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!inv_freq || !aligned(inv_freq, 4))) return FA_ERR_INVALID_ARG;
    if (position_offset < 0 || position_offset > (int64_t)1 << 40) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T > INT32_MAX) return FA_ERR_INVALID_ARG;
    if ((int64_t)B * T == 0) return FA_OK;
    const int D = cache->D;
    if (!rows_ok(K, B, cache->Hkv, T, D, false) || !rows_ok(V, B, cache->Hkv, T, D, false)) return FA_ERR_INVALID_ARG;
    const bool queries = Q && Hq > 0;
    if (queries && (!rows_ok(Q, B, Hq, T, D, false) || !rows_ok(Q_out, B, Hq, T, D, true))) return FA_ERR_INVALID_ARG;
    if (queries && Q_out->ptr == Q->ptr && !same_rows(*Q, *Q_out, B, Hq, T)) return FA_ERR_INVALID_ARG;
    if (queries && (Q_out->ptr == K->ptr || Q_out->ptr == V->ptr)) return FA_ERR_INVALID_ARG;
    if ((int64_t)(queries ? Hq : 0) + cache->Hkv > INT32_MAX / D) return FA_ERR_INVALID_ARG;

    fa::AppendParams p{};
    p.c = cache_of(*cache);
    p.k = static_cast<const uint16_t *>(K->ptr);
    strides_of(p.k_s, *K);
    p.v = static_cast<const uint16_t *>(V->ptr);
    strides_of(p.v_s, *V);
    if (queries) {
        p.q = static_cast<const uint16_t *>(Q->ptr);
        strides_of(p.q_s, *Q);
        p.q_out = static_cast<uint16_t *>(Q_out->ptr);
        strides_of(p.qo_s, *Q_out);
    }
    p.inv_freq = inv_freq;
    p.offset = position_offset;
    p.B = B;
    p.T = T;
    p.Hq = queries ? Hq : 0;
    p.rot = rot_dim;
    p.interleaved = interleaved ? 1 : 0;
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
