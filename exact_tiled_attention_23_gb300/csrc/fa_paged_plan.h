// fa_paged_plan.h -- what the host sides of the paged-cache operators share: argument
// checks, and how a call is cut into tiles and its workspace laid out (not part of the
// public C ABI).
#pragma once

#include "fa.h"
#include "fa_four_rows.h"
#include "fa_internal.h"
#include "fa_paged.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace fa::paged {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides that 16-byte accesses can follow.
inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0; }

// A [B, H, T, D] view: a pointer that 16-byte accesses can use, and strides.
// Outputs may not have two elements at one address.
inline bool rows_ok(const fa_rows *r, int B, int H, int T, int D, bool output)
{
    if (!r || !r->ptr || !aligned(r->ptr, 16)) return false;
    if (!stride_ok(r->stride_b) || !stride_ok(r->stride_h) || !stride_ok(r->stride_n)) return false;
    if (!output) return true;
    return (B <= 1 || r->stride_b >= D) && (H <= 1 || r->stride_h >= D) && (T <= 1 || r->stride_n >= D);
}

// Most keys of a sequence: places in it, up to the end of a block past the last
// key, are 32-bit numbers.
constexpr int64_t kMostKeys = INT32_MAX - 4095;

inline fa_status check_cache(const fa_paged_kv *c, int B)
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

inline fa::PagedCache cache_of(const fa_paged_kv &c)
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

inline fa_status check_cache4(const fa_paged_kv4 *c, int B)
{
    if (!c) return FA_ERR_INVALID_ARG;
    if (c->D <= 0 || c->Hkv <= 0 || c->num_pages < 0 || c->page_size <= 0 || c->table_width < 0) return FA_ERR_INVALID_ARG;
    if (c->D % 8 != 0 || (c->D > 128 && c->D != 256)) return FA_ERR_UNSUPPORTED;
    for (const void *x : {c->k, c->v, c->k_scales, c->v_scales})
        if (!x || !aligned(x, 16)) return FA_ERR_INVALID_ARG;
    const int P = fa::padded4(c->D);
    const int64_t row = P / 2, scales = P / 16;
    const int64_t s[6] = {c->stride_page, c->stride_head, c->stride_slot,
                          c->scale_stride_page, c->scale_stride_head, c->scale_stride_slot};
    const bool many[3] = {c->num_pages > 1, c->Hkv > 1, c->page_size > 1};
    for (int i = 0; i < 3; ++i) {
        if (s[i] < 0 || s[i] % 16 != 0 || s[3 + i] < 0 || s[3 + i] % scales != 0) return FA_ERR_INVALID_ARG;
        if (many[i] && (s[i] < row || s[3 + i] < scales)) return FA_ERR_INVALID_ARG;
    }
    if ((B > 0 && !c->seq_len) || !aligned(c->seq_len, 4)) return FA_ERR_INVALID_ARG;
    if ((B > 0 && c->table_width > 0 && !c->table) || !aligned(c->table, 4)) return FA_ERR_INVALID_ARG;
    if (B > 1 && c->table_stride < c->table_width) return FA_ERR_INVALID_ARG;
    if ((int64_t)c->table_width * c->page_size > kMostKeys) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

inline fa::PagedCache4 cache4_of(const fa_paged_kv4 &c)
{
    fa::PagedCache4 r{};
    r.k = static_cast<uint8_t *>(c.k);
    r.v = static_cast<uint8_t *>(c.v);
    r.ks = static_cast<uint8_t *>(c.k_scales);
    r.vs = static_cast<uint8_t *>(c.v_scales);
    r.s_page = c.stride_page;
    r.s_head = c.stride_head;
    r.s_slot = c.stride_slot;
    r.t_page = c.scale_stride_page;
    r.t_head = c.scale_stride_head;
    r.t_slot = c.scale_stride_slot;
    r.table = c.table;
    r.table_stride = c.table_stride;
    r.seq_len = c.seq_len;
    r.table_width = c.table_width;
    r.num_pages = c.num_pages;
    r.page_size = c.page_size;
    r.by_page = fa::make_fast_div((uint32_t)c.page_size);
    r.Hkv = c.Hkv;
    r.D = c.D;
    return r;
}

inline void strides_of(int64_t (&s)[3], const fa_rows &r)
{
    s[0] = r.stride_b;
    s[1] = r.stride_h;
    s[2] = r.stride_n;
}

// Whether rows of one address are the same rows.
inline bool same_rows(const fa_rows &x, const fa_rows &y, int B, int H, int T)
{
    return x.ptr == y.ptr && (B == 1 || x.stride_b == y.stride_b) && (H == 1 || x.stride_h == y.stride_h) &&
           (T == 1 || x.stride_n == y.stride_n);
}

inline size_t round_up(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// The rotation's arguments for so many tokens, checked.  (Positions of no tokens need
// no memory.)
inline fa_status check_turn(fa::TurnParams &t, int64_t tokens, int D, const float *inv_freq, int rot_dim, int interleaved,
                            const fa_positions *positions, int64_t position_offset)
{
    if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0) return FA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!inv_freq || !aligned(inv_freq, 4))) return FA_ERR_INVALID_ARG;
    if (position_offset < 0 || position_offset > (int64_t)1 << 40) return FA_ERR_INVALID_ARG;
    t = fa::TurnParams{};
    t.inv_freq = inv_freq;
    t.offset = position_offset;
    t.rot = rot_dim;
    t.interleaved = interleaved ? 1 : 0;
    if (positions) {
        if ((tokens > 0 && !positions->n) || !aligned(positions->n, 4) || positions->axes < 1 || !aligned(positions->pair_axis, 4)) return FA_ERR_INVALID_ARG;
        if (positions->stride_axis < 0 || positions->stride_b < 0 || positions->stride_t < 0) return FA_ERR_INVALID_ARG;
        t.pos = positions->n;
        t.pos_s[0] = positions->stride_axis;
        t.pos_s[1] = positions->stride_b;
        t.pos_s[2] = positions->stride_t;
        t.pair_axis = positions->pair_axis;
        t.axes = positions->axes;
    }
    return FA_OK;
}

// The tokens of an append, checked.  Hq: 0 without queries.
inline fa_status check_append(const fa_rows *K, const fa_rows *V, const fa_rows *Q, const fa_rows *Q_out, int B, int Hq,
                              int Hkv, int T, int D)
{
    if (!rows_ok(K, B, Hkv, T, D, false) || !rows_ok(V, B, Hkv, T, D, false)) return FA_ERR_INVALID_ARG;
    if (Hq > 0) {
        if (!rows_ok(Q, B, Hq, T, D, false) || !rows_ok(Q_out, B, Hq, T, D, true)) return FA_ERR_INVALID_ARG;
        if (Q_out->ptr == Q->ptr && !same_rows(*Q, *Q_out, B, Hq, T)) return FA_ERR_INVALID_ARG;
        if (Q_out->ptr == K->ptr || Q_out->ptr == V->ptr) return FA_ERR_INVALID_ARG;
    }
    return (int64_t)Hq + Hkv > INT32_MAX / D ? FA_ERR_INVALID_ARG : FA_OK;
}

template <typename P>
void put_rows(P &p, const fa_rows *K, const fa_rows *V, const fa_rows *Q, const fa_rows *Q_out)
{
    p.k = static_cast<const uint16_t *>(K->ptr);
    strides_of(p.k_s, *K);
    p.v = static_cast<const uint16_t *>(V->ptr);
    strides_of(p.v_s, *V);
    if (!Q) return;
    p.q = static_cast<const uint16_t *>(Q->ptr);
    strides_of(p.q_s, *Q);
    p.q_out = static_cast<uint16_t *>(Q_out->ptr);
    strides_of(p.qo_s, *Q_out);
}

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
inline int box_rows_of(const fa_paged_kv &c)
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
        const int D = c.D;
        box = box_rows_of(c);
        tc = box > 0 && D <= 128 && rows > kMostRows;    // (TMEM holds two O tiles of 128 columns at most)
        if (!tc) box = std::min(box, fa::paged_rows_chunk(D));
        part.rows = tc ? 128 : fa::paged_rows_per_tile(D, rows);
        part.chunk = tc ? fa::kBlockKeys : fa::paged_rows_chunk(D);
        cut(nseq, c.Hkv, D, rows, keys, stacked, joined, tc ? 1 : fa::paged_rows_ctas_per_sm(D, part.rows));
    }

    // Over a 4-bit cache.
    Plan(int nseq, const fa_paged_kv4 &c, int64_t rows, int64_t keys)
    {
        tc = rows > kMostRows && c.D <= 128 && c.page_size % 8 == 0;
        part.rows = tc ? 128 : fa::four_rows_per_tile(c.D, rows);
        part.chunk = tc ? fa::kBlockKeys : fa::four_rows_chunk(c.D);
        cut(nseq, c.Hkv, c.D, rows, keys, false, false, tc ? 1 : fa::four_rows_ctas_per_sm(c.D, part.rows));
    }

    void cut(int nseq, int Hkv, int D, int64_t rows, int64_t keys, bool stacked, bool joined, int ctas_per_sm)
    {
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
        ctas = (int64_t)fa::sm_count_of(fa::current_device()) * ctas_per_sm;
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
inline int team_size(int D, const Plan &own, int64_t chunks, int (*at_once)(int device, int team))
{
    constexpr int kMostChunks = 8;
    if (D > 128 || own.part.rows != 8 || own.part.tiles != 1) return 0;
    const int device = fa::current_device();
    if (own.items > fa::sm_count_of(device)) return 0;
    int team = 0;
    for (int t = 1; t <= fa::kMostTeam && own.items <= at_once(device, t); t *= 2) {
        const int64_t each = (chunks + t * fa::kTeamWarps - 1) / (t * fa::kTeamWarps);
        if (each <= kMostChunks) team = t;
        if (each <= 1) break;
    }
    return team;
}

}  // namespace fa::paged
