// kv8_api.cu -- the C ABI of a step over an 8-bit cache and of beam search
// (include/qgemv.h): argument checks, launch shapes, launches.  Host code only.
#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "kv8_ops.h"

using namespace qg;

namespace {

constexpr int kMaxPage = 1 << 16;  // rows of a page of an 8-bit cache

qgemv_status check_cache8(const qgemv_kv8_cache *c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return QGEMV_ERR_INVALID_ARG;
    if (c->type != QGEMV_CODE_INT8 && c->type != QGEMV_CODE_E4M3) return QGEMV_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->page_size < 16 || c->page_size > kMaxPage ||
        (c->page_size & (c->page_size - 1)) || c->block_size < 16 || c->block_size > c->page_size ||
        (c->block_size & (c->block_size - 1)) || c->n_heads < 1 || c->n_heads > 4096 || c->head_dim < 16 ||
        c->head_dim > 256 || c->head_dim % 16)
        return QGEMV_ERR_INVALID_ARG;
    if (!extent_ok(c->n_pages, c->page_stride) || !extent_ok(c->page_size, c->row_stride) ||
        !extent_ok(c->n_heads, c->head_stride) || !extent_ok(c->n_pages, c->scale_page_stride) ||
        !extent_ok(c->page_size / c->block_size, c->scale_block_stride) || !extent_ok(c->n_heads, c->scale_head_stride))
        return QGEMV_ERR_INVALID_ARG;
    if ((c->n_pages > 1 && c->page_stride == 0) || c->row_stride == 0 || (c->n_heads > 1 && c->head_stride == 0))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % 16 || c->row_stride % 16 || c->head_stride % 16 ||
        !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return QGEMV_ERR_MISALIGNED;
    return QGEMV_OK;
}

inline Span codes_span(const qgemv_kv8_cache *c, const void *base)
{
    return span(base, (c->n_pages - 1) * c->page_stride + (c->page_size - 1) * c->row_stride +
                          (c->n_heads - 1) * c->head_stride + c->head_dim);
}
inline Span scale_span(const qgemv_kv8_cache *c, const void *base)
{
    return span(base, 4 * ((c->n_pages - 1) * c->scale_page_stride +
                           (c->page_size / c->block_size - 1) * c->scale_block_stride +
                           (c->n_heads - 1) * c->scale_head_stride + 1));
}
// Whether each block and head has scales of its own, as a call that writes them needs (a read of one
// scale for several is well).
inline bool own_scales(const qgemv_kv8_cache *c)
{
    return (c->n_pages == 1 || c->scale_page_stride) && (c->page_size == c->block_size || c->scale_block_stride) &&
           (c->n_heads == 1 || c->scale_head_stride);
}
// Whether two arrays of one shape, the second `delta` bytes behind the first, share bytes: n[i] places
// at each of three strides s[i], falling, of `width` bytes each.  Arrays that interleave (k and v by pages, rows or
// heads of one buffer) do not; one whose strides do not nest counts as if it did wherever it may.
bool places_meet(long long delta, const long long (&n)[3], const long long (&s)[3], long long width, int i = 0)
{
    if (i == 3) return delta < width && -delta < width;
    if (n[i] == 1) return places_meet(delta, n, s, width, i + 1);
    long long inner = width;  // that one step of this stride reaches over
    for (int j = i + 1; j < 3; ++j) inner += (n[j] - 1) * s[j];
    const auto floor_div = [](long long a, long long b) { return a / b - (a % b < 0); };
    const long long lo = std::max(1 - n[i], floor_div(delta - inner, s[i]) + 1), hi = std::min(n[i] - 1, floor_div(delta + inner - 1, s[i]));
    if (hi - lo > 2) return true;
    for (long long k = lo; k <= hi; ++k)
        if (places_meet(delta - k * s[i], n, s, width, i + 1)) return true;
    return false;
}
bool arrays_meet(const void *a, const void *b, long long (&&n)[3], long long (&&s)[3], long long width)
{
    for (int i = 0; i < 2; ++i)
        for (int j = 2; j > i; --j)
            if (s[j] > s[j - 1]) std::swap(s[j], s[j - 1]), std::swap(n[j], n[j - 1]);
    return places_meet(static_cast<long long>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)), n, s, width);
}
// The four arrays of a cache lie apart; codes and scales in one buffer by whole pages.
bool arrays_apart(const qgemv_kv8_cache *c)
{
    const int blocks = c->page_size / c->block_size;
    if (overlap(codes_span(c, c->k), codes_span(c, c->v)) &&
        arrays_meet(c->k, c->v, {c->n_pages, c->page_size, c->n_heads}, {c->page_stride, c->row_stride, c->head_stride}, c->head_dim))
        return false;
    if (overlap(scale_span(c, c->k_scale), scale_span(c, c->v_scale)) &&
        arrays_meet(c->k_scale, c->v_scale, {c->n_pages, blocks, c->n_heads},
                    {4 * c->scale_page_stride, 4 * c->scale_block_stride, 4 * c->scale_head_stride}, 4))
        return false;
    for (const void *codes : {c->k, c->v})
        for (const float *scales : {c->k_scale, c->v_scale}) {
            const Rows a{codes, c->n_pages, c->page_stride, (c->page_size - 1) * c->row_stride + (c->n_heads - 1) * c->head_stride + c->head_dim};
            const Rows b{scales, c->n_pages, 4 * c->scale_page_stride,
                         4 * ((blocks - 1) * c->scale_block_stride + (c->n_heads - 1) * c->scale_head_stride + 1)};
            if (rows_overlap(a, b)) return false;
        }
    return true;
}

Kv8Layout layout_of(const qgemv_kv8_cache *c)
{
    Kv8Layout l;
    l.k = static_cast<uint8_t *>(c->k);
    l.v = static_cast<uint8_t *>(c->v);
    l.ks = c->k_scale;
    l.vs = c->v_scale;
    l.page_stride = c->page_stride;
    l.row_stride = c->row_stride;
    l.head_stride = c->head_stride;
    l.scale_page = c->scale_page_stride;
    l.scale_block = c->scale_block_stride;
    l.scale_head = c->scale_head_stride;
    l.n_pages = c->n_pages;
    l.page_shift = log2_of(c->page_size);
    l.block_shift = log2_of(c->block_size);
    return l;
}

// What append and attention ask of a batch.
qgemv_status check_batch8(const qgemv_kv8_batch *b, const qgemv_kv8_cache *c)
{
    if (!b) return QGEMV_ERR_INVALID_ARG;
    const qgemv_status s = check_cache8(c);
    if (s != QGEMV_OK) return s;
    if (b->n_seqs < 1 || b->n_seqs > (1 << 20) || b->n_q < 1 || b->n_q > 8 || b->max_len < 0 || b->max_len > (1 << 30))
        return QGEMV_ERR_INVALID_ARG;
    return QGEMV_OK;
}
qgemv_status check_attn8(const qgemv_kv8_batch *b, const qgemv_kv8_cache *c)
{
    const qgemv_status s = check_batch8(b, c);
    if (s != QGEMV_OK) return s;
    if (b->n_q_heads < 1 || b->n_q_heads > 4096 || b->n_q_heads % c->n_heads || b->window < 0 || b->window > (1 << 30) ||
        b->sinks < 0 || b->sinks > (1 << 30))
        return QGEMV_ERR_INVALID_ARG;
    if (static_cast<long long>(b->n_seqs) * b->n_q * b->n_q_heads > (1ll << 27)) return QGEMV_ERR_INVALID_ARG;
    if (!(b->scale >= 0.0f) || std::isinf(b->scale)) return QGEMV_ERR_INVALID_ARG;
    // the strides of a tensor map end there
    constexpr long long kMapStride = 1ll << 40;
    if (c->page_stride >= kMapStride || c->row_stride >= kMapStride || c->head_stride >= kMapStride)
        return QGEMV_ERR_UNSUPPORTED;
    return QGEMV_OK;
}
// The tables' entries that lengths may reach.
inline Span table_span(const qgemv_kv8_batch *b, const qgemv_kv8_cache *c)
{
    const long long own = ceil_div(b->max_len, c->page_size);
    return own ? strided(b->pages, b->n_seqs, b->pages_stride, own, 4) : Span{0, 0};
}

// Launch shape and workspace of the attention.
struct Kv8Plan {
    int group, rows, row_tiles, tile_rows, tile_pad;
    int balanced, ranges, grid, combine_lanes, by_unit, aligned, wide;
    long long ml_at, parts_at, ws_bytes;
};

qgemv_status plan_attn8(const qgemv_kv8_batch *b, const qgemv_kv8_cache *c, Kv8Plan &a)
{
    a.group = b->n_q_heads / c->n_heads;
    a.rows = b->n_q * a.group;
    a.row_tiles = static_cast<int>(ceil_div(a.rows, kv8_tile_rows(c->head_dim)));
    a.tile_rows = static_cast<int>(ceil_div(a.rows, a.row_tiles));
    const int nt = static_cast<int>(ceil_div(a.tile_rows, 8));
    a.tile_pad = 8 * nt;
    const long long units = static_cast<long long>(b->n_seqs) * c->n_heads * a.row_tiles;
    const long long all = ceil_div(b->max_len, KV8_KEYS);
    long long tiles = all;  // of a unit at most
    if (b->window)
        tiles = std::min(tiles, ceil_div(b->sinks, KV8_KEYS) + ceil_div(b->window + b->n_q - 1, KV8_KEYS) + 1);
    // A unit that has a multiprocessor to itself takes all its warps: a warp's time for a tile is
    // mostly waiting (2 sequences of 700 keys, 2 cache heads: 7.0 us instead of 8.1; of 200: 4.6
    // instead of 5.4; of 16: 4.2 instead of 3.9).
    const int warps1 = kv8_warps(c->head_dim, nt), blocks1 = kv8_blocks(c->head_dim, nt);
    const bool wide = blocks1 > 1 && units <= ATTN_SMS && tiles > warps1;
    // Balanced ranges cost a walk over all lengths, units cut in two and a second launch, as
    // much as three or four tiles of each warp: where full units leave less than that undone in the
    // last wave of blocks, each is a block.  Under a window of up to half of max_len most are as long
    // as one another; else this holds for 64 tiles at most, so that a long one among short ones
    // costs no more than ranges would.  32 + 8 heads of 128, window 4096 of 9000 .. 13000 keys, 8 / 16 / 20 / 32 / 38 / 48
    // sequences: 22.9 / 25.3 / 43.7 / 47.1 / 55.7 / 90.3 us with units, 18.1 / 30.7 / 36.1 / 50.3 / 61.4 /
    // 73.9 with ranges (idle 6.3 / 1.7 / 10.3 / 3.4 / 0 / 16 tiles a warp).  Without a window, max_len 2048,
    // 8 / 16 / 38 / 48 / 76 sequences of 2000 keys: 13.9 / 15.5 / 29.2 / 48.2 / 56.4 us with units, 14.9 / 19.6 /
    // 30.2 / 41.4 / 59.0 with ranges (idle 3.1 / 0.8 / 0 / 7.9 / 0).  How long the sequences are the rule cannot
    // see: 24 / 48 of 300 keys would take 6.7 / 11.8 as units there, and take 10.8 / 16.7 in ranges.  Units are
    // also those of very many sequences, which spread over the multiprocessors well enough by themselves.
    const long long slots = static_cast<long long>(ATTN_SMS) * (wide ? 1 : blocks1), warps = warps1 * (wide ? 2 : 1);
    const long long idle = ceil_div(units, slots) * slots - units;
    const bool even = (2 * tiles <= all || tiles <= 64) && 2 * idle * tiles <= 7 * slots * warps;
    a.balanced = !even && b->n_seqs <= 1024 && b->n_seqs * tiles < (1ll << 30);
    a.ml_at = a.parts_at = kCounterArea;
    a.ws_bytes = kCounterArea;
    a.combine_lanes = 1;
    a.by_unit = a.aligned = a.ranges = a.wide = 0;
    if (!a.balanced) {
        if (units > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;
        a.grid = static_cast<int>(units);
        a.wide = wide;
        return QGEMV_OK;
    }
    // the line of all sequences' tiles in ranges, a block for each range, cache head and tile of rows
    const long long per_seq = units / b->n_seqs, blocks = static_cast<long long>(ATTN_SMS) * blocks1;
    const long long ranges = std::min(std::max(1ll, blocks / per_seq), ceil_div(b->n_seqs * tiles, KV8_SPLIT_MIN) + b->n_seqs);
    if (ranges * per_seq > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;
    a.ranges = static_cast<int>(ranges);
    a.grid = static_cast<int>(ranges * per_seq);
    // parts of a sequence: about ranges / n_seqs, and of a long one up to ranges.  A group takes four at once.
    const long long parts = ranges / std::min<long long>(b->n_seqs, ranges);
    while (a.combine_lanes < 32 && 2 * a.combine_lanes < parts) a.combine_lanes *= 2;
    a.by_unit = units <= a.grid;
    a.aligned = 8ll * b->n_seqs <= ranges && b->n_seqs <= 32;
    a.ml_at = a.parts_at + 16ll * a.grid;
    const long long o_at = a.ml_at + 16ll * a.grid * a.tile_pad;
    a.ws_bytes = o_at + 8ll * a.grid * a.tile_pad * c->head_dim;
    return QGEMV_OK;
}

// Workspace of a beam step.
struct BeamPlan {
    int slice, slices;
    long long ml_at, part_at, ws_bytes;
};
bool plan_beam(const qgemv_beam_spec *s, BeamPlan &a)
{
    if (!s || s->n_groups < 1 || s->n_groups > (1 << 20) || s->n_beams < 1 || s->n_beams > 16 || s->n_best < 1 ||
        s->n_best > 32 || s->vocab < 1 || s->vocab > (1 << 26))
        return false;
    const long long rows = static_cast<long long>(std::min(s->n_groups, BEAM_GROUPS)) * s->n_beams;  // of a launch
    // a row may begin 7 elements into a 16-byte chunk
    a.slice = static_cast<int>(ceil_div(ceil_div(s->vocab + 7, beam_slices(rows, s->vocab)), 2048) * 2048);
    a.slices = static_cast<int>(ceil_div(s->vocab + 7, a.slice));
    a.ml_at = kCounterArea;
    a.part_at = a.ml_at + 8ll * rows * a.slices;
    a.ws_bytes = (a.part_at + 8ll * rows * a.slices * s->n_best + 15) / 16 * 16;
    return true;
}

}  // namespace

extern "C" {

// ------------------------------------------------------- norm and rotation

qgemv_status qgemv_norm_rope_kv(const qgemv_rope_plan *plan, const qgemv_qk_norm *norm, const void *q, const void *k,
                                const void *v, qgemv_dtype in_type, int64_t q_stride, int64_t k_stride,
                                int64_t v_stride, const int32_t *pos, const int32_t *slots, int64_t n_tokens,
                                int n_q_heads, int n_k_heads, int head_dim, void *q_out, qgemv_dtype q_type,
                                int64_t q_out_stride, void *k_out, qgemv_dtype k_type, int64_t k_out_stride,
                                const qgemv_kv_cache *cache, qgemv_stream_t stream)
{
    if (!plan || !norm || !pos || (!q && !k) || !type_ok(in_type) || (q && !type_ok(q_type)) ||
        (k && !cache && !type_ok(k_type)))
        return QGEMV_ERR_INVALID_ARG;
    const int rot = plan->rot_dim;
    if (rot < 2 || rot > 256 || rot % 2 || (plan->layout != QGEMV_ROPE_HALF && plan->layout != QGEMV_ROPE_INTERLEAVED))
        return QGEMV_ERR_INVALID_ARG;
    if (n_tokens < 1 || n_tokens > INT32_MAX || head_dim < 2 || head_dim > 256 || head_dim % 2 || rot > head_dim)
        return QGEMV_ERR_INVALID_ARG;
    if (!(norm->eps > 0.0f) || !std::isfinite(norm->eps) || (q && !norm->q_weight) || (k && !norm->k_weight))
        return QGEMV_ERR_INVALID_ARG;
    if (k && (n_k_heads < 1 || n_k_heads > 4096 || (cache ? !v || !slots : !k_out))) return QGEMV_ERR_INVALID_ARG;
    if (q && (!q_out || n_q_heads < 1 || n_q_heads > 4096)) return QGEMV_ERR_INVALID_ARG;
    const int ib = type_bytes(in_type), qb = type_bytes(q_type), kb = type_bytes(k_type);
    const long long qw = q ? static_cast<long long>(n_q_heads) * head_dim : 0;
    const long long kw = k ? static_cast<long long>(n_k_heads) * head_dim : 0;
    const bool to_cache = k && cache, to_k = k && !cache;
    if (q && (!extent_ok(n_tokens, q_stride) || !extent_ok(n_tokens, q_out_stride) ||
              (n_tokens > 1 && (q_stride < qw || q_out_stride < qw))))
        return QGEMV_ERR_INVALID_ARG;
    if (k && !extent_ok(n_tokens, k_stride)) return QGEMV_ERR_INVALID_ARG;
    if (to_cache && !extent_ok(n_tokens, v_stride)) return QGEMV_ERR_INVALID_ARG;
    if (to_k && (!extent_ok(n_tokens, k_out_stride) || (n_tokens > 1 && k_out_stride < kw))) return QGEMV_ERR_INVALID_ARG;
    if (to_cache) {
        const qgemv_status s = check_cache(cache);
        if (s != QGEMV_OK) return s;
        if (cache->head_dim != head_dim || cache->n_heads != n_k_heads || cache->n_pages * cache->page_size > INT32_MAX)
            return QGEMV_ERR_INVALID_ARG;
    }
    if ((q && (!aligned(q, ib) || !aligned(q_out, qb))) || (k && !aligned(k, ib)) || (to_k && !aligned(k_out, kb)) ||
        (to_cache && (!aligned(v, ib) || !aligned(slots, 4))) || !aligned(pos, 4) ||
        (q && !aligned(norm->q_weight, 4)) || (k && !aligned(norm->k_weight, 4)))
        return QGEMV_ERR_MISALIGNED;

    // What is written lies apart from what is read, but for q rotated in place;
    // rows of one buffer may interleave.
    const Rows rq{q, n_tokens, q_stride * ib, qw * ib}, rk{k, n_tokens, k_stride * ib, kw * ib};
    const Rows rv{v, n_tokens, v_stride * ib, kw * ib};
    const Span sp = span(pos, 4 * n_tokens);
    const Span wq = span(norm->q_weight, q ? 4ll * head_dim : 0), wk = span(norm->k_weight, k ? 4ll * head_dim : 0);
    const Span ss = span(slots, to_cache ? 4 * n_tokens : 0);
    const auto all = [](const Rows &r) { return span(r.p, (r.n - 1) * r.stride + r.width); };
    const Rows oq{q_out, n_tokens, q_out_stride * qb, qw * qb}, ok{k_out, n_tokens, k_out_stride * kb, kw * kb};
    if (q) {
        const bool in_place = q_out == q && q_type == in_type && (q_out_stride == q_stride || n_tokens == 1);
        if (!in_place && rows_overlap(oq, rq)) return QGEMV_ERR_INVALID_ARG;
        if ((k && rows_overlap(oq, rk)) || (to_cache && rows_overlap(oq, rv))) return QGEMV_ERR_INVALID_ARG;
        for (const Span in : {sp, wq, wk, ss})
            if (overlap(all(oq), in)) return QGEMV_ERR_INVALID_ARG;
    }
    if (to_k) {
        if (rows_overlap(ok, rk) || (q && (rows_overlap(ok, rq) || rows_overlap(ok, oq)))) return QGEMV_ERR_INVALID_ARG;
        for (const Span in : {sp, wq, wk})
            if (overlap(all(ok), in)) return QGEMV_ERR_INVALID_ARG;
    }
    if (to_cache) {
        for (const Span out : {cache_span(cache, cache->k), cache_span(cache, cache->v)}) {
            for (const Span in : {all(rk), all(rv), sp, wq, wk, ss})
                if (overlap(out, in)) return QGEMV_ERR_INVALID_ARG;
            if (q && (overlap(out, all(rq)) || overlap(out, all(oq)))) return QGEMV_ERR_INVALID_ARG;
        }
    }

    NormRopeParams p = {};
    p.q_weight = norm->q_weight;
    p.k_weight = norm->k_weight;
    p.eps = norm->eps;
    RopeParams &r = p.r;
    r.q = q;
    r.k = k;
    r.v = v;
    r.q_stride = q_stride;
    r.k_stride = k_stride;
    r.v_stride = v_stride;
    r.pos = pos;
    r.q_out = q_out;
    r.q_out_stride = q_out_stride;
    r.hq = q ? n_q_heads : 0;
    r.hkv = k ? n_k_heads : 0;
    r.d = head_dim;
    r.rot = rot;
    r.mscale = plan->mscale;
    for (int i = 0; i < 128; ++i) r.turns[i] = plan->turns[i];
    bool vec = head_dim % 8 == 0 && rot % 8 == 0;
    const auto fits16 = [](const void *a, long long stride, int bytes) { return aligned(a, 16) && stride * bytes % 16 == 0; };
    if (q) vec = vec && fits16(q, q_stride, ib) && fits16(q_out, q_out_stride, qb);
    if (k) vec = vec && fits16(k, k_stride, ib);
    if (to_cache) {
        p.v_heads = n_k_heads;
        r.slots = slots;
        r.ck = cache->k;
        r.cv = cache->v;
        r.page_stride = cache->page_stride;
        r.row_stride = cache->row_stride;
        r.head_stride = cache->head_stride;
        r.n_slots = cache->n_pages * cache->page_size;
        r.page_shift = log2_of(cache->page_size);
        vec = vec && fits16(v, v_stride, ib);
    } else if (to_k) {
        r.ck = k_out;
        r.row_stride = k_out_stride;
        r.head_stride = head_dim;
        vec = vec && fits16(k_out, k_out_stride, kb);
    }
    int sms = 0;
    const qgemv_status s = device_props(&sms, &r.status);
    if (s != QGEMV_OK) return s;
    return launch_norm_rope(p, in_type, q ? q_type : QGEMV_F32, to_cache ? cache->type : to_k ? k_type : QGEMV_BF16,
                            plan->layout == QGEMV_ROPE_HALF, vec,
                            n_tokens, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_ERR_CUDA;
}

// ------------------------------------------------------------ 8-bit cache

qgemv_status qgemv_kv8_append(const void *k, const void *v, qgemv_dtype in_type, int64_t k_stride, int64_t v_stride,
                              int64_t n_tokens, const qgemv_kv8_cache *cache, const qgemv_kv8_batch *batch,
                              const int32_t *first, int max_new, qgemv_stream_t stream)
{
    qgemv_status s = check_batch8(batch, cache);
    if (s != QGEMV_OK) return s;
    const qgemv_kv8_batch &b = *batch;
    if (!b.lens || (b.max_len > 0 && !b.pages) || b.pages_stride < 0 || !extent_ok(b.n_seqs, b.pages_stride) ||
        !type_ok(in_type) || n_tokens < 0 || n_tokens > INT32_MAX || max_new < 0 || max_new > (1 << 30))
        return QGEMV_ERR_INVALID_ARG;
    if (!first && (n_tokens != static_cast<long long>(b.n_seqs) * b.n_q || max_new < b.n_q)) return QGEMV_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!k || !v)) return QGEMV_ERR_INVALID_ARG;
    if (!extent_ok(n_tokens, k_stride) || !extent_ok(n_tokens, v_stride) || !own_scales(cache) || !arrays_apart(cache))
        return QGEMV_ERR_INVALID_ARG;
    const int ib = type_bytes(in_type), d = cache->head_dim;
    if (!aligned(k, ib) || !aligned(v, ib) || !aligned(b.lens, 4) || !aligned(b.pages, 4) || !aligned(first, 4))
        return QGEMV_ERR_MISALIGNED;
    const long long w = static_cast<long long>(cache->n_heads) * d;
    if (n_tokens > 0)
        for (const Span in : {strided(k, n_tokens, k_stride, w, ib), strided(v, n_tokens, v_stride, w, ib),
                              span(b.lens, 4ll * b.n_seqs), table_span(&b, cache), span(first, first ? 4ll * (b.n_seqs + 1) : 0)})
            for (const Span out : {codes_span(cache, cache->k), codes_span(cache, cache->v),
                                   scale_span(cache, cache->k_scale), scale_span(cache, cache->v_scale)})
                if (overlap(in, out)) return QGEMV_ERR_INVALID_ARG;
    const int most = static_cast<int>(std::min<long long>(std::min<long long>(max_new, n_tokens), b.max_len));
    if (n_tokens == 0 || max_new == 0) return QGEMV_OK;
    if (n_tokens == 1) k_stride = v_stride = 0;
    if (k_stride > INT32_MAX || v_stride > INT32_MAX || cache->row_stride > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;

    Kv8AppendParams p = {};
    p.c = layout_of(cache);
    p.k = k;
    p.v = v;
    p.k_stride = static_cast<int>(k_stride);
    p.v_stride = static_cast<int>(v_stride);
    p.code_row = static_cast<int>(cache->row_stride);
    p.n_tokens = n_tokens;
    p.first = first;
    p.lens = b.lens;
    p.pages = b.pages;
    p.pages_stride = b.pages_stride;
    p.n_new = b.n_q;
    p.max_new = max_new;
    p.max_len = b.max_len;
    // one block at least, so that a length or token out of its bounds is recorded
    p.blocks = std::max(1, (most + 2 * cache->block_size - 2) / cache->block_size);
    p.n_seqs = b.n_seqs;
    p.hkv = cache->n_heads;
    p.d = d;
    p.pieces = d / 8;
    if (static_cast<long long>(p.n_seqs) * p.blocks > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;
    const bool vec = aligned(k, 16) && aligned(v, 16) && k_stride * ib % 16 == 0 && v_stride * ib % 16 == 0;
    int sms = 0;
    s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    return launch_kv8_append(p, in_type, cache->type, vec, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_ERR_CUDA;
}

size_t qgemv_attn_kv8_workspace_bytes(const qgemv_kv8_batch *batch, const qgemv_kv8_cache *cache)
{
    Kv8Plan a;
    if (check_attn8(batch, cache) != QGEMV_OK || plan_attn8(batch, cache, a) != QGEMV_OK) return 0;
    return static_cast<size_t>(a.ws_bytes);
}

qgemv_status qgemv_attn_kv8(const void *q, qgemv_dtype q_type, int64_t q_token_stride, int64_t q_head_stride,
                            const qgemv_kv8_cache *cache, const qgemv_kv8_batch *batch, void *o, qgemv_dtype o_type,
                            int64_t o_token_stride, int64_t o_head_stride, float *lse_or_null, void *ws,
                            size_t ws_bytes, qgemv_stream_t stream)
{
    qgemv_status s = check_attn8(batch, cache);
    if (s != QGEMV_OK) return s;
    const qgemv_kv8_batch &b = *batch;
    if (!q || !o || !b.lens || (b.max_len > 0 && !b.pages) || b.pages_stride < 0 ||
        (q_type != QGEMV_F16 && q_type != QGEMV_BF16) || (o_type != QGEMV_F32 && o_type != q_type))
        return QGEMV_ERR_INVALID_ARG;
    const long long tokens = static_cast<long long>(b.n_seqs) * b.n_q;
    const int d = cache->head_dim, ob = type_bytes(o_type);
    if (!extent_ok(tokens, q_token_stride) || !extent_ok(b.n_q_heads, q_head_stride) ||
        !extent_ok(tokens, o_token_stride) || !extent_ok(b.n_q_heads, o_head_stride) ||
        !extent_ok(b.n_seqs, b.pages_stride) || !pieces_apart(tokens, o_token_stride, b.n_q_heads, o_head_stride, d))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 || !aligned(o, ob) || !aligned(b.lens, 4) ||
        !aligned(b.pages, 4) || !aligned(lse_or_null, 4))
        return QGEMV_ERR_MISALIGNED;
    Kv8Plan a;
    s = plan_attn8(batch, cache, a);
    if (s != QGEMV_OK) return s;
    if (!ws || ws_bytes < static_cast<size_t>(a.ws_bytes)) return QGEMV_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return QGEMV_ERR_MISALIGNED;
    const long long heads1 = b.n_q_heads - 1;
    const Span so = span(o, ((tokens - 1) * o_token_stride + heads1 * o_head_stride + d) * ob);
    const Span se = span(lse_or_null, lse_or_null ? 4 * tokens * b.n_q_heads : 0);
    const Span sw = span(ws, a.ws_bytes);
    for (const Span out : {so, se, sw})
        for (const Span in : {span(q, ((tokens - 1) * q_token_stride + heads1 * q_head_stride + d) * 2),
                              codes_span(cache, cache->k), codes_span(cache, cache->v), scale_span(cache, cache->k_scale),
                              scale_span(cache, cache->v_scale), span(b.lens, 4ll * b.n_seqs), table_span(&b, cache)})
            if (overlap(out, in)) return QGEMV_ERR_INVALID_ARG;
    if (overlap(so, se) || overlap(so, sw) || overlap(se, sw)) return QGEMV_ERR_INVALID_ARG;

    Kv8AttnParams p = {};
    p.c = layout_of(cache);
    p.q = q;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.q_bf16 = q_type == QGEMV_BF16;
    p.lens = b.lens;
    p.pages = b.pages;
    p.pages_stride = b.pages_stride;
    p.n_seqs = b.n_seqs;
    p.n_q = b.n_q;
    p.hq = b.n_q_heads;
    p.hkv = cache->n_heads;
    p.group = a.group;
    p.per_group = 1.0f / static_cast<float>(a.group);
    p.d = d;
    p.max_len = b.max_len;
    p.window = b.window;
    p.sinks = b.sinks;
    p.rows = a.rows;
    p.row_tiles = a.row_tiles;
    p.tile_rows = a.tile_rows;
    const double scale = b.scale != 0.0f ? b.scale : 1.0 / std::sqrt(static_cast<double>(d));
    p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    p.balanced = a.balanced;
    p.ranges = a.ranges;
    p.grid = a.grid;
    p.combine_lanes = a.combine_lanes;
    p.parts_by_unit = a.by_unit;
    p.aligned = a.aligned;
    p.wide = a.wide;
    uint8_t *at = static_cast<uint8_t *>(ws);
    p.parts = reinterpret_cast<int4 *>(at + a.parts_at);
    p.part_ml = reinterpret_cast<float2 *>(at + a.ml_at);
    p.part_o = reinterpret_cast<float *>(at + a.ml_at + 16ll * a.grid * a.tile_pad);
    p.o = o;
    p.o_type = o_type;
    p.o_token_stride = o_token_stride;
    p.o_head_stride = o_head_stride;
    p.lse = lse_or_null;
    int sms = 0;
    s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    const auto launch = cache->type == QGEMV_CODE_INT8 ? launch_kv8_attn_int8 : launch_kv8_attn_e4m3;
    return launch(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QGEMV_OK : QGEMV_ERR_CUDA;
}

// ------------------------------------------------------------------- beams

size_t qgemv_beam_workspace_bytes(const qgemv_beam_spec *spec)
{
    BeamPlan a;
    return plan_beam(spec, a) ? static_cast<size_t>(a.ws_bytes) : 0;
}

qgemv_status qgemv_beam_select(const void *logits, qgemv_dtype type, int64_t x_stride, const qgemv_beam_spec *spec,
                               float *score, int64_t *token, int32_t *parent, void *ws, size_t ws_bytes,
                               qgemv_stream_t stream)
{
    BeamPlan a;
    if (!plan_beam(spec, a) || !logits || !type_ok(type) || !spec->scores || !score || !token || !parent)
        return QGEMV_ERR_INVALID_ARG;
    const qgemv_beam_spec &c = *spec;
    const long long rows = static_cast<long long>(c.n_groups) * c.n_beams, outs = static_cast<long long>(c.n_groups) * c.n_best;
    const int eb = type_bytes(type);
    if (!extent_ok(rows, x_stride) || (rows > 1 && x_stride < c.vocab)) return QGEMV_ERR_INVALID_ARG;
    if (!ws || ws_bytes < static_cast<size_t>(a.ws_bytes)) return QGEMV_ERR_WORKSPACE;
    if (!aligned(logits, eb) || !aligned(c.scores, 4) || !aligned(c.done, 4) || !aligned(score, 4) || !aligned(token, 8) ||
        !aligned(parent, 4) || !aligned(ws, 16))
        return QGEMV_ERR_MISALIGNED;
    const Span out[4] = {span(score, 4 * outs), span(token, 8 * outs), span(parent, 4 * outs), span(ws, a.ws_bytes)};
    for (int i = 0; i < 4; ++i) {
        for (const Span in : {strided(logits, rows, x_stride, c.vocab, eb), span(c.scores, 4 * rows),
                              span(c.done, c.done ? 4 * rows : 0)})
            if (overlap(out[i], in)) return QGEMV_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j])) return QGEMV_ERR_INVALID_ARG;
    }

    BeamParams p = {};
    p.x_stride = x_stride;
    p.vocab = c.vocab;
    p.beams = c.n_beams;
    p.n_best = c.n_best;
    p.slice = a.slice;
    p.slices = a.slices;
    p.cnt = static_cast<unsigned *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + a.ml_at);
    p.part = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(ws) + a.part_at);
    for (int g = 0; g < c.n_groups; g += BEAM_GROUPS) {
        const long long r = static_cast<long long>(g) * c.n_beams, o = static_cast<long long>(g) * c.n_best;
        p.x = static_cast<const uint8_t *>(logits) + r * x_stride * eb;
        p.scores = c.scores + r;
        p.done = c.done ? c.done + r : nullptr;
        p.score = score + o;
        p.token = reinterpret_cast<long long *>(token) + o;
        p.parent = parent + o;
        p.row0 = static_cast<int>(r);
        if (launch_beam(p, type, std::min(BEAM_GROUPS, c.n_groups - g), reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
            return QGEMV_ERR_CUDA;
    }
    return QGEMV_OK;
}

// ------------------------------------------------------------------- pages

qgemv_status qgemv_fork_pages(const qgemv_fork *fork, const qgemv_kv_cache *caches, const qgemv_kv8_cache *caches8,
                              int n_caches, qgemv_stream_t stream)
{
    if (!fork || !caches == !caches8 || n_caches < 1 || n_caches > (1 << 16)) return QGEMV_ERR_INVALID_ARG;
    const qgemv_fork &f = *fork;
    if (f.n_in < 1 || f.n_in > (1 << 20) || f.n_out < 1 || f.n_out > (1 << 20) || f.n_columns < 1 || !f.parents || !f.lens ||
        !f.pages || !f.fresh || !f.pages_out || !f.lens_out || !extent_ok(f.n_in, f.pages_stride) ||
        !extent_ok(f.n_out, f.out_stride) || (f.n_in > 1 && f.pages_stride < f.n_columns) ||
        (f.n_out > 1 && f.out_stride < f.n_columns))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(f.parents, 4) || !aligned(f.lens, 4) || !aligned(f.pages, 4) || !aligned(f.fresh, 4) ||
        !aligned(f.pages_out, 4) || !aligned(f.lens_out, 4))
        return QGEMV_ERR_MISALIGNED;
    const Span in[4] = {span(f.parents, 4ll * f.n_out), span(f.lens, 4ll * f.n_in),
                        strided(f.pages, f.n_in, f.pages_stride, f.n_columns, 4), span(f.fresh, 4ll * f.n_out)};
    const Span out[2] = {strided(f.pages_out, f.n_out, f.out_stride, f.n_columns, 4), span(f.lens_out, 4ll * f.n_out)};
    if (overlap(out[0], out[1])) return QGEMV_ERR_INVALID_ARG;
    const auto clear_of = [&](Span s) {
        for (const Span t : in)
            if (overlap(s, t)) return false;
        return !overlap(s, out[0]) && !overlap(s, out[1]);
    };
    for (const Span o : out)
        for (const Span t : in)
            if (overlap(o, t)) return QGEMV_ERR_INVALID_ARG;
    long long n_pages = 0;
    int page_size = 0, block_size = 0, heads = 0, head_dim = 0, type = 0;
    for (int i = 0; i < n_caches; ++i) {
        const qgemv_status s = caches ? check_cache(caches + i) : check_cache8(caches8 + i);
        if (s != QGEMV_OK) return s;
        if (!caches && !own_scales(caches8 + i)) return QGEMV_ERR_INVALID_ARG;
        const long long pages = caches ? caches[i].n_pages : caches8[i].n_pages;
        const int shape[5] = {caches ? caches[i].page_size : caches8[i].page_size, caches ? 0 : caches8[i].block_size,
                              caches ? caches[i].n_heads : caches8[i].n_heads,
                              caches ? caches[i].head_dim : caches8[i].head_dim,
                              caches ? static_cast<int>(caches[i].type) : static_cast<int>(caches8[i].type)};
        if (i == 0) n_pages = pages, page_size = shape[0], block_size = shape[1], heads = shape[2], head_dim = shape[3], type = shape[4];
        if (pages != n_pages || shape[0] != page_size || shape[1] != block_size || shape[2] != heads || shape[3] != head_dim ||
            shape[4] != type)
            return QGEMV_ERR_INVALID_ARG;
        if (caches ? !clear_of(cache_span(caches + i, caches[i].k)) || !clear_of(cache_span(caches + i, caches[i].v))
                   : !clear_of(codes_span(caches8 + i, caches8[i].k)) || !clear_of(codes_span(caches8 + i, caches8[i].v)) ||
                         !clear_of(scale_span(caches8 + i, caches8[i].k_scale)) ||
                         !clear_of(scale_span(caches8 + i, caches8[i].v_scale)))
            return QGEMV_ERR_INVALID_ARG;
    }
    if (page_size > kMaxPage || static_cast<long long>(f.n_columns) * page_size > INT32_MAX) return QGEMV_ERR_INVALID_ARG;

    ForkParams p = {};
    p.f = f;
    p.page_shift = log2_of(page_size);
    p.block_shift = caches ? -1 : log2_of(block_size);
    p.heads = heads;
    p.head_bytes = head_dim * (caches ? 2 : 1);
    p.n_pages = n_pages;
    // 16-byte pieces of a page's rows are counted in 32 bits
    if (static_cast<long long>(page_size) * heads * (p.head_bytes / 16) > INT32_MAX / 2) return QGEMV_ERR_UNSUPPORTED;
    int sms = 0;
    const qgemv_status s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    for (int i0 = 0; i0 < n_caches; i0 += FORK_CACHES) {
        const int n = std::min(FORK_CACHES, n_caches - i0);
        p.n_arrays = 2 * n;
        p.first = i0 == 0;
        for (int i = 0; i < n; ++i) {
            const qgemv_kv_cache *c = caches ? caches + i0 + i : nullptr;
            const qgemv_kv8_cache *e = caches ? nullptr : caches8 + i0 + i;
            p.page_stride[i] = c ? 2 * c->page_stride : e->page_stride;
            p.row_stride[i] = c ? 2 * c->row_stride : e->row_stride;
            p.head_stride[i] = c ? 2 * c->head_stride : e->head_stride;
            p.base[2 * i] = c ? c->k : e->k;
            p.base[2 * i + 1] = c ? c->v : e->v;
            if (!e) continue;
            p.scale[2 * i] = e->k_scale;
            p.scale[2 * i + 1] = e->v_scale;
            p.scale_page[i] = e->scale_page_stride;
            p.scale_block[i] = e->scale_block_stride;
            p.scale_head[i] = e->scale_head_stride;
        }
        if (launch_fork(p, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return QGEMV_ERR_CUDA;
    }
    return QGEMV_OK;
}

}  // extern "C"
