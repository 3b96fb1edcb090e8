// decode_api.cu -- the C ABI of the decode step's operators between its
// GEMVs (include/qgemv.h): argument checks, launch shapes, launches.  Host
// code only.
#include <algorithm>
#include <cmath>

#include "decode_ops.h"

using namespace qg;

namespace {

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

struct Span {
    uintptr_t lo, hi;
};
inline Span span(const void *p, long long bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

inline bool type_ok(int t) { return t == QGEMV_F32 || t == QGEMV_F16 || t == QGEMV_BF16; }
inline int type_bytes(qgemv_dtype t) { return t == QGEMV_F32 ? 4 : 2; }

// From an address to the end of the last of `n` pieces of `last` elements,
// `stride` elements apart.
inline Span strided(const void *p, long long n, long long stride, long long last, int bytes)
{
    return span(p, ((n - 1) * stride + last) * bytes);
}

// n rows of `width` bytes, `stride` bytes apart.
struct Rows {
    const void *p;
    long long n, stride, width;
};

// Whether two sets of rows share bytes.  Parts of one row buffer interleave.
bool rows_overlap(const Rows &a, const Rows &b)
{
    const auto all = [](const Rows &r) { return span(r.p, (r.n - 1) * r.stride + r.width); };
    if (!overlap(all(a), all(b))) return false;
    // row u of b begins b0 + u * b.stride after row 0 of a
    const long long b0 = static_cast<long long>(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    // whether a row at `at` meets one of the rows first + i * stride, 0 <= i < n: the first that ends behind its begin
    const auto meets = [&](long long at, long long first, long long stride, long long n) {
        const long long i = at < first + b.width || !stride ? 0 : (at - first - b.width) / stride + 1;
        return i < n && first + i * stride < at + a.width && first + i * stride + b.width > at;
    };
    // of one stride: only the difference of the row numbers matters
    if (a.stride == b.stride) return meets(0, b0 - (a.n - 1) * b.stride, b.stride, a.n + b.n - 1);
    if (a.n > 65536) return true;  // not looked through
    for (long long t = 0; t < a.n; ++t)
        if (meets(t * a.stride, b0, b.stride, b.n)) return true;
    return false;
}

// Whether n1 x n2 pieces of d elements at i * s1 + j * s2 lie apart from one another.
inline bool pieces_apart(long long n1, long long s1, long long n2, long long s2, long long d)
{
    if ((n1 == 1 || s1 >= (n2 - 1) * s2 + d) && (n2 == 1 || s2 >= d)) return true;  // the usual orders
    if ((n2 == 1 || s2 >= (n1 - 1) * s1 + d) && (n1 == 1 || s1 >= d)) return true;
    if (n1 > 1 && s1 < d) return false;
    for (long long j = 1; j < n2; ++j) {  // a piece j steps along, against those nearest to it
        const long long at = j * s2, i = s1 ? std::min(at / s1, n1 - 1) : 0;
        if (at - i * s1 < d || (i + 1 < n1 && (i + 1) * s1 - at < d)) return false;
    }
    return true;
}

constexpr long long kMaxExtent = 1ll << 46;  // elements of a tensor: products of strides and counts stay in 64 bits

// A product of non-negative counts and strides that stays below kMaxExtent.
inline bool extent_ok(long long n, long long stride)
{
    return n >= 0 && stride >= 0 && (n == 0 || stride == 0 || n <= kMaxExtent / stride);
}

qgemv_status check_cache(const qgemv_kv_cache *c)
{
    if (!c || !c->k || !c->v) return QGEMV_ERR_INVALID_ARG;
    if (c->type != QGEMV_F16 && c->type != QGEMV_BF16) return QGEMV_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->page_size < 1 || (c->page_size & (c->page_size - 1)) ||
        c->n_heads < 1 || c->n_heads > 4096 || c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8)
        return QGEMV_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0) return QGEMV_ERR_INVALID_ARG;
    if (!extent_ok(c->n_pages, c->page_stride) || !extent_ok(c->page_size, c->row_stride) ||
        !extent_ok(c->n_heads, c->head_stride))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % 8 || c->row_stride % 8 || c->head_stride % 8)
        return QGEMV_ERR_MISALIGNED;
    return QGEMV_OK;
}

inline Span cache_span(const qgemv_kv_cache *c, const void *base)
{
    return span(base, 2 * ((c->n_pages - 1) * c->page_stride + (c->page_size - 1) * c->row_stride +
                           (c->n_heads - 1) * c->head_stride + c->head_dim));
}

inline int log2_of(int v)
{
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

// ------------------------------------------------------------- attention

// Launch shape and workspace of a batch.
struct AttnPlan {
    int rows, group;
    int p_tile, p_tiles, p_splits, p_keys;
    int s_tile, s_tiles, s_splits, s_keys;
    int t_mode, t_tiles, t_splits, t_keys, t_len, p_first;
    long long part_rows;  // partial rows: slots * heads * rows
    long long ws_bytes;
};
constexpr long long kCounterArea = 16384;  // the workspace's zero-kept head (include/qgemv.h), not touched here

qgemv_status check_batch(const qgemv_attn_batch *b, const qgemv_kv_cache *c)
{
    if (!b) return QGEMV_ERR_INVALID_ARG;
    const qgemv_status s = check_cache(c);
    if (s != QGEMV_OK) return s;
    if (b->n_seqs < 1 || b->n_seqs > (1 << 20) || b->n_q < 1 || b->n_q > 8 || b->n_q_heads < 1 || b->n_q_heads > 4096 ||
        b->n_q_heads % c->n_heads || b->prefix_len < 0 || b->prefix_len > (1 << 30) || b->max_suffix < 0 ||
        b->max_suffix > (1 << 30))
        return QGEMV_ERR_INVALID_ARG;
    if (static_cast<long long>(b->n_seqs) * b->n_q * b->n_q_heads > (1ll << 27)) return QGEMV_ERR_INVALID_ARG;
    if (!(b->scale >= 0.0f) || std::isinf(b->scale)) return QGEMV_ERR_INVALID_ARG;
    return QGEMV_OK;
}

// The split of a launch, for two blocks a multiprocessor.
qgemv_status plan_attn(const qgemv_attn_batch *b, const qgemv_kv_cache *c, AttnPlan &a)
{
    constexpr long long kSlots = 2 * ATTN_SMS;
    a.group = b->n_q_heads / c->n_heads;
    a.rows = b->n_seqs * b->n_q * a.group;
    a.p_tile = attn_tile_rows(a.rows, c->head_dim);
    a.p_tiles = static_cast<int>(ceil_div(a.rows, a.p_tile));
    // a suffix's rows that all its queries see
    const long long s_most = std::max(0, b->max_suffix - b->n_q + 1);
    const long long s_units = ceil_div(s_most, 64);
    const int per = b->n_q * a.group;
    a.s_tile = attn_tile_rows(per, c->head_dim);
    a.s_tiles = static_cast<int>(ceil_div(per, a.s_tile));
    const long long s_base = static_cast<long long>(b->n_seqs) * c->n_heads * a.s_tiles;

    // The tcgen05 kernel takes the whole tiles of 128 keys of the prefixes of
    // tall batches: a whole tile at least, more rows than one of the other
    // kernel's row tiles, and at least six of its tiles of 64 keys and rows per
    // slot (which a batch of 1824 row tiles has at 64 keys).  Measured (us a call,
    // tcgen05 / mma.sync; rows per cache head, cache heads, keys): 96 x 8: 18.5 /
    // 16.2 at 2048, 22.1 / 25.2 at 8192; 256 x 8: 21.8 / 23.5 at 2048, 47 / 114
    // at 32768; 128 x 2: 28 / 25 at 32768; 192 x 1: 19 / 15 there; 448 x 2, heads
    // of 64: 14.8 / 13.7 at 2048, 27 / 41 at 32768; 64 rows: never faster.
    // One block per multiprocessor, the split whose last wave ends first (a
    // block costs about two tiles before and after its own, and a part of 8192
    // rows, written and read again, about one).
    a.t_mode = a.t_tiles = a.t_splits = a.t_keys = a.t_len = a.p_first = 0;
    if (a.rows > 64 && b->prefix_len >= 128 &&
        static_cast<long long>(a.p_tiles) * c->n_heads * (b->prefix_len / 64) >= 6 * kSlots && attn_tc_takes(*c)) {
        a.t_mode = a.rows <= 128 ? 2 : 1;
        a.t_tiles = static_cast<int>(ceil_div(a.rows, 256));
        a.t_len = b->prefix_len / 128 * 128;
        const long long units = a.t_len / 128, base = static_cast<long long>(c->n_heads) * a.t_tiles;
        const int streams = a.t_mode == 2 ? 2 : 1;
        long long best = 1, best_cost = INT64_MAX;
        for (int waves = 1; waves <= 16; ++waves) {  // the most ranges whose blocks make so many waves
            const long long n = std::min(units, std::max(1ll, waves * static_cast<long long>(ATTN_SMS) / base));
            const long long each = ceil_div(units, n), ranges = ceil_div(units, each);
            const long long cost = ceil_div(base * ranges, ATTN_SMS) * (ceil_div(each, streams) + 2) * 8192 +
                                   ranges * streams * a.rows * c->n_heads;
            if (cost < best_cost) best_cost = cost, best = n;
        }
        a.t_keys = static_cast<int>(ceil_div(units, best) * 128);
        a.t_splits = static_cast<int>(ceil_div(a.t_len, a.t_keys));
        a.p_first = a.t_splits * streams;
        if (base * a.t_splits > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;
    }
    // ranges of the (rest of the) prefix: enough to fill the slots
    const long long rest = b->prefix_len - a.t_len, p_units = ceil_div(rest, 64);
    const long long p_base = static_cast<long long>(c->n_heads) * a.p_tiles;
    long long splits = std::min(std::max(1ll, p_units), std::max(1ll, kSlots / p_base));
    a.p_keys = static_cast<int>(p_units ? ceil_div(p_units, splits) * 64 : 64);
    a.p_splits = static_cast<int>(ceil_div(rest, a.p_keys));
    splits = std::min(std::max(1ll, s_units), std::max(ceil_div(s_units, 16), kSlots / s_base));
    a.s_keys = static_cast<int>(s_units ? ceil_div(s_units, splits) * 64 : 64);
    a.s_splits = static_cast<int>(ceil_div(s_most, a.s_keys));
    if (p_base * a.p_splits + s_base * a.s_splits > INT32_MAX) return QGEMV_ERR_UNSUPPORTED;
    a.part_rows = static_cast<long long>(a.p_first + a.p_splits + a.s_splits) * c->n_heads * a.rows;
    a.ws_bytes = kCounterArea + a.part_rows * (4ll * c->head_dim + 8);
    return QGEMV_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- rotary

qgemv_status qgemv_rope_init(const qgemv_rope_config *cfg, qgemv_rope_plan *plan)
{
    if (!cfg || !plan) return QGEMV_ERR_INVALID_ARG;
    const int rot = cfg->rot_dim, half = rot / 2;
    const int scaling = cfg->scaling, layout = cfg->layout;
    if (rot < 2 || rot > 256 || rot % 2 || scaling < QGEMV_ROPE_PLAIN || scaling > QGEMV_ROPE_YARN ||
        (layout != QGEMV_ROPE_HALF && layout != QGEMV_ROPE_INTERLEAVED))
        return QGEMV_ERR_INVALID_ARG;
    if (!(cfg->base > 1.0) || !std::isfinite(cfg->base) || !std::isfinite(cfg->mscale)) return QGEMV_ERR_INVALID_ARG;
    if (scaling != QGEMV_ROPE_PLAIN && (!(cfg->factor >= 1.0) || !std::isfinite(cfg->factor)))
        return QGEMV_ERR_INVALID_ARG;
    const bool ramps = scaling == QGEMV_ROPE_BANDS || scaling == QGEMV_ROPE_YARN;
    if (ramps && (!(cfg->orig_len > 0.0) || !std::isfinite(cfg->orig_len) || !(cfg->low > 0.0) ||
                  !(cfg->high > cfg->low) || !std::isfinite(cfg->high)))
        return QGEMV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    double a = 0.0, b = 1.0;
    if (scaling == QGEMV_ROPE_YARN) {
        const auto pair = [&](double turns) {
            return rot * std::log(cfg->orig_len / (turns * two_pi)) / (2.0 * std::log(cfg->base));
        };
        a = std::max(0.0, std::floor(pair(cfg->high)));
        b = std::min(rot - 1.0, std::ceil(pair(cfg->low)));
    }
    for (int i = 0; i < 128; ++i) plan->turns[i] = 0;
    for (int i = 0; i < half; ++i) {
        double t = std::pow(cfg->base, -2.0 * i / rot);
        if (scaling == QGEMV_ROPE_LINEAR) t /= cfg->factor;
        if (scaling == QGEMV_ROPE_BANDS) {
            const double s =
                std::min(1.0, std::max(0.0, (cfg->orig_len * t / two_pi - cfg->low) / (cfg->high - cfg->low)));
            t *= (1.0 - s) / cfg->factor + s;
        }
        if (scaling == QGEMV_ROPE_YARN) {
            const double w = std::min(1.0, std::max(0.0, (i - a) / std::max(b - a, 1e-3)));
            t = t * (1.0 - w) + t / cfg->factor * w;
        }
        // theta <= 1, so less than 2^62 units
        plan->turns[i] = static_cast<uint64_t>(std::llround(t / two_pi * 18446744073709551616.0));
    }
    const double by_type = scaling == QGEMV_ROPE_YARN ? 0.1 * std::log(cfg->factor) + 1.0 : 1.0;
    plan->mscale = static_cast<float>(cfg->mscale != 0.0 ? cfg->mscale : by_type);
    plan->rot_dim = rot;
    plan->layout = layout;
    return QGEMV_OK;
}

qgemv_status qgemv_rope_kv(const qgemv_rope_plan *plan, const void *q, const void *k, const void *v,
                           qgemv_dtype in_type, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           const int32_t *pos, const int32_t *slots, int64_t n_tokens, int n_q_heads, int head_dim,
                           void *q_out, qgemv_dtype q_type, int64_t q_out_stride, const qgemv_kv_cache *cache,
                           qgemv_stream_t stream)
{
    if (!plan || !pos || (!q && !k) || (!k != !v) || !type_ok(in_type)) return QGEMV_ERR_INVALID_ARG;
    const int rot = plan->rot_dim;
    if (rot < 2 || rot > 256 || rot % 2 || (plan->layout != QGEMV_ROPE_HALF && plan->layout != QGEMV_ROPE_INTERLEAVED))
        return QGEMV_ERR_INVALID_ARG;
    if (n_tokens < 1 || n_tokens > INT32_MAX || head_dim < 2 || head_dim > 1024 || head_dim % 2 || rot > head_dim)
        return QGEMV_ERR_INVALID_ARG;
    const int ib = type_bytes(in_type), qb = q ? type_bytes(q_type) : 1;
    long long hkv = 0;
    if (q) {
        if (!q_out || !type_ok(q_type) || n_q_heads < 1 || n_q_heads > 4096) return QGEMV_ERR_INVALID_ARG;
        const long long w = static_cast<long long>(n_q_heads) * head_dim;
        if (!extent_ok(n_tokens, q_stride) || !extent_ok(n_tokens, q_out_stride) ||
            (n_tokens > 1 && (q_stride < w || q_out_stride < w)))
            return QGEMV_ERR_INVALID_ARG;
        if (!aligned(q, ib) || !aligned(q_out, qb)) return QGEMV_ERR_MISALIGNED;
        const bool in_place = q_out == q && q_type == in_type && (q_out_stride == q_stride || n_tokens == 1);
        const Span so = strided(q_out, n_tokens, q_out_stride, w, qb);
        if (!in_place && rows_overlap(Rows{q_out, n_tokens, q_out_stride * qb, w * qb}, Rows{q, n_tokens, q_stride * ib, w * ib}))
            return QGEMV_ERR_INVALID_ARG;
        if (overlap(so, span(pos, 4 * n_tokens))) return QGEMV_ERR_INVALID_ARG;
    }
    if (k) {
        if (!slots) return QGEMV_ERR_INVALID_ARG;
        const qgemv_status s = check_cache(cache);
        if (s != QGEMV_OK) return s;
        if (cache->head_dim != head_dim || cache->n_pages * cache->page_size > INT32_MAX) return QGEMV_ERR_INVALID_ARG;
        hkv = cache->n_heads;
        const long long w = hkv * head_dim;
        if (!extent_ok(n_tokens, k_stride) || !extent_ok(n_tokens, v_stride)) return QGEMV_ERR_INVALID_ARG;
        if (!aligned(k, ib) || !aligned(v, ib) || !aligned(slots, 4)) return QGEMV_ERR_MISALIGNED;
        const Span sk = cache_span(cache, cache->k), sv = cache_span(cache, cache->v);
        for (const Span in : {strided(k, n_tokens, k_stride, w, ib), strided(v, n_tokens, v_stride, w, ib),
                              span(pos, 4 * n_tokens), span(slots, 4 * n_tokens)})
            if (overlap(in, sk) || overlap(in, sv)) return QGEMV_ERR_INVALID_ARG;
        if (q) {
            const long long qw = static_cast<long long>(n_q_heads) * head_dim;
            const Span sq = strided(q, n_tokens, q_stride, qw, ib), so = strided(q_out, n_tokens, q_out_stride, qw, qb);
            if (overlap(sq, sk) || overlap(sq, sv) || overlap(so, sk) || overlap(so, sv)) return QGEMV_ERR_INVALID_ARG;
            // also in place: a block may write a token's q before another reads its k and v
            const Rows ro{q_out, n_tokens, q_out_stride * qb, qw * qb};
            if (rows_overlap(ro, Rows{k, n_tokens, k_stride * ib, w * ib}) ||
                rows_overlap(ro, Rows{v, n_tokens, v_stride * ib, w * ib}))
                return QGEMV_ERR_INVALID_ARG;
            if (overlap(so, span(slots, 4 * n_tokens))) return QGEMV_ERR_INVALID_ARG;
        }
    }
    if (!aligned(pos, 4)) return QGEMV_ERR_MISALIGNED;

    RopeParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pos = pos;
    p.slots = slots;
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.hq = q ? n_q_heads : 0;
    p.hkv = static_cast<int>(hkv);
    p.d = head_dim;
    p.rot = rot;
    p.mscale = plan->mscale;
    for (int i = 0; i < 128; ++i) p.turns[i] = plan->turns[i];
    bool vec = head_dim % 8 == 0 && rot % 8 == 0;
    const auto fits16 = [](const void *a, long long stride, int bytes) { return aligned(a, 16) && stride * bytes % 16 == 0; };
    if (q) vec = vec && fits16(q, q_stride, ib) && fits16(q_out, q_out_stride, qb);
    if (k) {
        p.ck = cache->k;
        p.cv = cache->v;
        p.page_stride = cache->page_stride;
        p.row_stride = cache->row_stride;
        p.head_stride = cache->head_stride;
        p.n_slots = cache->n_pages * cache->page_size;
        p.page_shift = log2_of(cache->page_size);
        vec = vec && fits16(k, k_stride, ib) && fits16(v, v_stride, ib);
    }
    int sms = 0;
    const qgemv_status s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    return launch_rope(p, in_type, q ? q_type : QGEMV_F32, k ? cache->type : QGEMV_BF16, plan->layout == QGEMV_ROPE_HALF,
                       vec, n_tokens, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QGEMV_OK
               : QGEMV_ERR_CUDA;
}

// ------------------------------------------------------------- attention

size_t qgemv_attn_workspace_bytes(const qgemv_attn_batch *batch, const qgemv_kv_cache *cache)
{
    AttnPlan a;
    if (check_batch(batch, cache) != QGEMV_OK || plan_attn(batch, cache, a) != QGEMV_OK) return 0;
    return static_cast<size_t>(a.ws_bytes);
}

qgemv_status qgemv_attn_prefix(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                               const qgemv_kv_cache *cache, const qgemv_attn_batch *batch, void *o,
                               qgemv_dtype o_type, int64_t o_token_stride, int64_t o_head_stride, float *lse_or_null,
                               void *ws, size_t ws_bytes, qgemv_stream_t stream)
{
    qgemv_status s = check_batch(batch, cache);
    if (s != QGEMV_OK) return s;
    const qgemv_attn_batch &b = *batch;
    if (!q || !o || !b.suffix_len || (b.prefix_len > 0 && !b.prefix_pages) || (b.max_suffix > 0 && !b.suffix_pages) ||
        b.suffix_pages_stride < 0 || (o_type != QGEMV_F32 && o_type != cache->type))
        return QGEMV_ERR_INVALID_ARG;
    const long long tokens = static_cast<long long>(b.n_seqs) * b.n_q;
    const int d = cache->head_dim, ob = type_bytes(o_type);
    if (!extent_ok(tokens, q_token_stride) || !extent_ok(b.n_q_heads, q_head_stride) ||
        !extent_ok(tokens, o_token_stride) || !extent_ok(b.n_q_heads, o_head_stride) ||
        !extent_ok(b.n_seqs, b.suffix_pages_stride) ||
        !pieces_apart(tokens, o_token_stride, b.n_q_heads, o_head_stride, d))
        return QGEMV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 || !aligned(o, ob) || !aligned(b.suffix_len, 4) ||
        !aligned(b.prefix_pages, 4) || !aligned(b.suffix_pages, 4) || !aligned(lse_or_null, 4))
        return QGEMV_ERR_MISALIGNED;
    AttnPlan a;
    s = plan_attn(batch, cache, a);
    if (s != QGEMV_OK) return s;
    if (!ws || ws_bytes < static_cast<size_t>(a.ws_bytes)) return QGEMV_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return QGEMV_ERR_MISALIGNED;
    const long long heads1 = b.n_q_heads - 1;
    const Span so = span(o, ((tokens - 1) * o_token_stride + heads1 * o_head_stride + d) * ob);
    const Span sq = span(q, ((tokens - 1) * q_token_stride + heads1 * q_head_stride + d) * 2);
    const Span sw = span(ws, a.ws_bytes), sk = cache_span(cache, cache->k), sv = cache_span(cache, cache->v);
    const Span se = span(lse_or_null, lse_or_null ? 4 * tokens * b.n_q_heads : 0);
    const Span sl = span(b.suffix_len, 4ll * b.n_seqs);
    const Span sp = span(b.prefix_pages, 4 * ceil_div(b.prefix_len, cache->page_size));
    const long long own = ceil_div(b.max_suffix, cache->page_size);  // pages of a suffix
    const Span ss = own ? strided(b.suffix_pages, b.n_seqs, b.suffix_pages_stride, own, 4) : Span{0, 0};
    for (const Span out : {so, se, sw})
        for (const Span in : {sq, sk, sv, sl, sp, ss})
            if (overlap(out, in)) return QGEMV_ERR_INVALID_ARG;
    if (overlap(so, se) || overlap(so, sw) || overlap(se, sw)) return QGEMV_ERR_INVALID_ARG;

    AttnParams p = {};
    p.q = q;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.k = cache->k;
    p.v = cache->v;
    p.page_stride = cache->page_stride;
    p.row_stride = cache->row_stride;
    p.head_stride = cache->head_stride;
    p.n_pages = cache->n_pages;
    p.page_shift = log2_of(cache->page_size);
    p.d = d;
    p.prefix_pages = b.prefix_pages;
    p.suffix_pages = b.suffix_pages;
    p.suffix_len = b.suffix_len;
    p.suffix_pages_stride = b.suffix_pages_stride;
    p.n_seqs = b.n_seqs;
    p.n_q = b.n_q;
    p.hq = b.n_q_heads;
    p.hkv = cache->n_heads;
    p.group = a.group;
    p.rows = a.rows;
    p.prefix_len = b.prefix_len;
    p.max_suffix = b.max_suffix;
    p.scale = b.scale != 0.0f ? b.scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    p.scale_log2 = static_cast<float>(p.scale * 1.4426950408889634);
    p.p_tile = a.p_tile;
    p.p_tiles = a.p_tiles;
    p.p_splits = a.p_splits;
    p.p_keys = a.p_keys;
    p.s_tile = a.s_tile;
    p.s_tiles = a.s_tiles;
    p.s_splits = a.s_splits;
    p.s_keys = a.s_keys;
    p.p_first = a.p_first;
    p.p_blocks = p.hkv * a.p_tiles * a.p_splits;
    p.t_len = a.t_len;
    p.t_mode = a.t_mode;
    p.t_tiles = a.t_tiles;
    p.t_splits = a.t_splits;
    p.t_keys = a.t_keys;
    p.t_blocks = p.hkv * a.t_tiles * a.t_splits;
    p.t_wait = p.p_blocks == 0 && a.s_splits == 0;
    uint8_t *w = static_cast<uint8_t *>(ws) + kCounterArea;
    p.part_o = reinterpret_cast<float4 *>(w);
    p.o_row = a.t_mode ? 1 : d / 4;
    p.o_four = a.t_mode ? a.rows : 1;
    p.part_ml = reinterpret_cast<float2 *>(w + a.part_rows * 4 * d);
    p.o = o;
    p.o_token_stride = o_token_stride;
    p.o_head_stride = o_head_stride;
    p.lse = lse_or_null;
    int sms = 0;
    s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    return launch_attn(p, cache->type, o_type, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? QGEMV_OK
                                                                                                      : QGEMV_ERR_CUDA;
}

// ---------------------------------------------------------------- logits

static bool logits_shape_ok(const qgemv_logits_spec *s)
{
    return s && s->rows >= 1 && s->rows <= (1 << 24) && s->vocab >= 1 && s->vocab <= INT32_MAX;
}

size_t qgemv_logits_workspace_bytes(const qgemv_logits_spec *spec)
{
    return logits_shape_ok(spec) ? static_cast<size_t>(kCounterArea) : 0;
}

qgemv_status qgemv_logits_rules(const void *logits, qgemv_dtype type, int64_t x_stride, const qgemv_logits_spec *spec,
                                void *out, int64_t out_stride, int64_t *idx, float *val, void *ws, size_t ws_bytes,
                                qgemv_stream_t stream)
{
    if (!logits_shape_ok(spec) || !logits || !type_ok(type) || (!idx != !val) || (!out && !idx))
        return QGEMV_ERR_INVALID_ARG;
    const qgemv_logits_spec &c = *spec;
    const long long rows = c.rows, words = ceil_div(c.vocab, 32);
    const int eb = type_bytes(type);
    if (!extent_ok(rows, x_stride) || (rows > 1 && x_stride < c.vocab)) return QGEMV_ERR_INVALID_ARG;
    if (out && (!extent_ok(rows, out_stride) || (rows > 1 && out_stride < c.vocab))) return QGEMV_ERR_INVALID_ARG;
    if (!c.history && (c.repetition || c.frequency || c.presence)) return QGEMV_ERR_INVALID_ARG;
    if (c.history && (!c.history_len || c.max_history < 0 || c.max_history >= (1 << 20) ||
                      !extent_ok(rows, c.history_stride)))
        return QGEMV_ERR_INVALID_ARG;
    if ((!c.bias != !c.bias_ids) ||
        (c.bias && (!c.bias_len || c.max_bias < 0 || c.max_bias > 4095 || !extent_ok(rows, c.bias_stride))))
        return QGEMV_ERR_INVALID_ARG;
    if (c.mask && (!extent_ok(rows, c.mask_stride) || (c.mask_stride != 0 && c.mask_stride < words)))
        return QGEMV_ERR_INVALID_ARG;
    if (!ws || ws_bytes < static_cast<size_t>(kCounterArea)) return QGEMV_ERR_WORKSPACE;
    if (!aligned(logits, eb) || !aligned(out, eb) || !aligned(idx, 8) || !aligned(val, 4) || !aligned(ws, 16) ||
        !aligned(c.history, 8) || !aligned(c.history_len, 4) || !aligned(c.repetition, 4) ||
        !aligned(c.frequency, 4) || !aligned(c.presence, 4) || !aligned(c.bias_ids, 8) || !aligned(c.bias, 4) ||
        !aligned(c.bias_len, 4) || !aligned(c.mask, 4))
        return QGEMV_ERR_MISALIGNED;
    // what is written must not overlap what is read, nor each other
    Span outs[4], ins[10];
    int no = 0, ni = 0;
    const Span sx = strided(logits, rows, x_stride, c.vocab, eb);
    const bool in_place = out == logits && (out_stride == x_stride || rows == 1);
    if (!in_place) ins[ni++] = sx;
    if (c.history) {
        ins[ni++] = strided(c.history, rows, c.history_stride, c.max_history, 8);
        ins[ni++] = span(c.history_len, 4 * rows);
    }
    if (c.bias) {
        ins[ni++] = strided(c.bias_ids, rows, c.bias_stride, c.max_bias, 8);
        ins[ni++] = strided(c.bias, rows, c.bias_stride, c.max_bias, 4);
        ins[ni++] = span(c.bias_len, 4 * rows);
    }
    if (c.mask) ins[ni++] = strided(c.mask, rows, c.mask_stride, words, 4);
    for (const float *f : {c.repetition, c.frequency, c.presence})
        if (f) ins[ni++] = span(f, 4 * rows);
    if (out) outs[no++] = strided(out, rows, out_stride, c.vocab, eb);
    if (idx) {
        outs[no++] = span(idx, 8 * rows);
        outs[no++] = span(val, 4 * rows);
    }
    outs[no++] = span(ws, kCounterArea);
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return QGEMV_ERR_INVALID_ARG;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return QGEMV_ERR_INVALID_ARG;
    }

    int sms = 0;
    LogitsParams p = {};
    const qgemv_status s = device_props(&sms, &p.status);
    if (s != QGEMV_OK) return s;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.vocab = c.vocab;
    p.hist_stride = c.history_stride;
    p.max_hist = c.max_history;
    p.bias_stride = c.bias_stride;
    p.max_bias = c.max_bias;
    p.mask_stride = c.mask_stride;
    p.keys = static_cast<unsigned long long *>(ws);
    p.cnt = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(ws) + LOGITS_KEYS_BYTES);
    for (long long r = 0; r < rows; r += LOGITS_ROWS) {
        const auto at = [&](auto *base, long long stride) { return base ? base + r * stride : base; };
        p.x = static_cast<const uint8_t *>(logits) + r * x_stride * eb;
        p.out = out ? static_cast<uint8_t *>(out) + r * out_stride * eb : nullptr;
        p.hist = reinterpret_cast<const long long *>(at(c.history, c.history_stride));
        p.hist_len = at(c.history_len, 1);
        p.rep = at(c.repetition, 1);
        p.freq = at(c.frequency, 1);
        p.pres = at(c.presence, 1);
        p.bias_ids = reinterpret_cast<const long long *>(at(c.bias_ids, c.bias_stride));
        p.bias = at(c.bias, c.bias_stride);
        p.bias_len = at(c.bias_len, 1);
        p.mask = at(c.mask, c.mask_stride);
        p.idx = idx ? reinterpret_cast<long long *>(idx) + r : nullptr;
        p.val = val ? val + r : nullptr;
        if (launch_logits(p, type, static_cast<int>(std::min<long long>(LOGITS_ROWS, rows - r)), sms,
                          reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
            return QGEMV_ERR_CUDA;
    }
    return QGEMV_OK;
}

}  // extern "C"
