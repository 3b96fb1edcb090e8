// kv8_append.cu -- rows written to a paged cache of 8-bit codes with a scale
// for each block of rows and head.
//
// For a block and head, k and v each: s' = max(s, max |x| / Q) over the new rows
// x, s the scale of the rows it held before (0 without any); codes of the new rows
// rn(x * (1 / s')), and, where s' > s, old codes c become rn(c * (s * (1 / s'))).
//
// A thread block takes a block of one head after the other, so nobody else touches the
// codes and the scale that it reads and writes anew, and no atomics are needed.  The new rows
// stay in registers between the maximum and the codes (up to KA_PIECES pieces of eight
// elements a thread; more are read a second time, from L2).
//
// What bounds it: memory for prompts (rows read once, a code written for each
// element): 24000 rows of 8 + 8 heads of 128, bf16, in 26.6 us, 5.5 TB/s; the rest is
// that a block's loads stand still while it forms maximum and codes.  For single tokens the
// chain of dependent loads, lengths, page, row, scale: 2.8 us for 64 of 8 + 8 heads.
#include <float.h>

#include <type_traits>

#include "kv8_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int KA_PIECES = 4;  // of eight elements, in a thread's registers

template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
};
__device__ __forceinline__ void spread(const Eight<float> &v, float (&f)[8])
{
    memcpy(f, &v, 32);
}
__device__ __forceinline__ void spread(const Eight<__half> &v, float (&f)[8])
{
    const unsigned u[4] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
        f[2 * i] = a.x, f[2 * i + 1] = a.y;
    }
}
__device__ __forceinline__ void spread(const Eight<__nv_bfloat16> &v, float (&f)[8])
{
    const unsigned u[4] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
}
template <typename T, bool VEC>
__device__ __forceinline__ Eight<T> load8(const T *x)
{
    Eight<T> v;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v.w[i] = __ldg(reinterpret_cast<const uint4 *>(x) + i);
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = x[i];
        memcpy(&v, e, sizeof(v));
    }
    return v;
}

// The largest |x| of eight, as the bits of a non-negative number of the type, which order
// as the numbers do; NaN lies above infinity.
__device__ __forceinline__ unsigned largest_bits(const Eight<float> &v, unsigned top)
{
    const unsigned u[8] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w, v.w[1].x, v.w[1].y, v.w[1].z, v.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, u[i] & 0x7FFFFFFFu);
    return top;
}
template <typename T>
__device__ __forceinline__ unsigned largest_bits(const Eight<T> &v, unsigned top)  // in both halves of `top`
{
    const unsigned u[4] = {v.w[0].x, v.w[0].y, v.w[0].z, v.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, u[i] & 0x7FFF7FFFu);
    return top;
}
template <typename T>
__device__ __forceinline__ float from_bits(unsigned top);
template <>
__device__ __forceinline__ float from_bits<float>(unsigned top)
{
    return __uint_as_float(top);
}
template <>
__device__ __forceinline__ float from_bits<__half>(unsigned top)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(max(top & 0xFFFFu, top >> 16))));
}
template <>
__device__ __forceinline__ float from_bits<__nv_bfloat16>(unsigned top)
{
    return __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16);
}

template <int CODE>
constexpr float KA_TOP = CODE == QGEMV_CODE_INT8 ? 127.0f : 448.0f;

// Four values (already over their scale) as codes.  CAREFUL: NaN as 0, values beyond
// the codes as the last one; without it they are neither NaN nor above KA_TOP by more than a
// rounding.
template <int CODE, bool CAREFUL>
__device__ __forceinline__ unsigned encode4(const float *f)
{
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = !CAREFUL ? f[i] : f[i] == f[i] ? fminf(fmaxf(f[i], -KA_TOP<CODE>), KA_TOP<CODE>) : 0.0f;
    if constexpr (CODE == QGEMV_CODE_INT8) {
        // 1.5 * 2^23 + v ends, rounded to nearest even, in v as two's complement
        unsigned u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(__fadd_rn(v[i], 12582912.0f));
        return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    } else {
        unsigned short lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[1]), "f"(v[0]));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[3]), "f"(v[2]));
        return static_cast<unsigned>(lo) | static_cast<unsigned>(hi) << 16;
    }
}
template <int CODE>
__device__ __forceinline__ void decode4(unsigned w, float *f)
{
    if constexpr (CODE == QGEMV_CODE_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<signed char>(w >> (8 * i) & 0xFF));
    } else {
        unsigned a, b;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(w));
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
    }
}

// Block x: sequence x / blocks, its (x % blocks)-th block with new rows; block y:
// `items` of the heads of k and v (item 2 h is head h's k, 2 h + 1 its v), one
// after the other, the next one's rows on their way meanwhile.
template <typename T, int CODE, bool VEC, int THREADS, bool MANY>
__global__ void __launch_bounds__(THREADS) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p)
{
    __shared__ unsigned s_top[2][THREADS / 32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / p.blocks, jb = blockIdx.x % p.blocks;
    const int len = __ldg(p.lens + b);
    const long long t0 = p.first ? __ldg(p.first + b) : static_cast<long long>(b) * p.n_new;
    const long long t1 = p.first ? __ldg(p.first + b + 1) : t0 + p.n_new;
    const bool told = tid == 0 && jb == 0 && blockIdx.y == 0;
    const int n = len < 0 ? 0 : len > p.max_len ? p.max_len : len;
    if (n != len && told) atomicCAS(p.status, 0u, ST_BAD_ID);
    if (len == 0) return;  // a padded batch's place
    if (t0 < 0 || t1 > p.n_tokens || t1 < t0 || t1 - t0 > p.max_new || t1 - t0 > n) {
        if (told) atomicCAS(p.status, 0u, ST_BAD_ID);
        return;
    }
    const int old = n - static_cast<int>(t1 - t0);
    const int block = 1 << p.c.block_shift;
    const int start = ((old >> p.c.block_shift) + jb) << p.c.block_shift;
    if (start >= n || t0 == t1) return;
    const int lo = max(start, old), hi = min(start + block, n);
    const int page = __ldg(p.pages + b * p.pages_stride + (start >> p.c.page_shift));
    if (page < 0 || page >= p.c.n_pages) {
        if (tid == 0) atomicCAS(p.status, 0u, ST_BAD_ID);
        return;
    }
    const int in_page = start & ((1 << p.c.page_shift) - 1);
    const long long code_at = page * p.c.page_stride + in_page * p.c.row_stride;
    const long long scale_at = page * p.c.scale_page + (in_page >> p.c.block_shift) * p.c.scale_block;
    const long long token = t0 + (lo - old);
    const int total = (hi - lo) * p.pieces;
    // the thread's first pieces, the same of every head
    int row[KA_PIECES], col[KA_PIECES];
#pragma unroll
    for (int u = 0; u < KA_PIECES; ++u) {
        const int i = tid + u * THREADS;  // below 1024, and a row has 32 pieces at most: the product's top is the quotient
        row[u] = i * p.per_piece >> 16, col[u] = (i - row[u] * p.pieces) * 8;
    }

    const T *xk = static_cast<const T *>(p.k) + token * p.k_stride, *xv = static_cast<const T *>(p.v) + token * p.v_stride;
    Eight<T> next[KA_PIECES];
    float next_was = 0.0f;
    auto fetch = [&](int item) {
        const T *x = (item & 1 ? xv : xk) + static_cast<long long>(item >> 1) * p.d;
        const int stride = item & 1 ? p.v_stride : p.k_stride;
        if (old > start) next_was = __ldcg((item & 1 ? p.c.vs : p.c.ks) + scale_at + (item >> 1) * p.c.scale_head);
#pragma unroll
        for (int u = 0; u < KA_PIECES; ++u)
            if (tid + u * THREADS < total) next[u] = load8<T, VEC>(x + static_cast<long long>(row[u]) * stride + col[u]);
    };
    const int item0 = MANY ? blockIdx.y * p.items : blockIdx.y, item1 = MANY ? min(item0 + p.items, 2 * p.hkv) : item0 + 1;
    fetch(item0);
    for (int item = item0; item < item1; ++item) {
        const bool is_v = item & 1;
        const int h = item >> 1;
        uint8_t *codes = (is_v ? p.c.v : p.c.k) + code_at + h * p.c.head_stride;
        float *scale = (is_v ? p.c.vs : p.c.ks) + scale_at + h * p.c.scale_head;
        const int stride = is_v ? p.v_stride : p.k_stride;
        const T *x = (is_v ? xv : xk) + static_cast<long long>(h) * p.d;
        Eight<T> held[KA_PIECES];
#pragma unroll
        for (int u = 0; u < KA_PIECES; ++u) held[u] = next[u];
        const float was = next_was;
        bool odd = false;  // values or scales that the codes' conversion has to look at
        if (MANY && item + 1 < item1) fetch(item + 1);

        // pieces beyond those that registers hold
        auto rest = [&](auto f) {
            for (int i = tid + KA_PIECES * THREADS; i < total; i += THREADS) {
                const int r = i / p.pieces, c = (i - r * p.pieces) * 8;
                f(load8<T, VEC>(x + static_cast<long long>(r) * stride + c), r, c);
            }
        };
        // the largest of the block's values; one above infinity's bits tells of a NaN
        float top;
        auto all = [&](unsigned bits) {
            const float mine = from_bits<T>(bits);
            const unsigned u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mine));
            if ((tid & 31) == 0) s_top[item & 1][tid >> 5] = u;
            __syncthreads();
            unsigned most = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) most = max(most, s_top[item & 1][w]);
            top = __uint_as_float(most);
        };
        unsigned bits = 0;
#pragma unroll
        for (int u = 0; u < KA_PIECES; ++u)
            if (tid + u * THREADS < total) bits = largest_bits(held[u], bits);
        rest([&](const Eight<T> &v, int, int) { bits = largest_bits(v, bits); });
        all(bits);
        if (!(top <= FLT_MAX)) {  // infinities stay, NaN is passed over
            float most = 0.0f;
            auto pass = [&](const Eight<T> &v) {
                float f[8];
                spread(v, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(f[i]));
            };
#pragma unroll
            for (int u = 0; u < KA_PIECES; ++u)
                if (tid + u * THREADS < total) pass(held[u]);
            rest([&](const Eight<T> &v, int, int) { pass(v); });
            const unsigned u = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
            __syncthreads();
            if ((tid & 31) == 0) s_top[item & 1][tid >> 5] = u;
            __syncthreads();
            unsigned w_most = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) w_most = max(w_most, s_top[item & 1][w]);
            odd = true;
            top = __uint_as_float(w_most);
        }

        const float now = fmaxf(was, __fdiv_rn(top, KA_TOP<CODE>));
        const float inv = now > 0.0f ? __fdiv_rn(1.0f, now) : 0.0f;
        // scales that are subnormal, infinite or no number
        if (!(now >= FLT_MIN && now <= FLT_MAX)) odd = true;
        auto write = [&](const Eight<T> &v, int r, int c, auto careful) {
            float f[8];
            spread(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], inv);
            *reinterpret_cast<uint2 *>(codes + (lo - start + r) * static_cast<long long>(p.code_row) + c) =
                make_uint2(encode4<CODE, careful.value>(f), encode4<CODE, careful.value>(f + 4));
        };
        if (!odd) {
#pragma unroll
            for (int u = 0; u < KA_PIECES; ++u)
                if (tid + u * THREADS < total) write(held[u], row[u], col[u], std::false_type());
        } else {
#pragma unroll
            for (int u = 0; u < KA_PIECES; ++u)
                if (tid + u * THREADS < total) write(held[u], row[u], col[u], std::true_type());
        }
        rest([&](const Eight<T> &v, int r, int c) { write(v, r, c, std::true_type()); });
        if (old <= start) {
            if (tid == 0) *scale = now;
        } else if (now > was) {  // old codes to the new scale
            const float by = __fmul_rn(was, inv);
            for (int i = tid; i < (old - start) * p.pieces; i += THREADS) {
                const int r = i / p.pieces;
                uint2 *c = reinterpret_cast<uint2 *>(codes + r * p.c.row_stride + (i - r * p.pieces) * 8);
                const uint2 w = *c;
                float f[8];
                decode4<CODE>(w.x, f);
                decode4<CODE>(w.y, f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], by);
                *c = make_uint2(encode4<CODE, true>(f), encode4<CODE, true>(f + 4));
            }
            if (tid == 0) *scale = now;  // every thread has read it: a barrier lies between
        }
    }
}

template <typename T, int CODE, bool VEC>
cudaError_t launch_t(Kv8AppendParams p, cudaStream_t st)
{
    const long long blocks = static_cast<long long>(p.n_seqs) * p.blocks;
    // Items one after the other pay once there are some blocks for each multiprocessor; more than
    // four leave too few waves of blocks (24000 rows of 8 + 8 heads, up to 2 / 4 / 8 / 16 items: 29.1 /
    // 26.6 / 28.3 / 30.2 us).
    p.items = 1;
    p.per_piece = (65536 + p.pieces - 1) / p.pieces;
    while (p.items < 4 && blocks * 2 * p.hkv >= 16ll * ATTN_SMS * p.items && p.items < 2 * p.hkv) p.items *= 2;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((2 * p.hkv + p.items - 1) / p.items));
    const bool wide = min(1 << p.c.block_shift, p.max_new) * p.pieces > 128 * KA_PIECES;
    const auto go = [&](auto kernel, unsigned threads) { return launch_pdl(kernel, grid, threads, 0, st, p); };
    // one item a block: no second set of rows in registers, and twice the blocks a multiprocessor
    if (p.items == 1)
        return wide ? go(kv8_append_kernel<T, CODE, VEC, 256, false>, 256) : go(kv8_append_kernel<T, CODE, VEC, 128, false>, 128);
    return wide ? go(kv8_append_kernel<T, CODE, VEC, 256, true>, 256) : go(kv8_append_kernel<T, CODE, VEC, 128, true>, 128);
}
template <typename T>
cudaError_t launch_in(const Kv8AppendParams &p, qgemv_code_type code, bool vec, cudaStream_t st)
{
    if (code == QGEMV_CODE_INT8)
        return vec ? launch_t<T, QGEMV_CODE_INT8, true>(p, st) : launch_t<T, QGEMV_CODE_INT8, false>(p, st);
    return vec ? launch_t<T, QGEMV_CODE_E4M3, true>(p, st) : launch_t<T, QGEMV_CODE_E4M3, false>(p, st);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendParams &p, qgemv_dtype in, qgemv_code_type code, bool vec, cudaStream_t st)
{
    switch (in) {
    case QGEMV_F32: return launch_in<float>(p, code, vec, st);
    case QGEMV_F16: return launch_in<__half>(p, code, vec, st);
    default: return launch_in<__nv_bfloat16>(p, code, vec, st);
    }
}

}  // namespace qg
