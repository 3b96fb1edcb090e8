// kv8_append.cu -- rows written to a paged cache of 8-bit codes with a scale
// for each block of rows and head.
//
// For a block and head, k and v each: s' = max(s, max |x| / Q) over the new rows
// x, s the scale of the rows it held before (0 without any); codes of the new rows
// rn(x * (1 / s')), and, where s' > s, old codes c become rn(c * (s * (1 / s'))).
//
// A thread block takes one block of one head, so nobody else touches the codes and
// the scale that it reads and writes anew, and no atomics are needed.  The new rows
// stay in registers between the maximum and the codes (up to NR pieces of eight
// elements a thread; more are read a second time, from L2).
//
// What bounds it: memory for prompts (rows read once, a code written for each
// element), for single tokens the chain of dependent loads: lengths, page, row, scale.
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

template <int CODE>
constexpr float KA_TOP = CODE == QGEMV_CODE_INT8 ? 127.0f : 448.0f;

// Four values (already over their scale) as codes; NaN as 0.
template <int CODE>
__device__ __forceinline__ unsigned encode4(const float *f)
{
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f[i] == f[i] ? fminf(fmaxf(f[i], -KA_TOP<CODE>), KA_TOP<CODE>) : 0.0f;
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
// head y / 2, k or v.
template <typename T, int CODE, bool VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p)
{
    __shared__ float s_top[THREADS / 32];
    const int tid = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x / p.blocks, jb = blockIdx.x % p.blocks;
    const int h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const int len = __ldg(p.lens + b);
    const long long t0 = p.first ? __ldg(p.first + b) : static_cast<long long>(b) * p.n_new;
    const long long t1 = p.first ? __ldg(p.first + b + 1) : t0 + p.n_new;
    const bool told = tid == 0 && jb == 0 && blockIdx.y == 0;
    const int n = len < 0 ? 0 : len > p.max_len ? p.max_len : len;
    if (n != len && told) atomicCAS(p.status, 0u, ST_BAD_ID);
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
    uint8_t *codes = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + in_page * p.c.row_stride + h * p.c.head_stride;
    float *scale = (is_v ? p.c.vs : p.c.ks) + page * p.c.scale_page + (in_page >> p.c.block_shift) * p.c.scale_block +
                   h * p.c.scale_head;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const T *x = static_cast<const T *>(is_v ? p.v : p.k) + (t0 + (lo - old)) * stride + static_cast<long long>(h) * p.d;
    const float was = old > start ? *scale : 0.0f;

    const int total = (hi - lo) * p.pieces;
    Eight<T> held[KA_PIECES];
    float top = 0.0f;
    auto largest = [&](const Eight<T> &v) {
        float f[8];
        spread(v, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));  // passes NaN over
    };
    auto at = [&](int i) { return x + i / p.pieces * stride + i % p.pieces * 8; };
#pragma unroll
    for (int u = 0; u < KA_PIECES; ++u)
        if (tid + u * THREADS < total) held[u] = load8<T, VEC>(at(tid + u * THREADS));
#pragma unroll
    for (int u = 0; u < KA_PIECES; ++u)
        if (tid + u * THREADS < total) largest(held[u]);
    for (int i = tid + KA_PIECES * THREADS; i < total; i += THREADS) largest(load8<T, VEC>(at(i)));
    // non-negative floats order as their bits do
    top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_top[w]);

    const float now = fmaxf(was, __fdiv_rn(top, KA_TOP<CODE>));
    const float inv = now > 0.0f ? __fdiv_rn(1.0f, now) : 0.0f;
    auto write = [&](const Eight<T> &v, int i) {
        float f[8];
        spread(v, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], inv);
        *reinterpret_cast<uint2 *>(codes + (lo - start + i / p.pieces) * p.c.row_stride + i % p.pieces * 8) =
            make_uint2(encode4<CODE>(f), encode4<CODE>(f + 4));
    };
#pragma unroll
    for (int u = 0; u < KA_PIECES; ++u)
        if (tid + u * THREADS < total) write(held[u], tid + u * THREADS);
    for (int i = tid + KA_PIECES * THREADS; i < total; i += THREADS) write(load8<T, VEC>(at(i)), i);
    if (now > was || old <= start) {
        if (old > start) {  // old codes to the new scale
            const float by = __fmul_rn(was, inv);
            for (int i = tid; i < (old - start) * p.pieces; i += THREADS) {
                uint2 *c = reinterpret_cast<uint2 *>(codes + i / p.pieces * p.c.row_stride + i % p.pieces * 8);
                const uint2 w = *c;
                float f[8];
                decode4<CODE>(w.x, f);
                decode4<CODE>(w.y, f + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], by);
                *c = make_uint2(encode4<CODE>(f), encode4<CODE>(f + 4));
            }
        }
        if (tid == 0) *scale = now;  // every thread has read it: a barrier lies between
    }
}

template <typename T, int CODE, bool VEC>
cudaError_t launch_t(const Kv8AppendParams &p, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(p.n_seqs) * static_cast<unsigned>(p.blocks), 2 * static_cast<unsigned>(p.hkv));
    const int rows = min(1 << p.c.block_shift, p.max_new);
    return rows * p.pieces > 128 * KA_PIECES ? launch_pdl(kv8_append_kernel<T, CODE, VEC, 256>, grid, 256, 0, st, p)
                                             : launch_pdl(kv8_append_kernel<T, CODE, VEC, 128>, grid, 128, 0, st, p);
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
