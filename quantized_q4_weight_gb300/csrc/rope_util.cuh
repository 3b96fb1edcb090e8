// rope_util.cuh -- what the kernels that rotate q and k share (rope_kv.cu,
// norm_rope.cu): conversions, accesses of eight elements a thread, angles, and
// where a head comes from and goes.
#pragma once

#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v)
{
    return v;
}
template <>
__device__ __forceinline__ float to_f<__half>(__half v)
{
    return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v)
{
    return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v)
{
    return v;
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v)
{
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Four consecutive elements as they lie in memory (8 or 16 bytes, aligned to
// their size): whole words, which with the 16-byte accesses below bring 7970
// tokens of 32 + 8 + 8 heads of 128, bf16, interleaved, from 51 to 36 us.
template <typename T>
struct Four {
    uint2 w;
};
template <>
struct Four<float> {
    float4 w;
};

__device__ __forceinline__ void unpack(const Four<float> &v, float (&f)[4])
{
    f[0] = v.w.x, f[1] = v.w.y, f[2] = v.w.z, f[3] = v.w.w;
}
__device__ __forceinline__ void unpack(const Four<__half> &v, float (&f)[4])
{
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.w.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.w.y));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
__device__ __forceinline__ void unpack(const Four<__nv_bfloat16> &v, float (&f)[4])
{
    f[0] = __uint_as_float(v.w.x << 16), f[1] = __uint_as_float(v.w.x & 0xffff0000u);
    f[2] = __uint_as_float(v.w.y << 16), f[3] = __uint_as_float(v.w.y & 0xffff0000u);
}
__device__ __forceinline__ void pack(const float (&f)[4], Four<float> &v) { v.w = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void pack(const float (&f)[4], Four<__half> &v)
{
    const __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
    v.w = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
}
__device__ __forceinline__ void pack(const float (&f)[4], Four<__nv_bfloat16> &v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    v.w = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
}

// cos and sin of position * theta, by the turns' fraction.
__device__ __forceinline__ void angle(int pos, unsigned long long turns, float mscale, float &c, float &s)
{
    const unsigned long long frac = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
    const int half_turns = static_cast<int>(static_cast<unsigned>(frac >> 32));
    float sn, cs;
    sincospif(static_cast<float>(half_turns) * 4.656612873077393e-10f, &sn, &cs);  // * 2^-31
    c = cs * mscale;
    s = sn * mscale;
}

// Head h of token t: the q heads, then k's, then v's.  Where it comes from
// (nullptr: a k or v head without a cache row), and where it goes.
template <typename TI>
__device__ __forceinline__ const TI *head_src(const RopeParams &p, long long t, int h, bool row)
{
    if (h < p.hq) return static_cast<const TI *>(p.q) + t * p.q_stride + h * p.d;
    if (!row) return nullptr;
    if (h < p.hq + p.hkv) return static_cast<const TI *>(p.k) + t * p.k_stride + (h - p.hq) * p.d;
    return static_cast<const TI *>(p.v) + t * p.v_stride + (h - p.hq - p.hkv) * p.d;
}
template <typename TQ>
__device__ __forceinline__ TQ *q_dst(const RopeParams &p, long long t, int h)
{
    return static_cast<TQ *>(p.q_out) + t * p.q_out_stride + h * p.d;
}
template <typename TC>
__device__ __forceinline__ TC *kv_dst(const RopeParams &p, int h, long long row_off)
{
    const int g = h - p.hq;
    return g < p.hkv ? static_cast<TC *>(p.ck) + row_off + g * p.head_stride
                     : static_cast<TC *>(p.cv) + row_off + (g - p.hkv) * p.head_stride;
}

// A thread's two fours of a head.  Interleaved they are neighbours, and 16-bit
// ones travel as one 16-byte access: full sectors instead of halves.
template <typename T, bool HALF>
__device__ __forceinline__ void load8(const T *at, int a, int b, Four<T> &x, Four<T> &y)
{
    if constexpr (!HALF && sizeof(T) == 2) {
        const uint4 w = *reinterpret_cast<const uint4 *>(at + a);
        x.w = make_uint2(w.x, w.y), y.w = make_uint2(w.z, w.w);
    } else {
        x = *reinterpret_cast<const Four<T> *>(at + a);
        y = *reinterpret_cast<const Four<T> *>(at + b);
    }
}
template <typename T, bool HALF>
__device__ __forceinline__ void store8(T *at, int a, int b, const float (&x)[4], const float (&y)[4])
{
    Four<T> ox, oy;
    pack(x, ox);
    pack(y, oy);
    if constexpr (!HALF && sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(at + a) = make_uint4(ox.w.x, ox.w.y, oy.w.x, oy.w.y);
    } else {
        *reinterpret_cast<Four<T> *>(at + a) = ox;
        *reinterpret_cast<Four<T> *>(at + b) = oy;
    }
}

// The token's cache row in elements from the cache's base, -1 for none.
__device__ __forceinline__ long long cache_row(const RopeParams &p, long long t)
{
    if (p.hkv == 0) return -1;
    const int slot = __ldg(p.slots + t);
    if (slot < 0 || slot >= p.n_slots) {
        if (slot != -1 && threadIdx.x == 0) atomicCAS(p.status, 0u, ST_BAD_ID);
        return -1;
    }
    return static_cast<long long>(slot >> p.page_shift) * p.page_stride +
           static_cast<long long>(slot & ((1 << p.page_shift) - 1)) * p.row_stride;
}

}  // namespace
}  // namespace qg
