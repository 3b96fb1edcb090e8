// rope_kv.cu -- rotary positions on q and k with the write into the paged
// cache (minfer README "How it works": RoPE between the QKV product and the
// attention).
//
// A pair (x, y) at position p with frequency theta becomes
// (x c - y s, x s + y c), c = mscale cos(p theta), s = mscale sin(p theta).
// In fp32 the product p theta alone would be off by up to p theta 2^-24
// radians (4e-3 at position 131072), so the angle is formed in integers: the
// plan holds theta / (2 pi) in units of 2^-64 turns, and the low 64 bits of
// p * turns are the fraction of a turn, exact but for the rounding of the
// frequency itself, to 53 bits (p 2^-55 turns).  Its top 32 bits as a signed
// number of half turns / 2^31 go to sincospif: the angle is off by less than
// 1e-6 radians at every 32-bit position.
//
// What bounds it: memory for prompts (each element is read and written once,
// 3 flops per element), launch and load latency for a few tokens.  A block
// takes one token; a thread keeps one place within the head (four pairs: one
// or two 16-byte loads) and walks the heads, with the loads of several heads
// in flight.  The token's sines are formed once, a thread each, and passed
// through shared memory while those loads run.  Few tokens spread the heads
// over blocks, one head a thread: more blocks, the sines repeated.
//
// Measured: 16384 tokens of 32 + 8 + 8 heads of 128, fp32 to bf16: 89 us, 6.8
// TB/s, as a copy; blocks of 256 threads with four heads in flight 106, sines
// formed by every thread for itself 152, blocks of 64 threads 88 (but 1021
// tokens of 14 + 2 + 2 heads of 64: 3.4 us instead of 2.9).  One token 2.1 us,
// the time between launches.
#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_UNROLL = 3;  // heads in flight per thread

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

// Four consecutive elements (8 or 16 bytes, aligned to their size).
template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T e[4];
};

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

template <typename T>
__device__ __forceinline__ void store8(T *at, int a, int b, const float (&x)[4], const float (&y)[4])
{
    Four<T> ox, oy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ox.e[i] = from_f<T>(x[i]);
        oy.e[i] = from_f<T>(y[i]);
    }
    *reinterpret_cast<Four<T> *>(at + a) = ox;
    *reinterpret_cast<Four<T> *>(at + b) = oy;
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

// Eight elements of a head a thread: unit j < rot / 8 is four pairs (HALF:
// elements 4j.. and rot/2 + 4j..; interleaved: 8j..), later units are copied.
template <typename TI, typename TQ, typename TC, bool HALF>
__global__ void __launch_bounds__(ROPE_THREADS, 8) rope_vec_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float s_c[128], s_s[128];
    pdl_launch_dependents();
    const int units = p.d >> 3;
    const int j = static_cast<int>(threadIdx.x) % units, hb = static_cast<int>(threadIdx.x) / units;
    const long long t = blockIdx.x;
    const int heads = p.hq + 2 * p.hkv;
    const bool rot_unit = 8 * j < p.rot;
    const int a = HALF && rot_unit ? 4 * j : 8 * j;                  // first four elements
    const int b = HALF && rot_unit ? p.rot / 2 + 4 * j : 8 * j + 4;  // second four
    pdl_wait();
    const int pos = __ldg(p.pos + t);
    const long long row_off = cache_row(p, t);
    float c[4], s[4];
    bool have = false;
    const int step = p.heads_per_block * static_cast<int>(gridDim.y);
    // every thread passes the barrier below in its first turn, with heads or without
    for (int h0 = hb + p.heads_per_block * static_cast<int>(blockIdx.y); h0 < heads || !have; h0 += ROPE_UNROLL * step) {
        Four<TI> x[ROPE_UNROLL], y[ROPE_UNROLL];
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            const int h = h0 + u * step;
            const TI *src = h < heads ? head_src<TI>(p, t, h, row_off >= 0) : nullptr;
            if (src) {
                x[u] = *reinterpret_cast<const Four<TI> *>(src + a);
                y[u] = *reinterpret_cast<const Four<TI> *>(src + b);
            }
        }
        if (!have) {
            for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) angle(pos, p.turns[i], p.mscale, s_c[i], s_s[i]);
            __syncthreads();
            if (rot_unit) {
                const float4 cc = *reinterpret_cast<const float4 *>(s_c + 4 * j);
                const float4 ss = *reinterpret_cast<const float4 *>(s_s + 4 * j);
                c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
                s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
            }
            have = true;
        }
#pragma unroll
        for (int u = 0; u < ROPE_UNROLL; ++u) {
            const int h = h0 + u * step;
            if (h >= heads || (h >= p.hq && row_off < 0)) break;  // the heads that follow have no row either
            float fx[4], fy[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fx[i] = to_f(x[u].e[i]);
                fy[i] = to_f(y[u].e[i]);
            }
            if (rot_unit && h < p.hq + p.hkv) {
                if constexpr (HALF) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float px = fx[i], py = fy[i];
                        fx[i] = px * c[i] - py * s[i];
                        fy[i] = px * s[i] + py * c[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float px = fx[2 * i], py = fx[2 * i + 1];
                        fx[2 * i] = px * c[i] - py * s[i];
                        fx[2 * i + 1] = px * s[i] + py * c[i];
                        const float qx = fy[2 * i], qy = fy[2 * i + 1];
                        fy[2 * i] = qx * c[i + 2] - qy * s[i + 2];
                        fy[2 * i + 1] = qx * s[i + 2] + qy * c[i + 2];
                    }
                }
            }
            if (h < p.hq)
                store8(q_dst<TQ>(p, t, h), a, b, fx, fy);
            else
                store8(kv_dst<TC>(p, h, row_off), a, b, fx, fy);
        }
    }
}

// One pair of a head a thread, any alignment and even sizes.
template <typename TI, typename TQ, typename TC, bool HALF>
__global__ void __launch_bounds__(ROPE_THREADS) rope_any_kernel(const __grid_constant__ RopeParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x;
    const int heads = p.hq + 2 * p.hkv, pairs = p.d >> 1, rpairs = p.rot >> 1;
    const long long row_off = cache_row(p, t);
    const int pos = __ldg(p.pos + t);
    const int first = static_cast<int>(blockIdx.y * ROPE_THREADS + threadIdx.x);
    for (int i = first; i < heads * pairs; i += ROPE_THREADS * static_cast<int>(gridDim.y)) {
        const int h = i / pairs, j = i - h * pairs;
        const TI *src = head_src<TI>(p, t, h, row_off >= 0);
        if (!src) continue;
        const bool rot_pair = j < rpairs;
        const int a = HALF && rot_pair ? j : 2 * j, b = HALF && rot_pair ? rpairs + j : 2 * j + 1;
        float x = to_f(src[a]), y = to_f(src[b]);
        if (rot_pair && h < p.hq + p.hkv) {
            float c, s;
            angle(pos, p.turns[j], p.mscale, c, s);
            const float px = x, py = y;
            x = px * c - py * s;
            y = px * s + py * c;
        }
        if (h < p.hq) {
            TQ *dst = q_dst<TQ>(p, t, h);
            dst[a] = from_f<TQ>(x);
            dst[b] = from_f<TQ>(y);
        } else {
            TC *dst = kv_dst<TC>(p, h, row_off);
            dst[a] = from_f<TC>(x);
            dst[b] = from_f<TC>(y);
        }
    }
}

template <typename TI, typename TQ, typename TC, bool HALF>
cudaError_t launch4(RopeParams &p, bool vec, long long n, int sms, cudaStream_t st)
{
    const int heads = p.hq + 2 * p.hkv;
    const unsigned nx = static_cast<unsigned>(n);
    if (vec) {
        const int units = p.d / 8;
        p.heads_per_block = ROPE_THREADS / units;
        const int chunks = (heads + p.heads_per_block - 1) / p.heads_per_block;
        // blocks that share a token repeat its sines; they pay while the tokens alone leave multiprocessors idle
        const unsigned ny = static_cast<unsigned>(n * chunks <= 2ll * sms ? chunks : 1);
        return launch_pdl(rope_vec_kernel<TI, TQ, TC, HALF>, dim3(nx, ny), p.heads_per_block * units, 0, st, p);
    }
    const int chunks = (heads * (p.d / 2) + ROPE_THREADS - 1) / ROPE_THREADS;
    const unsigned ny = static_cast<unsigned>(n * chunks <= 2ll * sms ? chunks : 1);
    return launch_pdl(rope_any_kernel<TI, TQ, TC, HALF>, dim3(nx, ny), ROPE_THREADS, 0, st, p);
}

template <typename TI, typename TQ, typename TC>
cudaError_t launch3(RopeParams &p, bool half, bool vec, long long n, int sms, cudaStream_t st)
{
    return half ? launch4<TI, TQ, TC, true>(p, vec, n, sms, st) : launch4<TI, TQ, TC, false>(p, vec, n, sms, st);
}

template <typename TI, typename TQ>
cudaError_t launch2(RopeParams &p, qgemv_dtype cache, bool half, bool vec, long long n, int sms, cudaStream_t st)
{
    return cache == QGEMV_F16 ? launch3<TI, TQ, __half>(p, half, vec, n, sms, st)
                              : launch3<TI, TQ, __nv_bfloat16>(p, half, vec, n, sms, st);
}

template <typename TI>
cudaError_t launch1(RopeParams &p, qgemv_dtype qo, qgemv_dtype cache, bool half, bool vec, long long n, int sms,
                    cudaStream_t st)
{
    switch (qo) {
    case QGEMV_F32: return launch2<TI, float>(p, cache, half, vec, n, sms, st);
    case QGEMV_F16: return launch2<TI, __half>(p, cache, half, vec, n, sms, st);
    default: return launch2<TI, __nv_bfloat16>(p, cache, half, vec, n, sms, st);
    }
}

}  // namespace

cudaError_t launch_rope(RopeParams &p, qgemv_dtype in, qgemv_dtype q_out, qgemv_dtype cache, bool half_layout, bool vec,
                        long long n_tokens, int sms, cudaStream_t st)
{
    switch (in) {
    case QGEMV_F32: return launch1<float>(p, q_out, cache, half_layout, vec, n_tokens, sms, st);
    case QGEMV_F16: return launch1<__half>(p, q_out, cache, half_layout, vec, n_tokens, sms, st);
    default: return launch1<__nv_bfloat16>(p, q_out, cache, half_layout, vec, n_tokens, sms, st);
    }
}

}  // namespace qg
