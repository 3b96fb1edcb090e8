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
// the time between launches.  16122 tokens of 14 + 2 + 2 heads of 64, bf16:
// 20 us (memory alone: 11), bound by the wait for a token's loads.  Several
// tokens in a wide block instead of narrow blocks: 6168 of 16 + 2 + 2 heads of
// 128, f16, 15.7 us instead of 13.8, and 2 to 5 % on most other sizes.
#include "decode_ops.h"
#include "qgemv_internal.cuh"
#include "rope_util.cuh"

namespace qg {
namespace {

constexpr int ROPE_THREADS = 128;
// Heads in flight per thread: 96 bytes of loads, whatever the type.  With three
// of 16 bits 6168 tokens of 16 + 2 + 2 heads of 128 take 18.0 us, with six 13.8.
template <typename T>
constexpr int ROPE_UNROLL = sizeof(T) == 4 ? 3 : 6;

// Eight elements of a head a thread: unit j < rot / 8 is four pairs (HALF:
// elements 4j.. and rot/2 + 4j..; interleaved: 8j..), later units are copied.
template <typename TI, typename TQ, typename TC, bool HALF>
__global__ void __launch_bounds__(ROPE_THREADS, 8) rope_vec_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ __align__(16) float s_c[128], s_s[128];
    constexpr int UNROLL = ROPE_UNROLL<TI>;
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
    for (int h0 = hb + p.heads_per_block * static_cast<int>(blockIdx.y); h0 < heads || !have; h0 += UNROLL * step) {
        Four<TI> x[UNROLL], y[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int h = h0 + u * step;
            const TI *src = h < heads ? head_src<TI>(p, t, h, row_off >= 0) : nullptr;
            if (src) load8<TI, HALF>(src, a, b, x[u], y[u]);
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
        for (int u = 0; u < UNROLL; ++u) {
            const int h = h0 + u * step;
            if (h >= heads || (h >= p.hq && row_off < 0)) break;  // the heads that follow have no row either
            float fx[4], fy[4];
            unpack(x[u], fx);
            unpack(y[u], fy);
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
                store8<TQ, HALF>(q_dst<TQ>(p, t, h), a, b, fx, fy);
            else
                store8<TC, HALF>(kv_dst<TC>(p, h, row_off), a, b, fx, fy);
        }
    }
}

// One pair of a head a thread, any alignment and even sizes.  Bound by its
// instructions: a sine for every pair of every head, and accesses of one element.
// 16384 tokens of 32 + 8 + 8 heads of 128, fp32, take 361 us (the bytes alone 90),
// 16122 of 14 + 2 + 2 of 64, bf16, 75 (11); one token 2.0, as with wide accesses.
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
        // Many tokens: a block no wider than its heads fill, the same in each of
        // its turns, and more blocks beside it: 16122 tokens of 14 + 2 + 2 heads
        // of 64, bf16, 33.6 -> 20 us; 6168 of 16 + 2 + 2 of 128, f16, 17.6 ->
        // 13.8.  Tokens for fewer than ten blocks a multiprocessor keep wide
        // ones: 1277 of 12 + 2 + 2 of 128, bf16, 5.1 us instead of 5.9.
        constexpr int U = ROPE_UNROLL<TI>;
        if (n >= 10ll * sms) {
            const int turns = (heads + U * p.heads_per_block - 1) / (U * p.heads_per_block);
            p.heads_per_block = (heads + U * turns - 1) / (U * turns);
        }
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
