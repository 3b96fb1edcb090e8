// norm_rope.cu -- norms of q and k head by head, the rotary positions and the
// write into the cache in one pass (minfer README "How it works": RoPE between
// the QKV product and the attention).
//
//   y = x / sqrt(mean x^2 + eps) * w over a head, then the pairs' rotation
// (rope_kv.cu has the angles).  A head's elements lie in the registers of a group
// of lanes (a power of two of them, eight elements each, chosen so that a thread
// has both elements of its pairs), the sum of squares is a few shuffles, and norm,
// rotation and rounding follow without another look at memory.
//
// What bounds it: memory for prompts (each element read and written once: 16381 tokens of
// 32 + 8 + 8 heads of 128, fp32 to f16, 96 us, 6.3 TB/s; 16 bits to 16 bits 78 us, 5.2 TB/s;
// without a cache, fp32 to bf16 and fp32, 85 us, 6.3 TB/s), launch and load latency for a
// few tokens (8 of 16 + 2 + 2 heads 2.75 us).  As in rope_kv.cu a block takes one token and
// its threads walk the heads with several heads' loads in flight, while the token's
// sines are formed once; few tokens spread their heads over blocks.
#include "kv8_ops.h"
#include "qgemv_internal.cuh"
#include "rope_util.cuh"

namespace qg {
namespace {

// MANY tokens: blocks of 64 threads, 96 bytes of loads in flight for each.  16381 of
// 32 + 8 + 8 heads of 128, fp32: 96 us; with 128 threads 102, and 106 with 64 bytes in
// flight (three quarters as many multiprocessor's threads 111).  Few tokens: 128 threads and
// 64 bytes, 2.7 us instead of 3.0 for eight tokens.  All of these are of fp32 inputs.
template <bool MANY>
constexpr int NR_THREADS = MANY ? 64 : 128;
template <typename T, bool MANY>
constexpr int NR_UNROLL = sizeof(T) == 4 ? (MANY ? 3 : 2) : 4;  // heads (six of 16 bits do not fit the registers)
constexpr int NR_ANY = 128;  // threads of the element-wise kernel

// Where token t's k goes, in elements from r.ck (and its v from r.cv): its cache
// row, -1 for none; without a cache, its place in k_out.
__device__ __forceinline__ long long k_row(const RopeParams &r, long long t)
{
    return r.slots ? cache_row(r, t) : t * r.row_stride;
}

// Eight elements of a head a thread (rope_kv.cu: which eight) as four pairs; a head is
// `lanes` threads, a power of two, those beyond its units idle.  With r = 1 / sqrt(mean
// x^2 + eps) a pair becomes r (x wx c - y wy s), r (x wx s + y wy c): the products of
// weights and sines are formed once for the q heads and once for the k heads of a
// thread (elements that do not rotate: c = 1, s = 0).
template <typename TI, typename TQ, typename TC, bool HALF, bool MANY>
__global__ void __launch_bounds__(NR_THREADS<MANY>, MANY ? 16 : 8) norm_rope_vec_kernel(const __grid_constant__ NormRopeParams p, int lanes)
{
    __shared__ __align__(16) float s_c[128], s_s[128];
    constexpr int UNROLL = NR_UNROLL<TI, MANY>;
    const RopeParams &r = p.r;
    pdl_launch_dependents();
    const int j = static_cast<int>(threadIdx.x) & (lanes - 1), hb = static_cast<int>(threadIdx.x) / lanes;
    const int at_once = NR_THREADS<MANY> / lanes;
    const long long t = blockIdx.x;
    const int normed = r.hq + r.hkv, heads = normed + p.v_heads;
    const bool mine = 8 * j < r.d, rot_unit = 8 * j < r.rot;
    const int a = HALF && rot_unit ? 4 * j : 8 * j;                  // first four elements
    const int b = HALF && rot_unit ? r.rot / 2 + 4 * j : 8 * j + 4;  // second four
    pdl_wait();
    const int pos = __ldg(r.pos + t);
    const long long row_off = r.hkv ? k_row(r, t) : -1;
    const TI *q_at = static_cast<const TI *>(r.q) + t * r.q_stride, *k_at = static_cast<const TI *>(r.k) + t * r.k_stride;
    const TI *v_at = static_cast<const TI *>(r.v) + t * r.v_stride;
    const float per = 1.0f / static_cast<float>(r.d);
    float xc[4], ys[4], xs[4], yc[4];  // wx c, wy s, wx s, wy c
    const float *formed = nullptr;     // of these weights
    bool have = false;
    const int step = at_once * static_cast<int>(gridDim.y);
    // all threads of the block take the same turns: shuffles and a barrier lie in them
    for (int base = at_once * static_cast<int>(blockIdx.y); base < heads; base += UNROLL * step) {
        Four<TI> x[UNROLL], y[UNROLL];
        bool there[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int h = base + hb + u * step;
            there[u] = false;
            if (!mine) continue;
            if (h < r.hq) {  // not behind the slot's load
                load8<TI, HALF>(q_at + h * r.d, a, b, x[u], y[u]);
                there[u] = true;
            } else if (h < heads && row_off >= 0) {
                load8<TI, HALF>(h < normed ? k_at + (h - r.hq) * r.d : v_at + (h - normed) * r.d, a, b, x[u], y[u]);
                there[u] = true;
            }
        }
        if (!have) {
            for (int i = threadIdx.x; i < r.rot / 2; i += NR_THREADS<MANY>) angle(pos, r.turns[i], r.mscale, s_c[i], s_s[i]);
            __syncthreads();
            have = true;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int h = base + hb + u * step;
            float fx[4] = {}, fy[4] = {};
            if (there[u]) {
                unpack(x[u], fx);
                unpack(y[u], fy);
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = fmaf(fx[i], fx[i], fmaf(fy[i], fy[i], sum));
#pragma unroll
            for (int o = 16; o; o >>= 1)
                if (o < lanes) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (!there[u]) continue;
            if (h < normed) {
                const float *w = h < r.hq ? p.q_weight : p.k_weight;
                if (w != formed) {
                    formed = w;
                    float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {};
                    if (rot_unit) {
                        const float4 cc = *reinterpret_cast<const float4 *>(s_c + 4 * j);
                        const float4 ss = *reinterpret_cast<const float4 *>(s_s + 4 * j);
                        c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
                        s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float wx = __ldg(w + (HALF ? a + i : 8 * j + 2 * i)), wy = __ldg(w + (HALF ? b + i : 8 * j + 2 * i + 1));
                        xc[i] = wx * c[i], ys[i] = wy * s[i], xs[i] = wx * s[i], yc[i] = wy * c[i];
                    }
                }
                const float by = rsqrtf(fmaf(sum, per, p.eps));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // pair i: (fx[i], fy[i]), interleaved two neighbours
                    float &u0 = HALF ? fx[i] : i < 2 ? fx[2 * i & 3] : fy[2 * i & 3];
                    float &u1 = HALF ? fy[i] : i < 2 ? fx[(2 * i + 1) & 3] : fy[(2 * i + 1) & 3];
                    const float px = u0 * by, py = u1 * by;
                    u0 = px * xc[i] - py * ys[i];
                    u1 = px * xs[i] + py * yc[i];
                }
            }
            if (h < r.hq)
                store8<TQ, HALF>(q_dst<TQ>(r, t, h), a, b, fx, fy);
            else
                store8<TC, HALF>(kv_dst<TC>(r, h, row_off), a, b, fx, fy);
        }
    }
}

// A warp a head, element by element: any alignment and even sizes up to 256.
template <typename TI, typename TQ, typename TC, bool HALF>
__global__ void __launch_bounds__(NR_ANY) norm_rope_any_kernel(const __grid_constant__ NormRopeParams p)
{
    const RopeParams &r = p.r;
    pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x;
    const int lane = threadIdx.x & 31, warps = NR_ANY / 32 * static_cast<int>(gridDim.y);
    const int normed = r.hq + r.hkv, heads = normed + p.v_heads, pairs = r.d >> 1, rpairs = r.rot >> 1;
    const long long row_off = r.hkv ? k_row(r, t) : -1;
    const int pos = __ldg(r.pos + t);
    for (int h = static_cast<int>(blockIdx.y * (NR_ANY / 32) + threadIdx.x / 32); h < heads; h += warps) {
        const TI *src = head_src<TI>(r, t, h, row_off >= 0);
        if (!src) continue;  // the whole warp
        float x[4] = {}, y[4] = {}, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = lane + 32 * k;
            if (j >= pairs) continue;
            const bool rot_pair = j < rpairs;
            x[k] = to_f(src[HALF && rot_pair ? j : 2 * j]);
            y[k] = to_f(src[HALF && rot_pair ? rpairs + j : 2 * j + 1]);
            sum = fmaf(x[k], x[k], fmaf(y[k], y[k], sum));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float by = rsqrtf(fmaf(sum, 1.0f / static_cast<float>(r.d), p.eps));
        const float *w = h < r.hq ? p.q_weight : p.k_weight;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = lane + 32 * k;
            if (j >= pairs) continue;
            const bool rot_pair = j < rpairs;
            const int a = HALF && rot_pair ? j : 2 * j, b = HALF && rot_pair ? rpairs + j : 2 * j + 1;
            float u = x[k], v = y[k];
            if (h < normed) {
                u *= by * __ldg(w + a);
                v *= by * __ldg(w + b);
                if (rot_pair) {
                    float c, s;
                    angle(pos, r.turns[j], r.mscale, c, s);
                    const float pu = u, pv = v;
                    u = pu * c - pv * s;
                    v = pu * s + pv * c;
                }
            }
            if (h < r.hq) {
                TQ *dst = q_dst<TQ>(r, t, h);
                dst[a] = from_f<TQ>(u);
                dst[b] = from_f<TQ>(v);
            } else {
                TC *dst = kv_dst<TC>(r, h, row_off);
                dst[a] = from_f<TC>(u);
                dst[b] = from_f<TC>(v);
            }
        }
    }
}

template <typename TI, typename TQ, typename TC, bool HALF>
cudaError_t launch4(NormRopeParams &p, bool vec, long long n, int sms, cudaStream_t st)
{
    const int heads = p.r.hq + p.r.hkv + p.v_heads;
    const unsigned nx = static_cast<unsigned>(n);
    int lanes = 32;
    if (vec)
        while (lanes > 1 && (lanes >> 1) * 8 >= p.r.d) lanes >>= 1;
    if (vec && n >= 10ll * sms)
        return launch_pdl(norm_rope_vec_kernel<TI, TQ, TC, HALF, true>, dim3(nx), NR_THREADS<true>, 0, st, p, lanes);
    const int at_once = NR_ANY / lanes, chunks = (heads + at_once - 1) / at_once;
    // blocks that share a token repeat its sines; they pay while the tokens alone leave multiprocessors idle
    const unsigned ny = static_cast<unsigned>(n * chunks <= 2ll * sms ? chunks : 1);
    if (vec)
        return launch_pdl(norm_rope_vec_kernel<TI, TQ, TC, HALF, false>, dim3(nx, ny), NR_THREADS<false>, 0, st, p, lanes);
    return launch_pdl(norm_rope_any_kernel<TI, TQ, TC, HALF>, dim3(nx, ny), NR_ANY, 0, st, p);
}

template <typename TI, typename TQ, typename TC>
cudaError_t launch3(NormRopeParams &p, bool half, bool vec, long long n, int sms, cudaStream_t st)
{
    return half ? launch4<TI, TQ, TC, true>(p, vec, n, sms, st) : launch4<TI, TQ, TC, false>(p, vec, n, sms, st);
}

template <typename TI, typename TQ>
cudaError_t launch2(NormRopeParams &p, qgemv_dtype k_out, bool half, bool vec, long long n, int sms, cudaStream_t st)
{
    if (k_out == QGEMV_F32) return launch3<TI, TQ, float>(p, half, vec, n, sms, st);
    return k_out == QGEMV_F16 ? launch3<TI, TQ, __half>(p, half, vec, n, sms, st)
                              : launch3<TI, TQ, __nv_bfloat16>(p, half, vec, n, sms, st);
}

template <typename TI>
cudaError_t launch1(NormRopeParams &p, qgemv_dtype qo, qgemv_dtype k_out, bool half, bool vec, long long n, int sms,
                    cudaStream_t st)
{
    switch (qo) {
    case QGEMV_F32: return launch2<TI, float>(p, k_out, half, vec, n, sms, st);
    case QGEMV_F16: return launch2<TI, __half>(p, k_out, half, vec, n, sms, st);
    default: return launch2<TI, __nv_bfloat16>(p, k_out, half, vec, n, sms, st);
    }
}

}  // namespace

cudaError_t launch_norm_rope(NormRopeParams &p, qgemv_dtype in, qgemv_dtype q_out, qgemv_dtype k_out, bool half_layout,
                             bool vec, long long n_tokens, int sms, cudaStream_t st)
{
    switch (in) {
    case QGEMV_F32: return launch1<float>(p, q_out, k_out, half_layout, vec, n_tokens, sms, st);
    case QGEMV_F16: return launch1<__half>(p, q_out, k_out, half_layout, vec, n_tokens, sms, st);
    default: return launch1<__nv_bfloat16>(p, q_out, k_out, half_layout, vec, n_tokens, sms, st);
    }
}

}  // namespace qg
