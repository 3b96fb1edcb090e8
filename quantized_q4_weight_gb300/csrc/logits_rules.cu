// logits_rules.cu -- penalties for repeated tokens, biases and grammar masks
// on logits, with the argmax of the result (minfer README "How it works":
// device-side argmax; the rules come between the lm_head and that argmax).
//
// Per row, with c the token's count in the row's history:
//   x = c > 0 ? (x > 0 ? x / rep : x * rep) : x;  x -= freq * c;
//   x -= pres * [c > 0];  x += bias;  x = -inf where the mask's bit is 0.
//
// A block takes a slice of one row's vocabulary.  The tokens that a history
// or a bias list touches are few, so the block keeps one bit per token of
// its slice (touched or not) and one 32-bit word for the touched ones:
//   bits 0..19: the count c;  bits 20..31: 1 + the entry of the bias list.
// The words are never cleared as a whole: a first pass over the two lists
// sets a token's bit and zeroes its word, a second one raises the words
// (atomicMax of the bias entry: the last entry counts; then atomicAdd of
// the counts).  All of that is integer arithmetic, so the order in which
// threads run changes nothing.  Then the logits stream through once, 16
// bytes a load, four or eight mask and touched bits at a time.
//
// What bounds it: memory for many rows (logits read and written once); for
// one row, the latency of the chain launch, lists, logits, merge, which is
// why the slices get small then.  Every slice reads its row's whole lists
// (from L2); slices of 16384 tokens keep that under a tenth of the row's
// own bytes for histories of a thousand tokens.
#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int LG_THREADS = 256;
constexpr int LG_SLICE_MAX = 8192;   // 32 KB of words: six blocks per multiprocessor
constexpr int LG_SLICE_MIN = 1024;   // one 16-byte load of fp32 a thread
constexpr int LG_AHEAD = 1;          // chunks in flight per thread
constexpr int LG_KEEP = 4;           // list entries kept per thread: 1024 of a row's
constexpr unsigned LG_COUNT_MASK = (1u << 20) - 1;

__device__ __forceinline__ float lg_to_f(float v) { return v; }
__device__ __forceinline__ float lg_to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float lg_to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void lg_from_f(float &o, float v) { o = v; }
__device__ __forceinline__ void lg_from_f(__half &o, float v) { o = __float2half_rn(v); }
__device__ __forceinline__ void lg_from_f(__nv_bfloat16 &o, float v) { o = __float2bfloat16_rn(v); }

// A float's bits in an order that unsigned comparison respects.
__device__ __forceinline__ unsigned ordered(float f)
{
    const unsigned u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(unsigned o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

template <typename T>
struct alignas(16) Chunk {
    T e[16 / sizeof(T)];
};

// A chunk that is read once (it may be written in place, so not through the
// read-only path).
template <typename T>
__device__ __forceinline__ Chunk<T> ld_stream(const Chunk<T> *a)
{
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(a));
    Chunk<T> c;
    memcpy(&c, &v, 16);
    return c;
}

template <typename T>
__device__ __forceinline__ uint4 as_uint4(const Chunk<T> &c)
{
    uint4 v;
    memcpy(&v, &c, 16);
    return v;
}

// A list's length within its bound; a length outside is recorded.
__device__ __forceinline__ int bounded(int n, int most, unsigned *status)
{
    if (n < 0 || n > most) {
        if (threadIdx.x == 0) atomicCAS(status, 0u, ST_BAD_ID);
        return n < 0 ? 0 : most;
    }
    return n;
}

template <typename T>
__global__ void __launch_bounds__(LG_THREADS, 6) logits_kernel(const __grid_constant__ LogitsParams p)
{
    constexpr int E = 16 / sizeof(T);
    extern __shared__ __align__(16) unsigned lg_smem[];
    __shared__ unsigned long long s_best[LG_THREADS / 32];
    unsigned *words = lg_smem;                  // [slice]
    unsigned *touched = lg_smem + p.slice;      // [slice / 32]
    const int tid = threadIdx.x;
    const long long r = blockIdx.y;

    pdl_launch_dependents();
    for (int i = tid; i < p.slice / 32; i += LG_THREADS) touched[i] = 0;
    pdl_wait();

    const T *x = static_cast<const T *>(p.x) + r * p.x_stride;
    T *out = p.out ? static_cast<T *>(p.out) + r * p.out_stride : nullptr;
    // The row in 16-byte chunks of memory: chunk c holds tokens c E - shift ..
    // + E - 1.  The slice is a range of chunks, its first token t0 (the
    // first chunk's tokens below 0 and the last one's from vocab on are not
    // there: such chunks go element by element).
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const bool out_vec = out && (reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T) == static_cast<unsigned>(shift);
    const long long t0 = static_cast<long long>(blockIdx.x) * p.slice - shift;
    const long long t1 = min(p.vocab, t0 + p.slice);

    // Chunks [c_lo, c_hi) of the slice lie in the row as a whole; the first
    // chunk of the row and the last may not.  They go LG_AHEAD at a time, their
    // loads and mask words first; the first ones are on their way while the
    // lists are read.  A slice is counted in 32 bits from t0.
    const uint32_t *mask = p.mask ? p.mask + r * p.mask_stride : nullptr;
    const int tokens = static_cast<int>(t1 - t0);  // below 0 for a slice past the row
    const int c_lo = t0 < 0 ? 1 : 0, c_hi = tokens < 0 ? 0 : tokens / E;
    const Chunk<T> *xc = reinterpret_cast<const Chunk<T> *>(x + t0);
    const int bit0 = static_cast<int>(t0);  // a token's mask bit is bit0 + its place
    Chunk<T> in[LG_AHEAD];
    unsigned allow[LG_AHEAD];
    auto fetch = [&](int ch0) {
#pragma unroll
        for (int u = 0; u < LG_AHEAD; ++u) {
            const int ch = ch0 + u * LG_THREADS;
            allow[u] = 0xFFFFFFFFu;
            if (ch < c_hi && ch >= c_lo) {
                in[u] = ld_stream(xc + ch);
                if (mask) {
                    const int bit = bit0 + ch * E;
                    allow[u] = __ldg(mask + (bit >> 5)) >> (bit & 31);
                    // a chunk of a row that is not aligned may run into the next word
                    if ((bit & 31) + E > 32) allow[u] |= __ldg(mask + (bit >> 5) + 1) << (32 - (bit & 31));
                }
            }
        }
    };
    const int len_h = p.hist ? __ldg(p.hist_len + r) : 0, len_b = p.bias ? __ldg(p.bias_len + r) : 0;
    fetch(tid);
    const int nh = bounded(len_h, p.max_hist, p.status), nb = bounded(len_b, p.max_bias, p.status);
    const long long *hist = p.hist + r * p.hist_stride;
    const long long *bid = p.bias_ids + r * p.bias_stride;
    const float *bias = p.bias + r * p.bias_stride;
    const float rep = p.rep ? __ldg(p.rep + r) : 1.0f;
    const float freq = p.freq ? __ldg(p.freq + r) : 0.0f;
    const float pres = p.pres ? __ldg(p.pres + r) : 0.0f;
    const long long lo = max(t0, 0ll);

    if (nh | nb) {
        // the lists' first entries stay in registers between the passes
        long long id[LG_KEEP];
#pragma unroll
        for (int u = 0; u < LG_KEEP; ++u) {
            const int i = tid + u * LG_THREADS;
            id[u] = i < nh ? __ldg(hist + i) : i < nh + nb ? __ldg(bid + (i - nh)) : -1;
        }
        __syncthreads();
        auto touch = [&](long long t) {
            if (t >= lo && t < t1) {
                const int l = static_cast<int>(t) - bit0;
                words[l] = 0;
                atomicOr(&touched[l >> 5], 1u << (l & 31));
            }
        };
#pragma unroll
        for (int u = 0; u < LG_KEEP; ++u) touch(id[u]);
        for (int i = tid + LG_KEEP * LG_THREADS; i < nh + nb; i += LG_THREADS)
            touch(i < nh ? __ldg(hist + i) : __ldg(bid + (i - nh)));
        __syncthreads();
        // a bias entry i of token t, then an occurrence of t
        auto entry = [&](long long t, int i) {
            if (t >= lo && t < t1) atomicMax(&words[t - t0], static_cast<unsigned>(i + 1) << 20);
        };
        auto occurs = [&](long long t) {
            if (t >= lo && t < t1) atomicAdd(&words[t - t0], 1u);
        };
        if (nb) {
#pragma unroll
            for (int u = 0; u < LG_KEEP; ++u)
                if (tid + u * LG_THREADS >= nh) entry(id[u], tid + u * LG_THREADS - nh);
            for (int i = tid + LG_KEEP * LG_THREADS; i < nh + nb; i += LG_THREADS)
                if (i >= nh) entry(__ldg(bid + (i - nh)), i - nh);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < LG_KEEP; ++u)
            if (tid + u * LG_THREADS < nh) occurs(id[u]);
        for (int i = tid + LG_KEEP * LG_THREADS; i < nh; i += LG_THREADS) occurs(__ldg(hist + i));
    }
    __syncthreads();

    auto rule = [&](float v, int l) {  // the touched token t0 + l
        const unsigned w = words[l], c = w & LG_COUNT_MASK, b = w >> 20;
        if (c) {
            v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
            v = __fsub_rn(v, __fmul_rn(freq, static_cast<float>(c)));
            v = __fsub_rn(v, pres);
        }
        return b ? __fadd_rn(v, __ldg(bias + (b - 1))) : v;
    };

    const float NEG = __int_as_float(0xFF800000);
    float best = NEG;
    int best_l = 0;
    Chunk<T> *oc = reinterpret_cast<Chunk<T> *>(out + t0);
    for (int ch0 = tid; ch0 < c_hi; ch0 += LG_AHEAD * LG_THREADS) {
        if (ch0 != tid) fetch(ch0);
#pragma unroll
        for (int u = 0; u < LG_AHEAD; ++u) {
            const int ch = ch0 + u * LG_THREADS;
            if (ch >= c_hi || ch < c_lo) continue;
            const int l0 = ch * E;
            const unsigned hit = touched[l0 >> 5] >> (l0 & 31) & ((1u << E) - 1);
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = lg_to_f(in[u].e[e]);
            if (hit) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (hit >> e & 1) f[e] = rule(f[e], l0 + e);
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!(allow[u] >> e & 1)) f[e] = NEG;
            float top = f[0];
#pragma unroll
            for (int e = 1; e < E; ++e) top = fmaxf(top, f[e]);  // passes NaN over
            if (top > best) {
                best = top;
                int first = E - 1;
#pragma unroll
                for (int e = E - 2; e >= 0; --e) first = f[e] == top ? e : first;
                best_l = l0 + first;
            }
            if (out) {
                Chunk<T> o;
#pragma unroll
                for (int e = 0; e < E; ++e) lg_from_f(o.e[e], f[e]);
                if (out_vec) {
                    __stcs(reinterpret_cast<uint4 *>(oc + ch), as_uint4(o));
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) out[t0 + l0 + e] = o.e[e];
                }
            }
        }
    }
    // the row's ends, a token a thread
    auto single = [&](int l) {
        float f = lg_to_f(x[t0 + l]);
        if (touched[l >> 5] >> (l & 31) & 1) f = rule(f, l);
        const int bit = bit0 + l;
        if (mask && !(__ldg(mask + (bit >> 5)) >> (bit & 31) & 1)) f = NEG;
        if (f > best || (f == best && l < best_l && best > NEG)) {
            best = f;
            best_l = l;
        }
        if (out) lg_from_f(out[t0 + l], f);
    };
    if (c_lo && tid < min(E, tokens) && t0 + tid >= 0) single(tid);
    if (tokens > 0 && c_hi >= c_lo && tid < tokens - c_hi * E) single(c_hi * E + tid);
    if (!p.idx) return;

    // The best of the block, then of the row: a key orders by value, then by
    // the lower token; 0 stands for none.  Maxima do not depend on the order.
    unsigned long long key = 0;
    if (best > NEG)
        key = static_cast<unsigned long long>(ordered(best + 0.0f)) << 32 | (0xFFFFFFFFu - static_cast<unsigned>(bit0 + best_l));
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
        key = o > key ? o : key;
    }
    if ((tid & 31) == 0) s_best[tid >> 5] = key;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < LG_THREADS / 32; ++w) key = s_best[w] > key ? s_best[w] : key;
        if (gridDim.x > 1) {
            if (key) atomicMax(&p.keys[r], key);
            __threadfence();
            if (atomicAdd(&p.cnt[r], 1u) + 1 < gridDim.x) return;
            __threadfence();
            key = atomicExch(&p.keys[r], 0ull);  // the last block: both words are zero again
            p.cnt[r] = 0;
        }
        p.idx[r] = key ? static_cast<long long>(0xFFFFFFFFu - static_cast<unsigned>(key)) : -1;
        p.val[r] = key ? from_ordered(static_cast<unsigned>(key >> 32)) : NEG;
    }
}

template <typename T>
cudaError_t launch_t(LogitsParams &p, int rows, int sms, cudaStream_t st)
{
    // Slices: about two blocks per multiprocessor in all, within the bounds
    // above.  A row that does not start on 16 bytes has one chunk more.
    const long long span = p.vocab + 16 / sizeof(T) - 1;
    long long want = (2ll * sms + rows - 1) / rows;
    long long slice = (span + want - 1) / want;
    slice = (slice + 31) / 32 * 32;
    slice = slice < LG_SLICE_MIN ? LG_SLICE_MIN : slice > LG_SLICE_MAX ? LG_SLICE_MAX : slice;
    p.slice = static_cast<int>(slice);
    const size_t smem = 4 * slice + slice / 8;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(logits_kernel<T>),
                                     4 * LG_SLICE_MAX + LG_SLICE_MAX / 8, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(logits_kernel<T>, dim3(static_cast<unsigned>((span + slice - 1) / slice), rows), LG_THREADS, smem,
                      st, p);
}

}  // namespace

cudaError_t launch_logits(LogitsParams &p, qgemv_dtype type, int rows, int sms, cudaStream_t st)
{
    switch (type) {
    case QGEMV_F32: return launch_t<float>(p, rows, sms, st);
    case QGEMV_F16: return launch_t<__half>(p, rows, sms, st);
    default: return launch_t<__nv_bfloat16>(p, rows, sms, st);
    }
}

}  // namespace qg
