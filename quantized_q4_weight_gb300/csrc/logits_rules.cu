// logits_rules.cu -- penalties for repeated tokens, biases and grammar masks
// on logits, with the argmax of the result (minfer README "How it works":
// device-side argmax; the rules come between the lm_head and that argmax).
//
// Per row, with c the token's count in the row's history:
//   x = c > 0 ? (x > 0 ? x / rep : x * rep) : x;  x -= freq * c;
//   x -= pres * [c > 0];  x += bias;  x = -inf where the mask's bit is 0.
//
// A block takes a slice of one row's vocabulary.  The tokens that a history
// or a bias list touches are few: one bit a token (touched by either list or
// not) tells the logits' stream which they are, and a word in shared memory
// holds a token's count (bits 0..19) and 1 + the entry of the bias list that
// names it (from bit 20; raised first, by atomicMax: the last entry counts;
// then atomicAdd of the counts).  All of that is integer arithmetic, so the
// order in which threads run changes nothing.  The words are cleared while the
// preceding kernel drains.  The logits stream through once, 16 bytes a load,
// four or eight mask and touched bits at a time; the first ones are loaded
// before the lists.
//
// What bounds it: memory for many rows (logits read and written once); for
// one row, the latency of the chain launch, lists, logits, merge, which is why
// few rows have small slices (as few as 1024 tokens).  Many rows have slices
// of 8192, since every slice reads its row's whole lists before it can begin.
// 192 rows of 151936 fp32, histories up to 2048, 64 biases, masked, written:
// 55 us, 4.3 TB/s (a copy of the logits takes 37); 48 without lists and mask.
// 1 row 4.6 us, 5 rows of 50257 bf16, histories up to 2000, 6.8 us.
// Tried there and slower: slices of 4096 (69) or 16384 tokens, more loads in
// flight per thread (58), contiguous ranges per block with words at the rank
// of the touched bits and the logits from a ring of bulk copies (70), the same
// with warps that prepare the next 4096 tokens' lists (98), touched tokens
// taken after the stream instead of in it (85).  The barriers and dependent
// loads that these need cost more than the beginnings of blocks they save.
#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int LG_THREADS = 256;
constexpr int LG_SLICE_MAX = 8192;   // 32 KB of words: six blocks per multiprocessor
constexpr unsigned LG_COUNT_MASK = (1u << 20) - 1;
constexpr int LG_SLICE_MIN = 1024;   // one 16-byte load of fp32 a thread
constexpr int LG_BATCH = 4;          // list entries in flight per thread

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

// Rules of a row.
struct RowRules {
    float rep, freq, pres;
    const float *bias;

    __device__ __forceinline__ RowRules(const LogitsParams &p, long long r)
        : rep(p.rep ? __ldg(p.rep + r) : 1.0f), freq(p.freq ? __ldg(p.freq + r) : 0.0f),
          pres(p.pres ? __ldg(p.pres + r) : 0.0f), bias(p.bias + r * p.bias_stride)
    {
    }
    // a touched token's logit: c occurrences, b = 1 + its entry of the bias list (0: none)
    __device__ __forceinline__ float operator()(float v, unsigned c, unsigned b) const
    {
        if (c) {
            v = v > 0.0f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
            v = __fsub_rn(v, __fmul_rn(freq, static_cast<float>(c)));
            v = __fsub_rn(v, pres);
        }
        return b ? __fadd_rn(v, __ldg(bias + (b - 1))) : v;
    }
};

// A thread's best result so far: the lowest token among the largest.
struct Best {
    float v = -INFINITY;
    int t = 0;

    // tokens t0 .. t0 + E - 1, later than all before
    template <int E>
    __device__ __forceinline__ void take(const float (&f)[E], int t0)
    {
        float top = f[0];
#pragma unroll
        for (int e = 1; e < E; ++e) top = fmaxf(top, f[e]);  // passes NaN over
        if (top > v) {
            v = top;
            int first = E - 1;
#pragma unroll
            for (int e = E - 2; e >= 0; --e) first = f[e] == top ? e : first;
            t = t0 + first;
        }
    }
    __device__ __forceinline__ void take1(float f, int at)
    {
        if (f > v || (f == v && at < t && v > -INFINITY)) {
            v = f;
            t = at;
        }
    }
    // A key orders by value, then by the lower token; 0 stands for none.
    __device__ __forceinline__ unsigned long long key() const
    {
        return v > -INFINITY ? static_cast<unsigned long long>(ordered(v + 0.0f)) << 32 |
                                   (0xFFFFFFFFu - static_cast<unsigned>(t))
                             : 0;
    }
};

// The largest key of a warp.
__device__ __forceinline__ unsigned long long warp_best(unsigned long long key)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
        key = o > key ? o : key;
    }
    return key;
}

// One thread: a slice of row r has the best `key`; the last of the row's
// slices writes the result.  Maxima do not depend on the order.
__device__ __forceinline__ void merge_row(const LogitsParams &p, long long r, unsigned long long key, unsigned slices)
{
    if (slices > 1) {
        if (key) atomicMax(&p.keys[r], key);
        __threadfence();
        if (atomicAdd(&p.cnt[r], 1u) + 1 < slices) return;
        __threadfence();
        key = atomicExch(&p.keys[r], 0ull);  // both words are zero again
        p.cnt[r] = 0;
    }
    p.idx[r] = key ? static_cast<long long>(0xFFFFFFFFu - static_cast<unsigned>(key)) : -1;
    p.val[r] = key ? from_ordered(static_cast<unsigned>(key >> 32)) : -INFINITY;
}

// A list's length within its bound; a length outside is recorded.
__device__ __forceinline__ int bounded(int n, int most, unsigned *status, bool record)
{
    if (n < 0 || n > most) {
        if (record) atomicCAS(status, 0u, ST_BAD_ID);
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
    unsigned *words = lg_smem;              // [slice] count, and 1 + the bias list's entry from bit 20 on
    unsigned *touched = lg_smem + p.slice;  // [slice / 32]
    const int tid = threadIdx.x;
    const long long r = blockIdx.y;

    const int clear = p.slice + p.slice / 32;
    for (int i = tid; i < clear / 4; i += LG_THREADS) reinterpret_cast<uint4 *>(lg_smem)[i] = make_uint4(0, 0, 0, 0);
    for (int i = clear / 4 * 4 + tid; i < clear; i += LG_THREADS) lg_smem[i] = 0;
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
    // chunk of the row and the last may not.  A slice is counted in 32 bits
    // from t0.
    const uint32_t *mask = p.mask ? p.mask + r * p.mask_stride : nullptr;
    const int tokens = static_cast<int>(t1 - t0);  // below 0 for a slice past the row
    const int c_lo = t0 < 0 ? 1 : 0, c_hi = tokens < 0 ? 0 : tokens / E;
    const Chunk<T> *xc = reinterpret_cast<const Chunk<T> *>(x + t0);
    const int bit0 = static_cast<int>(t0);  // a token's mask bit is bit0 + its place
    Chunk<T> in;
    unsigned allow = 0;
    auto fetch = [&](int ch) {
        if (ch >= c_hi || ch < c_lo) return;
        in = ld_stream(xc + ch);
        allow = 0xFFFFFFFFu;
        if (mask) {
            const int bit = bit0 + ch * E;
            allow = __ldg(mask + (bit >> 5)) >> (bit & 31);
            // a chunk of a row that is not aligned may run into the next word
            if ((bit & 31) + E > 32) allow |= __ldg(mask + (bit >> 5) + 1) << (32 - (bit & 31));
        }
    };
    const int len_h = p.hist ? __ldg(p.hist_len + r) : 0, len_b = p.bias ? __ldg(p.bias_len + r) : 0;
    fetch(tid);
    const int nh = bounded(len_h, p.max_hist, p.status, tid == 0), nb = bounded(len_b, p.max_bias, p.status, tid == 0);
    const long long *hist = p.hist + r * p.hist_stride;
    const long long *bid = p.bias_ids + r * p.bias_stride;
    const RowRules rules(p, r);
    const long long lo = max(t0, 0ll);

    __syncthreads();
    auto place = [&](long long t) {  // the token's place in the slice, marked as touched; -1 for others
        if (t < lo || t >= t1) return -1;
        const int l = static_cast<int>(t) - bit0;
        atomicOr(&touched[l >> 5], 1u << (l & 31));
        return l;
    };
    if (nb) {
        for (int i = tid; i < nb; i += LG_THREADS) {
            const int l = place(__ldg(bid + i));
            if (l >= 0) atomicMax(&words[l], static_cast<unsigned>(i + 1) << 20);
        }
        __syncthreads();
    }
    for (int i0 = tid; i0 < nh; i0 += LG_BATCH * LG_THREADS) {
        long long t[LG_BATCH];
#pragma unroll
        for (int k = 0; k < LG_BATCH; ++k) t[k] = i0 + k * LG_THREADS < nh ? __ldg(hist + i0 + k * LG_THREADS) : -1;
#pragma unroll
        for (int k = 0; k < LG_BATCH; ++k) {
            const int l = place(t[k]);
            if (l >= 0) atomicAdd(&words[l], 1u);
        }
    }
    __syncthreads();

    auto rule = [&](float v, int l) { return rules(v, words[l] & LG_COUNT_MASK, words[l] >> 20); };

    // The next kernel may come from here on.  (Let in at the start, its blocks
    // clear their words and wait between this one's lists: 1 row 5.9 us a call
    // in a stream instead of 4.6.)
    pdl_launch_dependents();
    const float NEG = __int_as_float(0xFF800000);
    Best best;
    Chunk<T> *oc = reinterpret_cast<Chunk<T> *>(out + t0);
    for (int ch = tid; ch < c_hi; ch += LG_THREADS) {
        if (ch != tid) fetch(ch);
        if (ch < c_lo) continue;
        const int l0 = ch * E;
        const unsigned hit = touched[l0 >> 5] >> (l0 & 31) & ((1u << E) - 1);
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = lg_to_f(in.e[e]);
        for (unsigned rest = hit; rest; rest &= rest - 1) {  // one at a time: the rule's code once
            const int at = __ffs(rest) - 1;
            float v = f[0];
#pragma unroll
            for (int e = 1; e < E; ++e) v = e == at ? f[e] : v;
            v = rule(v, l0 + at);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = e == at ? v : f[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (!(allow >> e & 1)) f[e] = NEG;
        best.take<E>(f, bit0 + l0);
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
    // the row's ends, a token a thread
    auto single = [&](int l) {
        float f = lg_to_f(x[t0 + l]);
        if (touched[l >> 5] >> (l & 31) & 1) f = rule(f, l);
        const int bit = bit0 + l;
        if (mask && !(__ldg(mask + (bit >> 5)) >> (bit & 31) & 1)) f = NEG;
        best.take1(f, bit0 + l);
        if (out) lg_from_f(out[t0 + l], f);
    };
    if (c_lo && tid < min(E, tokens) && t0 + tid >= 0) single(tid);
    if (tokens > 0 && c_hi >= c_lo && tid < tokens - c_hi * E) single(c_hi * E + tid);
    if (!p.idx) return;

    unsigned long long key = warp_best(best.key());
    if ((tid & 31) == 0) s_best[tid >> 5] = key;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < LG_THREADS / 32; ++w) key = s_best[w] > key ? s_best[w] : key;
        merge_row(p, r, key, gridDim.x);
    }
}

template <typename T>
cudaError_t launch_t(LogitsParams &p, int rows, int sms, cudaStream_t st)
{
    // About two blocks per multiprocessor in all, within the bounds above.  A
    // row that does not start on 16 bytes has one chunk more.
    const long long span = p.vocab + 16 / sizeof(T) - 1;
    const long long want = (2ll * sms + rows - 1) / rows;
    const long long slice = ((span + want - 1) / want + 31) / 32 * 32;
    p.slice = static_cast<int>(slice < LG_SLICE_MIN ? LG_SLICE_MIN : slice > LG_SLICE_MAX ? LG_SLICE_MAX : slice);
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(logits_kernel<T>), 4 * LG_SLICE_MAX + LG_SLICE_MAX / 8,
                                     done);
    if (e != cudaSuccess) return e;
    return launch_pdl(logits_kernel<T>, dim3(static_cast<unsigned>((span + p.slice - 1) / p.slice), rows), LG_THREADS,
                      static_cast<size_t>(4 * p.slice + p.slice / 8), st, p);
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
