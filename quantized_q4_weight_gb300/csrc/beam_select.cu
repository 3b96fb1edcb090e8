// beam_select.cu -- the best continuations of each beam search over its beams and
// the vocabulary (minfer README "How it works": device-side argmax; here of many).
//
//   s(r, t) = run[r] + x[r][t] - lse[r],  lse[r] = M + log(sum exp(x[r][t] - M))
// Within a row the order of s is that of x, so a block that streams a slice of a
// row needs no sum to find the slice's n best.  It leaves their keys in order, the
// slice's maximum and its sum of exponentials; the last block of a search to
// arrive joins them, forms s in 64 bits and takes the n best of all.  Nothing depends on
// which block that is.
//
// A key holds a logit's bits in an order that integers have, and the token upside
// down, so that a larger key is a larger logit or a lower token.  Each warp keeps the n
// best keys it has met in its lanes, in order.  A value is compared with the n-th of
// them (or a better n-th that another warp has shown), which few pass: those are
// collected in shared memory and inserted one by one, a ballot and a shuffle each.  The
// first values of a warp go by the n-th largest of the lanes' largest (a bitonic network
// of shuffles), a bound that lets few more than n through.
//
// What bounds it: memory for many rows (logits read once; a maximum, a product, an
// exponential and a sum for each); the chain launch, logits, insertions, arrival, join for
// one search, so few rows have small slices.
#include "kv8_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int BM_THREADS = 256, BM_WARPS = BM_THREADS / 32, BM_BLOCKS = 4;
constexpr int BM_CHUNKS = 4;   // 16-byte chunks of a thread's batch; as many are on their way
constexpr int BM_LIST = 64;    // keys of a warp that wait for their insertion
constexpr int BM_BEAMS = 16;
constexpr float LOG2E = 1.4426950408889634f;

typedef unsigned long long Key;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A float's bits in an order that unsigned comparison respects; -0 as +0.
__device__ __forceinline__ unsigned ordered(float f)
{
    const unsigned u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(unsigned o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(float v, unsigned token)
{
    return static_cast<Key>(ordered(v)) << 32 | (0xFFFFFFFFu - token);
}
__device__ __forceinline__ float value_of(Key k) { return from_ordered(static_cast<unsigned>(k >> 32)); }
__device__ __forceinline__ unsigned token_of(Key k) { return 0xFFFFFFFFu - static_cast<unsigned>(k); }

// Elements of a 16-byte chunk as floats, and the largest of them (NaN passed over).
template <typename T>
struct Chunk16;
template <>
struct Chunk16<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float at(const uint4 &w, int i)
    {
        return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
    }
    static __device__ __forceinline__ float largest(const uint4 &w)
    {
        return fmaxf(fmaxf(at(w, 0), at(w, 1)), fmaxf(at(w, 2), at(w, 3)));
    }
};
template <>
struct Chunk16<__half> {
    static constexpr int E = 8;
    static __device__ __forceinline__ __half2 pair(const uint4 &w, int i)
    {
        const unsigned u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        return *reinterpret_cast<const __half2 *>(&u);
    }
    static __device__ __forceinline__ float at(const uint4 &w, int i)
    {
        return i & 1 ? __high2float(pair(w, i >> 1)) : __low2float(pair(w, i >> 1));
    }
    static __device__ __forceinline__ float largest(const uint4 &w)
    {
        const __half2 m = __hmax2(__hmax2(pair(w, 0), pair(w, 1)), __hmax2(pair(w, 2), pair(w, 3)));
        return fmaxf(__low2float(m), __high2float(m));
    }
};
template <>
struct Chunk16<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ unsigned word(const uint4 &w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    static __device__ __forceinline__ __nv_bfloat162 pair(const uint4 &w, int i)
    {
        const unsigned u = word(w, i);
        return *reinterpret_cast<const __nv_bfloat162 *>(&u);
    }
    static __device__ __forceinline__ float at(const uint4 &w, int i)
    {
        return __uint_as_float(i & 1 ? word(w, i >> 1) & 0xFFFF0000u : word(w, i >> 1) << 16);
    }
    static __device__ __forceinline__ float largest(const uint4 &w)
    {
        const __nv_bfloat162 m = __hmax2(__hmax2(pair(w, 0), pair(w, 1)), __hmax2(pair(w, 2), pair(w, 3)));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

// The n-th largest of a warp's 32 values.
template <typename V>
__device__ __forceinline__ V nth_of_warp(V v, int n)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int d = k >> 1; d; d >>= 1) {
            const V o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
            const bool larger = ((lane & k) == 0) == ((lane & d) == 0);  // k = 32: falling over the warp
            v = (o > v) == larger ? o : v;
        }
    return __shfl_sync(0xFFFFFFFFu, v, n - 1);
}

// The warp's best keys, falling over the lanes (0: none).
struct Best {
    Key mine = 0;

    __device__ __forceinline__ void insert(Key k)  // the same for all lanes, none of the list's
    {
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, mine > k));
        const Key up = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
        const int lane = threadIdx.x & 31;
        mine = lane < at ? mine : lane == at ? k : up;
    }
    __device__ __forceinline__ Key nth(int n) const { return __shfl_sync(0xFFFFFFFFu, mine, n - 1); }
};

// How many of a falling list of `n` are above k.
template <typename K>
__device__ __forceinline__ int above(const K *list, int n, K k)
{
    int at = 0;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        if (at + d <= n && list[at + d - 1] > k) at += d;
    return at + (at < n && list[at] > k);
}

struct BeamShared {
    Key lists[BM_BEAMS][32];        // of the warps, then of the join's rows
    Key wait[BM_WARPS][BM_LIST];
    Key shown;                      // the best n-th key of a warp
    float m[BM_BEAMS], sum[BM_BEAMS];
    int count[BM_BEAMS];
    double lse[BM_BEAMS];
    int last;
};

// The join of group gi of the launch, by the block that arrived last.
__device__ void join(const BeamParams &p, int gi, BeamShared &s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r0 = static_cast<long long>(gi) * p.beams;
    const int per = p.slices * p.n_best;
    constexpr int ROWS = BM_BEAMS / BM_WARPS;  // of a warp
    Best best[ROWS];
    // each row's n best keys, maximum and sum
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        const int w = warp + q * BM_WARPS;
        if (w >= p.beams) break;
        const Key *part = p.part + (r0 + w) * per;
        const float2 *ml = p.part_ml + (r0 + w) * p.slices;
        float m = -INFINITY, sum = 0.0f;
        float2 mine = lane < p.slices ? ml[lane] : make_float2(-INFINITY, 0.0f);
        if (p.slices == 1) {
            best[q].mine = lane < p.n_best ? part[lane] : 0;
        } else {
            Key kth = 0;
            for (int i0 = 0; i0 < per; i0 += 128) {
                Key k[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) k[u] = i0 + 32 * u + lane < per ? part[i0 + 32 * u + lane] : 0;
                if (i0 == 0) {
                    const Key a = k[0] > k[1] ? k[0] : k[1], b = k[2] > k[3] ? k[2] : k[3];
                    kth = nth_of_warp(a > b ? a : b, p.n_best);
                    kth -= kth != 0;  // it may be among them itself
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    for (unsigned in = __ballot_sync(0xFFFFFFFFu, k[u] > kth); in; in &= in - 1) {
                        const Key c = __shfl_sync(0xFFFFFFFFu, k[u], __ffs(in) - 1);
                        if (c > kth) {
                            best[q].insert(c);
                            const Key n = best[q].nth(p.n_best);
                            kth = n > kth ? n : kth;
                        }
                    }
            }
        }
        for (int i = lane; i < p.slices; i += 32) m = fmaxf(m, i == lane ? mine.x : ml[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        for (int i = lane; i < p.slices; i += 32) {
            const float2 v = i == lane ? mine : ml[i];
            if (v.x > -INFINITY) sum = fmaf(v.y, expf(v.x - m), sum);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) s.m[w] = m, s.sum[w] = sum;
    }
    __syncthreads();
    const double INF = __longlong_as_double(0x7FF0000000000000ll);
    if (tid < p.beams) {
        const float m = s.m[tid], run = __ldg(p.scores + r0 + tid);
        // +infinity among the logits, none above -infinity, or a NaN score: no continuation
        const bool none = !(m < INFINITY) || !(m > -INFINITY) || !(run > -INFINITY);
        s.lse[tid] = none ? INF : static_cast<double>(m) + log(static_cast<double>(s.sum[tid]));
        s.m[tid] = none ? 0.0f : run;
    }
    __syncthreads();
    double score[ROWS];
    Key order[ROWS];  // of the scores: their bits in an order that integers have
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        const int w = warp + q * BM_WARPS;
        if (w >= p.beams) break;
        score[q] = static_cast<double>(value_of(best[q].mine)) - s.lse[w] + static_cast<double>(s.m[w]);
        const long long b = __double_as_longlong(score[q] + 0.0);
        order[q] = b < 0 ? ~static_cast<Key>(b) : static_cast<Key>(b) | 0x8000000000000000ull;
        if (best[q].mine == 0 || lane >= p.n_best || !(score[q] > -INF)) order[q] = 0;
        s.lists[w][lane] = order[q];
        const int count = __popc(__ballot_sync(0xFFFFFFFFu, order[q] != 0));
        if (lane == 0) s.count[w] = count;
    }
    __syncthreads();
    const long long out = static_cast<long long>(gi) * p.n_best;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
        const int w = warp + q * BM_WARPS;
        if (w >= p.beams) break;
        if (order[q] == 0) continue;
        // equal scores of other rows: the lower row comes first
        int rank = lane;
        for (int o = 0; o < p.beams; ++o)
            if (o != w) rank += above(s.lists[o], s.count[o], order[q] - (o < w));
        if (rank < p.n_best) {
            p.score[out + rank] = static_cast<float>(score[q]);
            p.token[out + rank] = token_of(best[q].mine);
            p.parent[out + rank] = static_cast<int32_t>(p.row0 + r0 + w);
        }
    }
    int count = 0;
    for (int w = 0; w < p.beams; ++w) count += s.count[w];
    for (int k = count + tid; k < p.n_best; k += BM_THREADS) {
        p.score[out + k] = -INFINITY;
        p.token[out + k] = -1;
        p.parent[out + k] = -1;
    }
}

// Block (slice, row).
template <typename T>
__global__ void __launch_bounds__(BM_THREADS, BM_BLOCKS) beam_kernel(const __grid_constant__ BeamParams p)
{
    using C = Chunk16<T>;
    constexpr int E = C::E;
    __shared__ BeamShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r = blockIdx.y;
    if (tid == 0) s.shown = 0;
    pdl_launch_dependents();
    pdl_wait();

    const long long out = r * p.slices + blockIdx.x;
    const int done = p.done ? __ldg(p.done + r) : -1;
    if (done >= 0) {
        // one continuation, at the running score: logit 0, sum of exponentials 1
        if (tid < p.n_best) p.part[out * p.n_best + tid] = blockIdx.x == 0 && tid == 0 ? key_of(0.0f, done) : 0;
        if (tid == 0) p.part_ml[out] = blockIdx.x == 0 ? make_float2(0.0f, 1.0f) : make_float2(-INFINITY, 0.0f);
    } else {
        // The row in 16-byte chunks of memory: chunk c holds tokens c E - shift .. + E - 1.
        const T *x = static_cast<const T *>(p.x) + r * p.x_stride;
        const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        const long long t0 = static_cast<long long>(blockIdx.x) * p.slice - shift;
        auto fetch = [&](int l) {  // the chunk at place l of the slice; -infinity beyond its ends
            const long long t = t0 + l;
            if (l < p.slice && t >= 0 && t + E <= p.vocab) return __ldcs(reinterpret_cast<const uint4 *>(x + t));
            T e[E];
#pragma unroll
            for (int i = 0; i < E; ++i)
                e[i] = l < p.slice && t + i >= 0 && t + i < p.vocab ? x[t + i] : static_cast<T>(-INFINITY);
            uint4 w;
            memcpy(&w, e, 16);
            return w;
        };
        auto pick = [](const uint4 (&c)[BM_CHUNKS], int k) {
            uint4 w = c[0];
#pragma unroll
            for (int i = 1; i < BM_CHUNKS; ++i) w = i == k ? c[i] : w;
            return w;
        };
        constexpr int BATCH = BM_THREADS * BM_CHUNKS * E;
        uint4 next[BM_CHUNKS];
#pragma unroll
        for (int k = 0; k < BM_CHUNKS; ++k) next[k] = fetch((k * BM_THREADS + tid) * E);
        __syncthreads();  // s.shown
        Best best;
        Key kth = 0;
        float m = -INFINITY, sum = 0.0f;
        const int span = static_cast<int>(min(static_cast<long long>(p.slice), p.vocab - t0));
        for (int l0 = 0; l0 < span; l0 += BATCH) {
            uint4 cur[BM_CHUNKS];
#pragma unroll
            for (int k = 0; k < BM_CHUNKS; ++k) cur[k] = next[k];
            if (l0 + BATCH < span) {
#pragma unroll
                for (int k = 0; k < BM_CHUNKS; ++k) next[k] = fetch(l0 + BATCH + (k * BM_THREADS + tid) * E);
            }
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < BM_CHUNKS; ++k) top = fmaxf(top, C::largest(cur[k]));

            // the sum, against the thread's own running maximum
            if (top > m) {
                sum *= ex2((m - top) * LOG2E);
                m = top;
            }
            if (m > -INFINITY) {
                const float m2 = m * LOG2E, before = sum;
#pragma unroll
                for (int k = 0; k < BM_CHUNKS; ++k)
#pragma unroll
                    for (int i = 0; i < E; ++i) sum += ex2(fmaf(C::at(cur[k], i), LOG2E, -m2));
                if (!(sum < INFINITY)) {  // a NaN among them counts nothing
                    sum = before;
#pragma unroll 1
                    for (int k = 0; k < BM_CHUNKS; ++k) {
                        const uint4 c = pick(cur, k);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float v = C::at(c, i);
                            if (v == v) sum += ex2(fmaf(v, LOG2E, -m2));
                        }
                    }
                }
            }

            // keys above the n-th
            const Key shown = *static_cast<volatile Key *>(&s.shown);
            if (shown > kth) kth = shown - 1;  // the key itself may be one of this warp's
            float bound = kth ? value_of(kth) : -INFINITY;
            if (!__any_sync(0xFFFFFFFFu, top >= bound && top > -INFINITY)) continue;
            unsigned bound_token = token_of(kth);
            if (l0 == 0) {
                const float b = nth_of_warp(top, p.n_best);
                if (b > bound) bound = b, bound_token = 0xFFFFFFFFu;
            }
            // Few come here, so the code is short rather than unrolled: kernels of one
            // batch wait for their instructions.
            int count = 0, k = 0;
            auto flush = [&]() {
                __syncwarp();
                for (int i = 0; i < count; ++i) {
                    const Key key = s.wait[warp][i];
                    if (key > kth) {
                        best.insert(key);
                        const Key n = best.nth(p.n_best);
                        kth = n > kth ? n : kth;
                    }
                }
                count = 0;
                __syncwarp();
            };
            unsigned mine = 0;  // the thread's elements of chunk k - 1 that wait
            uint4 c = cur[0];
            unsigned t = 0;
            for (;;) {
                if (!__any_sync(0xFFFFFFFFu, mine)) {
                    if (k == BM_CHUNKS) break;
                    c = pick(cur, k);
                    t = static_cast<unsigned>(t0 + l0 + (k * BM_THREADS + tid) * E);
                    ++k;
                    const float c_top = C::largest(c);
                    if (!__any_sync(0xFFFFFFFFu, c_top >= bound && c_top > -INFINITY)) continue;
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float v = C::at(c, i);
                        if (v > -INFINITY && (v > bound || (v == bound && t + i <= bound_token))) mine |= 1u << i;
                    }
                    continue;
                }
                const unsigned in = __ballot_sync(0xFFFFFFFFu, mine != 0);
                if (mine) {
                    const int i = __ffs(mine) - 1;
                    mine &= mine - 1;
                    float v = C::at(c, 0);
#pragma unroll
                    for (int e = 1; e < E; ++e) v = e == i ? C::at(c, e) : v;
                    s.wait[warp][count + __popc(in & ((1u << lane) - 1))] = key_of(v, t + i);
                }
                count += __popc(in);
                if (count > BM_LIST - 32) flush();
            }
            flush();
            const Key n = best.nth(p.n_best);
            if (lane == 0 && n > shown) atomicMax(&s.shown, n);
        }

        // the warps' lists, maxima and sums
        float wm = m;
#pragma unroll
        for (int d = 16; d; d >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, d));
        sum = m > -INFINITY ? sum * ex2((m - wm) * LOG2E) : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane >= p.n_best) best.mine = 0;
        s.lists[warp][lane] = best.mine;
        const int count = __popc(__ballot_sync(0xFFFFFFFFu, best.mine != 0));
        if (lane == 0) s.m[warp] = wm, s.sum[warp] = sum, s.count[warp] = count;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < BM_WARPS; ++w) all += s.count[w];
        if (best.mine) {
            int rank = lane;
#pragma unroll
            for (int w = 0; w < BM_WARPS; ++w)
                if (w != warp) rank += above(s.lists[w], s.count[w], best.mine);
            if (rank < p.n_best) p.part[out * p.n_best + rank] = best.mine;
        }
        if (tid >= all && tid < p.n_best) p.part[out * p.n_best + tid] = 0;
        if (tid == 0) {
            float bm = s.m[0], total = 0.0f;
#pragma unroll
            for (int w = 1; w < BM_WARPS; ++w) bm = fmaxf(bm, s.m[w]);
#pragma unroll
            for (int w = 0; w < BM_WARPS; ++w)
                if (s.m[w] > -INFINITY) total = fmaf(s.sum[w], ex2((s.m[w] - bm) * LOG2E), total);
            p.part_ml[out] = make_float2(bm, total);
        }
    }

    // the last of the group's blocks joins them
    const int gi = static_cast<int>(r / p.beams);
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned blocks = static_cast<unsigned>(p.beams) * static_cast<unsigned>(p.slices);
        s.last = atomicAdd(&p.cnt[gi], 1u) + 1 == blocks;
        if (s.last) p.cnt[gi] = 0;
    }
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    join(p, gi, s);
}

template <typename T>
cudaError_t launch_t(const BeamParams &p, int groups, cudaStream_t st)
{
    return launch_pdl(beam_kernel<T>, dim3(static_cast<unsigned>(p.slices), static_cast<unsigned>(groups * p.beams)),
                      BM_THREADS, 0, st, p);
}

}  // namespace

// The number of slices whose last wave of blocks ends first.  A block costs about
// as much as 8192 elements beside its own, a slice more for the join about 64.
int beam_slices(long long rows, long long vocab)
{
    constexpr long long SLOTS = BM_BLOCKS * ATTN_SMS;
    long long best = 1, best_cost = INT64_MAX;
    for (long long n = 1; n <= 64 && (n == 1 || vocab / n >= 2048); ++n) {
        const long long cost = (rows * n + SLOTS - 1) / SLOTS * (vocab / n + 8192) + 64 * n;
        if (cost < best_cost) best_cost = cost, best = n;
    }
    return static_cast<int>(best);
}

cudaError_t launch_beam(const BeamParams &p, qgemv_dtype type, int groups, cudaStream_t st)
{
    switch (type) {
    case QGEMV_F32: return launch_t<float>(p, groups, st);
    case QGEMV_F16: return launch_t<__half>(p, groups, st);
    default: return launch_t<__nv_bfloat16>(p, groups, st);
    }
}

}  // namespace qg
