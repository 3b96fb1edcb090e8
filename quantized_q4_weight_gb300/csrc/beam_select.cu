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
// down, so that a larger key is a larger logit or a lower token.  The block keeps the n
// best keys it has met in shared memory, in order, and compares every value with the
// n-th of them, which few pass; those are appended, and from time to time ranked together
// with the best by counting.  The first values go by the lowest of the warps' (n / 8)-th
// largest lanes, which n values of the block reach and not many more.  More equal or rising
// values than the list holds are read again and taken n at a time, each by a maximum over
// the block.
//
// What bounds it: for one search the chain launch, logits, ranks, arrival, join (four rows
// of 151936 fp32 7.4 us, the join 3 of them), so few rows have small slices.  For many rows
// memory at its rate behind what does not shrink with the row: 512 rows of 128257 bf16 with 16
// best take 33.4 us, 67 MB more take 10 (6.7 TB/s), rows of 8192 take 10.6, with one best 9.9.
// With 608, 760 or 1024 blocks for the 512 rows it took 43 to 61, with blocks of 128 threads 45:
// each meets its own first values, ranks and arrives.  Rings of three batches filled by TMA or by
// 16-byte copies took 43.
#include <type_traits>

#include "f32x2.cuh"
#include "kv8_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int BM_THREADS = 256, BM_WARPS = BM_THREADS / 32, BM_BLOCKS = 4;
constexpr int BM_CHUNKS = 4;   // 16-byte chunks of a thread's batch; as many are on their way
constexpr int BM_LIST = 512;   // keys of a block that are ranked at once
constexpr int BM_FULL = 16;    // appended keys that are worth a ranking: it raises the bound
constexpr int BM_WAIT = 128;   // keys of a warp in the join
constexpr int BM_BEAMS = 16;
constexpr int BM_SLICES = 64;  // of a row at most
constexpr float LOG2E = 1.4426950408889634f;

typedef unsigned long long Key;

// log(x) of a sum x > 0: the exponent's part in 64 bits, the rest, a logarithm
// below 0.35, in 32 (off by 2^-25).
__device__ __forceinline__ double log_of(float x)
{
    const int bits = __float_as_int(x), k = (bits - 0x3F3504F3) >> 23;  // x / 2^k in 0.707 .. 1.414
    const float f = __int_as_float(bits - (k << 23));
    return k * 0.6931471805599453 + static_cast<double>(logf(f));
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

// Elements of a 16-byte chunk as floats; of a batch the largest (NaN passed over), a bit for
// each element that reaches a bound (a value of the type), and where such an element is:
// chunk, place in it.
template <typename T>
struct Chunk16;
template <>
struct Chunk16<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ float at(const uint4 &w, int i)
    {
        return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
    }
    static __device__ __forceinline__ float largest(const uint4 (&c)[BM_CHUNKS])
    {
        float m = at(c[0], 0);
#pragma unroll
        for (int k = 1; k < 4 * BM_CHUNKS; ++k) m = fmaxf(m, at(c[k >> 2], k & 3));
        return m;
    }
    static __device__ __forceinline__ unsigned reach(const uint4 (&c)[BM_CHUNKS], float bound)
    {
        unsigned bits = 0;
#pragma unroll
        for (int k = 0; k < 4 * BM_CHUNKS; ++k) bits |= at(c[k >> 2], k & 3) >= bound ? 1u << k : 0;
        return bits;
    }
    static __device__ __forceinline__ int2 place(int bit) { return make_int2(bit >> 2, bit & 3); }
    static __device__ __forceinline__ float value(unsigned word, int) { return __uint_as_float(word); }
    static __device__ __forceinline__ int word(int i) { return i; }
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
    static __device__ __forceinline__ float largest(const uint4 (&c)[BM_CHUNKS])
    {
        __half2 m = pair(c[0], 0);
#pragma unroll
        for (int k = 1; k < 4 * BM_CHUNKS; ++k) m = __hmax2(m, pair(c[k >> 2], k & 3));
        return fmaxf(__low2float(m), __high2float(m));
    }
    // bit w: the lower element of word w, bit 16 + w its upper one
    static __device__ __forceinline__ unsigned reach(const uint4 (&c)[BM_CHUNKS], float bound)
    {
        const __half2 b = __half2half2(__float2half_rn(bound));
        unsigned bits = 0;
#pragma unroll
        for (int k = 0; k < 4 * BM_CHUNKS; ++k) bits |= __hge2_mask(pair(c[k >> 2], k & 3), b) & 0x10001u << k;
        return bits;
    }
    static __device__ __forceinline__ int2 place(int bit) { return make_int2(bit >> 2 & 3, 2 * (bit & 3) + (bit >> 4)); }
    static __device__ __forceinline__ float value(unsigned word, int i)
    {
        const __half2 p = *reinterpret_cast<const __half2 *>(&word);
        return i & 1 ? __high2float(p) : __low2float(p);
    }
    static __device__ __forceinline__ int word(int i) { return i >> 1; }
};
template <>
struct Chunk16<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ unsigned part(const uint4 &w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    static __device__ __forceinline__ __nv_bfloat162 pair(const uint4 &w, int i)
    {
        const unsigned u = part(w, i);
        return *reinterpret_cast<const __nv_bfloat162 *>(&u);
    }
    static __device__ __forceinline__ float at(const uint4 &w, int i)
    {
        return __uint_as_float(i & 1 ? part(w, i >> 1) & 0xFFFF0000u : part(w, i >> 1) << 16);
    }
    static __device__ __forceinline__ float largest(const uint4 (&c)[BM_CHUNKS])
    {
        __nv_bfloat162 m = pair(c[0], 0);
#pragma unroll
        for (int k = 1; k < 4 * BM_CHUNKS; ++k) m = __hmax2(m, pair(c[k >> 2], k & 3));
        return fmaxf(__low2float(m), __high2float(m));
    }
    // bit w: the lower element of word w, bit 16 + w its upper one
    static __device__ __forceinline__ unsigned reach(const uint4 (&c)[BM_CHUNKS], float bound)
    {
        const __nv_bfloat162 b = __bfloat162bfloat162(__float2bfloat16_rn(bound));
        unsigned bits = 0;
#pragma unroll
        for (int k = 0; k < 4 * BM_CHUNKS; ++k) bits |= __hge2_mask(pair(c[k >> 2], k & 3), b) & 0x10001u << k;
        return bits;
    }
    static __device__ __forceinline__ int2 place(int bit) { return make_int2(bit >> 2 & 3, 2 * (bit & 3) + (bit >> 4)); }
    static __device__ __forceinline__ float value(unsigned word, int i)
    {
        return __uint_as_float(word << (i & 1 ? 0 : 16) & 0xFFFF0000u);
    }
    static __device__ __forceinline__ int word(int i) { return i >> 1; }
};

// A warp's 32 values falling over its lanes.
template <typename V>
__device__ __forceinline__ void sort_warp(V &v)
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
}

// A bound that at least n of the block's values reach, to all threads, given each
// thread's largest value v and that all threads of the first `warps` warps have values: the
// lowest of those warps' ceil(n / warps)-th, or, where one has too few above -infinity, the
// n-th of all threads' (-infinity where there are fewer).  `all` is scratch.
__device__ __forceinline__ float low_bound(float v, int n, int warps, unsigned (&s)[BM_WARPS], unsigned *all)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned mine = ordered(v);
    unsigned u = mine, top = 0;
    const int each = (n + warps - 1) / warps;
    for (int k = 0; k < each; ++k) {  // the largest `each` times, each taken out
        top = __reduce_max_sync(0xFFFFFFFFu, u);
        if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, u == top)) - 1) u = 0;
    }
    if (lane == 0) s[warp] = warp < warps ? top : 0xFFFFFFFFu;
    __syncthreads();
    const float low = from_ordered(__reduce_min_sync(0xFFFFFFFFu, s[lane & (BM_WARPS - 1)]));
    if (low > -INFINITY) return low;
    all[tid] = mine;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < BM_THREADS; ++i) rank += all[i] > mine || (all[i] == mine && i < tid);
    __syncthreads();
    if (rank == n - 1) s[0] = mine;
    __syncthreads();
    return from_ordered(s[0]);
}

// The best n of list[0 .. total), in order, to its front; THREADS threads, `t` of them this
// one, `sync` their barrier, PER keys each.
template <int THREADS, int PER, typename Sync>
__device__ __forceinline__ void rank_keys(Key *list, int total, int n, int t, Sync sync)
{
    sync();
    Key k[PER];
    int rank[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) k[u] = t + u * THREADS < total ? list[t + u * THREADS] : 0, rank[u] = 0;
    if (t < total)
        for (int i = 0; i < total; ++i) {
            const Key o = list[i];
#pragma unroll
            for (int u = 0; u < PER; ++u) rank[u] += o > k[u];
        }
    sync();
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (t + u * THREADS < total && rank[u] < n) list[rank[u]] = k[u];
    sync();
}

// The largest key of the block, to all threads.
__device__ __forceinline__ Key block_largest(Key key, Key *s)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const Key o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
        key = o > key ? o : key;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = key;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < BM_WARPS; ++w) key = s[w] > key ? s[w] : key;
    return key;
}

struct BeamShared {
    union {
        Key list[BM_LIST];              // the best of the block so far, then those appended
        Key wait[BM_WARPS][BM_WAIT];    // the same of a row's warp in the join
    };
    Key rows[BM_BEAMS][32];             // the join's rows: their best keys,
    Key order[BM_BEAMS][32];            // the scores of those as integers (0: none)
    float score[BM_BEAMS][32];          // and rounded
    Key best[BM_WARPS];
    unsigned first[BM_WARPS];
    int total;                          // keys of the list
    int places[BM_WARPS];               // of a warp's list in the join
    int last;
    float m[BM_BEAMS], sum[BM_BEAMS];
    int count;                          // continuations of all rows
};

// The join of group gi of the launch, by the block that arrived last.
__device__ void join(const BeamParams &p, int gi, BeamShared &s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r0 = static_cast<long long>(gi) * p.beams;
    const int per = p.slices * p.n_best;
    int nth = 1;
    while (nth < p.n_best && 2 * ((p.n_best + nth - 1) / nth) > min(32, p.slices)) nth = min(2 * nth, p.n_best);
    // Code that one block of a search runs once waits for its instructions: the loops over a
    // warp's rows are not unrolled.
    // each row's n best keys, maximum and sum
    const double INF = __longlong_as_double(0x7FF0000000000000ll);
#pragma unroll 1
    for (int w = warp; w < p.beams; w += BM_WARPS) {
        const float run = __ldg(p.scores + r0 + w);
        const Key *part = p.part + (r0 + w) * per;
        const float2 *ml = p.part_ml + (r0 + w) * p.slices;
        float m = -INFINITY, sum = 0.0f;
        float2 mine[BM_SLICES / 32];
#pragma unroll
        for (int u = 0; u < BM_SLICES / 32; ++u)
            mine[u] = lane + 32 * u < p.slices ? __ldcg(ml + lane + 32 * u) : make_float2(-INFINITY, 0.0f);
        Key best;
        if (p.slices == 1) {
            best = lane < p.n_best ? __ldcg(part + lane) : 0;
        } else {
            constexpr int U = 10;
            Key k[U];
            auto fetch = [&](int i0) {
#pragma unroll
                for (int u = 0; u < U; ++u) k[u] = i0 + 32 * u + lane < per ? __ldcg(part + i0 + 32 * u + lane) : 0;
            };
            // Where n / j of the slices have a j-th key of some size, n keys are as large: the bound that
            // a warp's lanes take first.  j is the least for which half of the slices do.
            unsigned head = lane < p.slices ? static_cast<unsigned>(__ldcg(part + lane * p.n_best + nth - 1) >> 32) : 0;
            fetch(0);
            sort_warp(head);
            head = __shfl_sync(0xFFFFFFFFu, head, (p.n_best + nth - 1) / nth - 1);
            Key kth = head ? (static_cast<Key>(head) << 32) - 1 : 0;
            Key *list = s.wait[warp];
            auto rank_some = [&](int total) {
                if (total <= 64)
                    rank_keys<32, 2>(list, total, p.n_best, lane, [] { __syncwarp(); });
                else
                    rank_keys<32, BM_WAIT / 32>(list, total, p.n_best, lane, [] { __syncwarp(); });
            };
            int total = 0;
            int *places = &s.places[warp];
            if (lane == 0) *places = 0;
            __syncwarp();
            for (int i0 = 0;;) {  // few pass: places in any order, as they are ranked
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k[u] > kth) {
                        const int i = atomicAdd(places, 1);
                        if (i < BM_WAIT) list[i] = k[u];
                    }
                i0 += 32 * U;
                if (i0 >= per) break;
                fetch(i0);
            }
            __syncwarp();
            total = *places;
            const bool listed = total <= BM_WAIT;
            if (listed) {
                rank_some(total);
                total = min(total, p.n_best);
            } else {  // all of them again, ranked whenever the list is full
                total = 0;
                fetch(0);
            }
            for (int i0 = 0; !listed;) {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    Key c = k[0];
#pragma unroll
                    for (int v = 1; v < U; ++v) c = u == v ? k[v] : c;
                    const unsigned in = __ballot_sync(0xFFFFFFFFu, c > kth);
                    if (c > kth) list[total + __popc(in & ((1u << lane) - 1))] = c;
                    total += __popc(in);
                    const bool end = u == U - 1 && i0 + 32 * U >= per;
                    if (total > BM_WAIT - 32 || end) {
                        rank_some(total);
                        total = min(total, p.n_best);
                        if (total == p.n_best) kth = list[p.n_best - 1];
                    }
                }
                i0 += 32 * U;
                if (i0 >= per) break;
                fetch(i0);
            }
            best = lane < total ? list[lane] : 0;
        }
#pragma unroll
        for (int u = 0; u < BM_SLICES / 32; ++u) m = fmaxf(m, mine[u].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll
        for (int u = 0; u < BM_SLICES / 32; ++u)
            if (mine[u].x > -INFINITY) sum = fmaf(mine[u].y, ex2((mine[u].x - m) * LOG2E), sum);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        // +infinity among the logits, none above -infinity, or a NaN score: no continuation
        const bool none = !(m < INFINITY) || !(m > -INFINITY) || !(run > -INFINITY);
        // x - M first: beside an M of any size the logarithm would be lost
        const double rel = static_cast<double>(value_of(best)) - static_cast<double>(m);
        const double v = none ? -INF : rel - log_of(sum) + static_cast<double>(run);
        const long long b = __double_as_longlong(v + 0.0);
        const Key order = b < 0 ? ~static_cast<Key>(b) : static_cast<Key>(b) | 0x8000000000000000ull;
        const bool there = best != 0 && lane < p.n_best && v > -INF;
        s.rows[w][lane] = best;
        s.order[w][lane] = there ? order : 0;
        s.score[w][lane] = static_cast<float>(v);
        const unsigned in = __ballot_sync(0xFFFFFFFFu, there);
        if (lane == 0) atomicAdd(&s.count, __popc(in));
    }
    __syncthreads();
    const long long out = static_cast<long long>(gi) * p.n_best;
#pragma unroll 1
    for (int w = warp; w < p.beams; w += BM_WARPS) {
        const Key mine = s.order[w][lane];
        // how many of the other rows' come before: all above, and equal ones of lower rows.  A row's
        // fall, with zeros behind them.
        int rank = lane;
#pragma unroll 4
        for (int o = 0; o < p.beams; ++o) {
            const Key than = mine - (o < w);
            int at = 0;
#pragma unroll
            for (int step = 16; step; step >>= 1) at += s.order[o][at + step - 1] > than ? step : 0;
            at += s.order[o][at] > than;
            rank += o != w ? at : 0;
        }
        if (mine && rank < p.n_best) {
            p.score[out + rank] = s.score[w][lane];
            p.token[out + rank] = token_of(s.rows[w][lane]);
            p.parent[out + rank] = static_cast<int32_t>(p.row0 + r0 + w);
        }
    }
    for (int k = s.count + tid; k < p.n_best; k += BM_THREADS) {
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
        const int span = static_cast<int>(min(static_cast<long long>(p.slice), p.vocab - t0));  // below 1: nothing
        const int whole_from = t0 < 0 ? 1 : 0;  // batches from here on that end within the span lie in the row
        const uint4 *base = reinterpret_cast<const uint4 *>(x + t0) + tid;
        auto fetch_batch = [&](int l0) {
            if (l0 >= whole_from && l0 + BATCH <= span) {
                const uint4 *from = base + l0 / E;
#pragma unroll
                for (int k = 0; k < BM_CHUNKS; ++k) next[k] = __ldcs(from + k * BM_THREADS);
            } else {
#pragma unroll
                for (int k = 0; k < BM_CHUNKS; ++k) next[k] = fetch(l0 + (k * BM_THREADS + tid) * E);
            }
        };
        fetch_batch(0);
        float m = -INFINITY, sum = 0.0f, bound = -INFINITY;
        unsigned bound_token = 0xFFFFFFFFu;  // a value equal to the bound counts up to this token
        int have = 0, kept = 0, since = 0;   // keys of the list that are the best so far, and with those after them; where it was
                                             // looked at last
        for (int l0 = 0; l0 < span; l0 += BATCH) {
            uint4 cur[BM_CHUNKS];
#pragma unroll
            for (int k = 0; k < BM_CHUNKS; ++k) cur[k] = next[k];
            if (l0 + BATCH < span) fetch_batch(l0 + BATCH);
            const float top = fmaxf(C::largest(cur), -INFINITY);  // of nothing but NaN: -infinity

            // The sum, against the thread's first maximum, or one that stands 8 above it: an exponent of 55, as
            // 40 above, is off by 1.3e-6 of its term, one of 11 by 3e-7, and few threads meet such a one later.
            if (top > m + 8.0f) {
                sum *= ex2((m - top) * LOG2E);
                m = top;
            }
            // Its terms are 2^(v log2e - m2) with m2 = m log2e rounded, one fused operation each, and what that
            // rounding leaves, r, is known exactly and taken out of the batch's sum: left in, it would stay in
            // every term.  Beyond 2^20 (masks of a type's lowest value) r is no longer small, and the
            // difference v - m is formed first, which for all took 34.6 us instead of 33.6 (512 rows of 128257 bf16).
            if (m > -INFINITY) {
                const float m2 = m * LOG2E;
                auto terms = [&](auto far) {
                    float2 two = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int k = 0; k < BM_CHUNKS; ++k)
#pragma unroll
                        for (int i = 0; i < E; i += 2) {
                            const float2 v = make_float2(C::at(cur[k], i), C::at(cur[k], i + 1)), l2 = make_float2(LOG2E, LOG2E);
                            const float2 e = far.value ? mul2(add2(v, make_float2(-m, -m)), l2) : fma2(v, l2, make_float2(-m2, -m2));
                            two = add2(two, make_float2(ex2(e.x), ex2(e.y)));
                        }
                    return two.x + two.y;
                };
                float more;
                if (fabsf(m) <= 1048576.0f)
                    more = terms(std::false_type()) * ex2(-fmaf(m, LOG2E, -m2));
                else
                    more = terms(std::true_type());
                if (!(more < INFINITY)) {  // a NaN among them counts nothing
                    more = 0.0f;
#pragma unroll 1
                    for (int k = 0; k < BM_CHUNKS; ++k) {
                        const uint4 c = pick(cur, k);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float v = C::at(c, i);
                            if (v == v) more += ex2((v - m) * LOG2E);
                        }
                    }
                }
                sum += more;
            }

            if (l0 == 0) {
                if (tid == 0) s.total = 0;
                bound = low_bound(top, p.n_best, max(1, min(BM_WARPS, span / (32 * E))), s.first,
                                  reinterpret_cast<unsigned *>(s.list));
            }
            const auto taken = [&](float v, unsigned t) { return v > -INFINITY && (v > bound || (v == bound && t <= bound_token)); };
            if (top >= bound && top > -INFINITY) {
                for (unsigned bits = C::reach(cur, bound); bits; bits &= bits - 1) {
                    const int2 at = C::place(__ffs(bits) - 1);
                    const uint4 c = pick(cur, at.x);
                    const int w = C::word(at.y);
                    const float v = C::value(w == 0 ? c.x : w == 1 ? c.y : w == 2 ? c.z : c.w, at.y);
                    const unsigned t = static_cast<unsigned>(t0 + l0 + (at.x * BM_THREADS + tid) * E + at.y);
                    if (taken(v, t)) {
                        const int i = atomicAdd(&s.total, 1);
                        if (i < BM_LIST) s.list[i] = key_of(v, t);
                    }
                }
            }
            // the list is looked at after 1, 2, 4, 8 ... batches, between which about n keys are
            // appended each, and at the end
            const int no = l0 / BATCH;
            const bool first = no == 0, end = l0 + BATCH >= span;
            if ((no & (no + 1)) && !end) continue;
            __syncthreads();
            int total = s.total;
            const bool over = total > BM_LIST;
            if (over) {
                // all since the last look again, one at a time: the largest key below the last
                Key last = ~0ull;
                int found = 0;
                for (; found < p.n_best; ++found) {
                    Key key = 0;
#pragma unroll 1
                    for (int l = since + tid * E; l < l0 + BATCH; l += BM_THREADS * E) {
                        const uint4 c = fetch(l);
                        const unsigned t = static_cast<unsigned>(t0 + l);
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            const float v = C::at(c, i);
                            const Key mine = key_of(v, t + i);
                            if (taken(v, t + i) && mine < last && mine > key) key = mine;
                        }
                    }
                    last = block_largest(key, s.best);
                    if (last == 0) break;
                    if (tid == 0) s.list[kept + found] = last;
                }
                total = kept + found;
            }
            if (total > have + BM_FULL || first || end || over) {
                if (total <= BM_THREADS)
                    rank_keys<BM_THREADS, 1>(s.list, total, p.n_best, tid, [] { __syncthreads(); });
                else
                    rank_keys<BM_THREADS, BM_LIST / BM_THREADS>(s.list, total, p.n_best, tid, [] { __syncthreads(); });
                total = have = min(total, p.n_best);
                if (tid == 0) s.total = have;
                if (have == p.n_best) {
                    bound = value_of(s.list[have - 1]);
                    bound_token = token_of(s.list[have - 1]);
                }
            }
            kept = total;
            since = l0 + BATCH;
            __syncthreads();
        }

        // the block's list, maximum and sum
        float wm = m;
#pragma unroll
        for (int d = 16; d; d >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xFFFFFFFFu, wm, d));
        sum = m > -INFINITY ? sum * ex2((m - wm) * LOG2E) : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) s.m[warp] = wm, s.sum[warp] = sum;
        __syncthreads();
        if (tid < p.n_best) p.part[out * p.n_best + tid] = tid < have ? s.list[tid] : 0;
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
    __syncthreads();
    if (tid == 0) {
        const unsigned blocks = static_cast<unsigned>(p.beams) * static_cast<unsigned>(p.slices);
        unsigned before;  // releases the block's parts, and acquires the others'
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.cnt + gi) : "memory");
        s.last = before + 1 == blocks;
        if (s.last) p.cnt[gi] = 0;
        s.count = 0;
    }
    __syncthreads();
    if (s.last) join(p, gi, s);
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
    for (long long n = 1; n <= BM_SLICES && (n == 1 || vocab / n >= 2048); ++n) {
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
