// beam_select.cu -- the best continuations of each beam search over its beams and
// the vocabulary (minfer README "How it works": device-side argmax; here of many).
//
//   s(r, t) = run[r] + x[r][t] - lse[r],  lse[r] = M + log(sum exp(x[r][t] - M))
// Within a row the order of s is that of x, so a block that holds a slice of a
// row needs no sum to find the slice's n best: it keeps its values in registers,
// leaves their maximum, their sum of exponentials and their n best in order, and
// the last block of a search to arrive joins them, forms s in 64 bits and takes the
// n best of all.  Nothing depends on which block that is.
//
// The n best of a block's values: every warp orders its lanes' largest values
// (a bitonic network of shuffles); the n-th largest of all threads' largest is no
// more than the n-th largest value, so the few values from there on are
// collected and ranked by counting.  Where equal values overflow the list, the n
// best are taken one at a time instead.
//
// What bounds it: memory for many rows (logits read once); the chain launch,
// logits, ranks, arrival, join for one search, so few rows have small slices.
#include "kv8_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int BM_THREADS = 256, BM_WARPS = BM_THREADS / 32;
constexpr int BM_VALUES = BEAM_SLICE_MAX / BM_THREADS;  // of a thread: 32
constexpr int BM_LIST = 512;                            // values that are ranked by counting
constexpr int BM_BEAMS = 16;

__device__ __forceinline__ float bm_f(float v) { return v; }
__device__ __forceinline__ float bm_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float bm_f(__nv_bfloat16 v) { return __bfloat162float(v); }

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

// The n-th largest (n <= 32) of 256 threads' values `v`, a lower bound of the n-th
// largest of anything that they are the largest of.  s: [BM_WARPS][32] and a word.
__device__ __forceinline__ float nth_of_threads(float v, int n, float (*s)[32], float *s_bound)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int d = k >> 1; d; d >>= 1) {
            const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
            const bool down = (lane & k) == 0, low = (lane & d) == 0;  // k = 32: descending over the warp
            v = down == low ? fmaxf(v, o) : fminf(v, o);
        }
    s[warp][lane] = v;
    __syncthreads();
    // a value's rank: its place in its own list, and in each other list the values that come before it
    int rank = lane;
#pragma unroll
    for (int w = 0; w < BM_WARPS; ++w) {
        int at = 0;
#pragma unroll
        for (int d = 32; d; d >>= 1) {  // the first `at` of list w come before
            if (at + d <= 32) {
                const float o = s[w][at + d - 1];
                if (o > v || (o == v && w < warp)) at += d;
            }
        }
        rank += w == warp ? 0 : at;
    }
    if (rank == n - 1) *s_bound = v;
    __syncthreads();
    return *s_bound;
}

// The largest key of the block, to all threads.  s: [BM_WARPS].
__device__ __forceinline__ unsigned long long block_largest(unsigned long long key, unsigned long long *s)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, key, d);
        key = o > key ? o : key;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = key;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < BM_WARPS; ++w) key = s[w] > key ? s[w] : key;
    return key;
}

// A candidate of the join: s, then the lower row, the larger logit, the lower token.
struct Cand {
    double s;
    unsigned row, x, token;  // x: ordered bits

    __device__ __forceinline__ bool before(const Cand &o) const
    {
        if (s != o.s) return s > o.s;
        if (row != o.row) return row < o.row;
        if (x != o.x) return x > o.x;
        return token < o.token;
    }
};

struct BeamShared {
    float sorted[BM_WARPS][32];
    float bound, red[BM_WARPS];
    unsigned long long best[BM_WARPS];
    int count, last;
    double lse[BM_BEAMS];
    float run[BM_BEAMS];
    union {
        unsigned long long keys[BM_LIST];
        Cand list[BM_LIST];
    };
};

// The join of group gi of the launch, by the block that arrived last.
__device__ void join(const BeamParams &p, int gi, BeamShared &s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r0 = static_cast<long long>(gi) * p.beams;
    const double NONE = -__longlong_as_double(0x7FF0000000000000ll);
    for (int w = warp; w < p.beams; w += BM_WARPS) {
        const float2 *ml = p.part_ml + (r0 + w) * p.slices;
        float m = -INFINITY, sum = 0.0f;
        for (int i = lane; i < p.slices; i += 32) m = fmaxf(m, ml[i].x);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        if (m > -INFINITY)
            for (int i = lane; i < p.slices; i += 32) sum = fmaf(ml[i].y, expf(ml[i].x - m), sum);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) {
            const float run = __ldg(p.scores + r0 + w);
            // +infinity among the logits, none above -infinity, or a NaN score: no continuation
            const bool none = !(m < INFINITY) || !(m > -INFINITY) || !(run > -INFINITY);
            s.lse[w] = none ? -NONE : static_cast<double>(m) + log(static_cast<double>(sum));
            s.run[w] = none ? 0.0f : run;
        }
    }
    if (tid == 0) s.count = 0;
    __syncthreads();

    const int per = p.slices * p.n_best, total = p.beams * per;
    const uint2 *part = p.part + r0 * per;
    auto cand = [&](int i, Cand &c) {  // whether there is one
        const uint2 v = part[i];
        const int w = i / per;
        const float x = __uint_as_float(v.x);
        c.s = static_cast<double>(x) - s.lse[w] + static_cast<double>(s.run[w]);
        c.row = w, c.x = ordered(x), c.token = v.y;
        return v.y != 0xFFFFFFFFu && c.s > NONE;
    };
    // in 32 bits first, with room for their rounding: a few survive
    auto rough = [&](int i) {
        const uint2 v = part[i];
        const int w = i / per;
        return v.y == 0xFFFFFFFFu ? -INFINITY : __uint_as_float(v.x) - static_cast<float>(s.lse[w]) + s.run[w];
    };
    float top = -INFINITY;
    for (int i = tid; i < total; i += BM_THREADS) top = fmaxf(top, rough(i));
    float bound = nth_of_threads(top, p.n_best, s.sorted, &s.bound);
    if (bound > -INFINITY && bound < INFINITY) {
        float off = fabsf(bound);
        for (int w = 0; w < p.beams; ++w) off = fmaxf(off, fmaxf(fabsf(static_cast<float>(s.lse[w])) < INFINITY ? fabsf(static_cast<float>(s.lse[w])) : 0.0f, fabsf(s.run[w])));
        // x, lse, run and two sums, each within 2^-24 of at most 4 * off
        bound -= off * 4.0f * 6.0e-7f;
    }
    for (int i = tid; i < total; i += BM_THREADS) {
        const float f = rough(i);
        Cand c;
        if (f >= bound && f > -INFINITY && cand(i, c)) {
            const int at = atomicAdd(&s.count, 1);
            if (at < BM_LIST) s.list[at] = c;
        }
    }
    __syncthreads();
    const int count = s.count;
    const long long out = static_cast<long long>(gi) * p.n_best;
    auto put = [&](int k, const Cand &c) {
        p.score[out + k] = static_cast<float>(c.s);
        p.token[out + k] = c.token;
        p.parent[out + k] = static_cast<int32_t>(p.row0 + r0 + c.row);
    };
    auto put_none = [&](int k) {
        p.score[out + k] = -INFINITY;
        p.token[out + k] = -1;
        p.parent[out + k] = -1;
    };
    if (count <= BM_LIST) {
        for (int i = tid; i < count; i += BM_THREADS) {
            const Cand c = s.list[i];
            int rank = 0;
            for (int k = 0; k < count; ++k) rank += s.list[k].before(c);
            if (rank < p.n_best) put(rank, c);
        }
        for (int k = count + tid; k < p.n_best; k += BM_THREADS) put_none(k);
        return;
    }
    // more equal values than the list holds: one at a time
    Cand last;
    for (int k = 0; k < p.n_best; ++k) {
        Cand best;
        bool have = false;
        for (int i = tid; i < total; i += BM_THREADS) {
            Cand c;
            if (cand(i, c) && (k == 0 || last.before(c)) && (!have || c.before(best))) best = c, have = true;
        }
        __syncthreads();
        if (!have) best.s = NONE, best.row = 0xFFFFFFFFu, best.x = 0, best.token = 0xFFFFFFFFu;
        s.list[tid] = best;
        __syncthreads();
        for (int d = BM_THREADS / 2; d; d >>= 1) {
            if (tid < d && s.list[tid + d].before(s.list[tid])) s.list[tid] = s.list[tid + d];
            __syncthreads();
        }
        last = s.list[0];
        if (tid == 0) {
            if (last.row != 0xFFFFFFFFu)
                put(k, last);
            else
                put_none(k);
        }
    }
}

// Block (slice, row).
template <typename T>
__global__ void __launch_bounds__(BM_THREADS, 3) beam_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int E = 16 / sizeof(T), CHUNKS = BM_VALUES / E;
    __shared__ BeamShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long r = blockIdx.y;
    pdl_launch_dependents();
    pdl_wait();

    const long long out = r * p.slices + blockIdx.x;
    const int done = p.done ? __ldg(p.done + r) : -1;
    if (done >= 0) {
        // one continuation, at the running score: logit 0, sum of exponentials 1
        if (tid < p.n_best) p.part[out * p.n_best + tid] = make_uint2(0u, blockIdx.x == 0 && tid == 0 ? done : 0xFFFFFFFFu);
        if (tid == 0) p.part_ml[out] = blockIdx.x == 0 ? make_float2(0.0f, 1.0f) : make_float2(-INFINITY, 0.0f);
    } else {
        // The row in 16-byte chunks of memory: chunk c holds tokens c E - shift .. + E - 1.
        const T *x = static_cast<const T *>(p.x) + r * p.x_stride;
        const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        const long long t0 = static_cast<long long>(blockIdx.x) * p.slice - shift;
        float v[BM_VALUES];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int l = (k * BM_THREADS + tid) * E;  // place in the slice
            const long long t = t0 + l;
            if (l < p.slice && t >= 0 && t + E <= p.vocab) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(x + t));
                T e[E];
                memcpy(e, &w, 16);
#pragma unroll
                for (int i = 0; i < E; ++i) v[k * E + i] = bm_f(e[i]);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i)
                    v[k * E + i] = l < p.slice && t + i >= 0 && t + i < p.vocab ? bm_f(x[t + i]) : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < BM_VALUES; ++k) {
            v[k] = v[k] == v[k] ? v[k] : -INFINITY;
            top = fmaxf(top, v[k]);
        }
        if (tid == 0) s.count = 0;
        const float bound = nth_of_threads(top, p.n_best, s.sorted, &s.bound);
        float m = s.sorted[0][0];
#pragma unroll
        for (int w = 1; w < BM_WARPS; ++w) m = fmaxf(m, s.sorted[w][0]);

        // the values from the bound on, and the sum
        float sum = 0.0f;
        const float m2 = m * 1.4426950408889634f;
#pragma unroll
        for (int k = 0; k < BM_VALUES; ++k) {
            if (v[k] >= bound && v[k] > -INFINITY) {
                const int at = atomicAdd(&s.count, 1);
                const unsigned token = static_cast<unsigned>(t0 + (k / E * BM_THREADS + tid) * E + k % E);
                if (at < BM_LIST) s.keys[at] = static_cast<unsigned long long>(ordered(v[k])) << 32 | (0xFFFFFFFFu - token);
            }
            sum += ex2(fmaf(v[k], 1.4426950408889634f, -m2));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) s.red[warp] = sum;
        __syncthreads();
        const int count = s.count;
        uint2 *part = p.part + out * p.n_best;
        auto put = [&](int k, unsigned long long key) {
            const unsigned o = static_cast<unsigned>(key >> 32);
            part[k] = make_uint2(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o, 0xFFFFFFFFu - static_cast<unsigned>(key));
        };
        if (count <= BM_LIST) {
            for (int i = tid; i < count; i += BM_THREADS) {
                const unsigned long long key = s.keys[i];
                int rank = 0;
                for (int k = 0; k < count; ++k) rank += s.keys[k] > key;
                if (rank < p.n_best) put(rank, key);
            }
            for (int k = count + tid; k < p.n_best; k += BM_THREADS) part[k] = make_uint2(0u, 0xFFFFFFFFu);
        } else {
            unsigned long long last = ~0ull;
            for (int k = 0; k < p.n_best; ++k) {
                unsigned long long key = 0;
#pragma unroll
                for (int i = 0; i < BM_VALUES; ++i) {
                    const unsigned token = static_cast<unsigned>(t0 + (i / E * BM_THREADS + tid) * E + i % E);
                    const unsigned long long mine = static_cast<unsigned long long>(ordered(v[i])) << 32 | (0xFFFFFFFFu - token);
                    if (v[i] > -INFINITY && mine < last && mine > key) key = mine;
                }
                last = block_largest(key, s.best);
                if (tid == 0) put(k, last);  // the bound says that there are n
            }
        }
        if (tid == 0) {
            float all = s.red[0];
#pragma unroll
            for (int w = 1; w < BM_WARPS; ++w) all += s.red[w];
            p.part_ml[out] = make_float2(m, m > -INFINITY ? all : 0.0f);
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

// About two blocks for each of 152 multiprocessors, in whole chunks a thread.
int beam_slice(long long rows, long long vocab)
{
    const long long want = (2 * ATTN_SMS + rows - 1) / rows;
    const long long slice = ((vocab + want - 1) / want + 2047) / 2048 * 2048;
    return static_cast<int>(slice < 2048 ? 2048 : slice > BEAM_SLICE_MAX ? BEAM_SLICE_MAX : slice);
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
