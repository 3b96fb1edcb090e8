// attn_prefix.cu -- attention of a batch of sequences that share a prefix,
// over a paged cache (minfer README "How it works": GQA attention whose keys
// are split over blocks and whose partial results are combined).
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j - max)
// over the keys a query sees.  The keys are cut into parts: ranges of the
// prefix, each for a tile of the rows of *all* sequences (so the prefix is
// read once for the batch, not once per sequence), and ranges of each
// suffix for its own sequence's rows.  A block takes one part and one cache
// head and keeps, per row, the running maximum m, the sum l of the weights
// and the weighted sum of v; it leaves (m, l, sum) in the workspace.  A
// second launch combines the parts of each row: with M the largest m,
// o = sum 2^(m - M) sum_part / sum 2^(m - M) l.  Both launches work in the
// base-2 domain (scale log2 e folded into the scores).
//
// A sequence's last n_q - 1 suffix rows are seen by some of its queries
// only.  They (at most seven) go to the combining launch, which takes each
// of them for each row that sees it as a part of one key: the blocks of the
// first launch then need no mask but the end of their range, and what such
// a row holds (infinities, NaN) cannot reach a query that does not see it
// through a product with a zero weight.
//
// Tiles of 64 keys come through a ring of cp.async stages in shared memory,
// 16-byte chunks XOR-swizzled by row so that ldmatrix is free of conflicts;
// the scores and the weighted sums are mma.sync products (16 x 8 x 16).  Row
// tiles of up to 16 or 32 rows (a suffix's few queries) give each of the
// four warps 16 of a tile's keys and merge the warps at the end, so that all
// warps work and each key is read from shared memory once; taller tiles (64
// rows) give each warp 16 rows.
#include <type_traits>

#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int AT_THREADS = 128;
constexpr int AT_KEYS = 64;    // keys of a stage
constexpr int AT_RING = 8;     // row-offset ring (tiles)
constexpr float AT_NEG = -1e30f;  // below every finite score; differences of it stay finite

template <int DP>
struct AttnCfg {
    static constexpr int STAGES = DP == 64 ? 4 : DP == 128 ? 3 : 2;
    static constexpr int ROW_BYTES = DP * 2;
    static constexpr int TILE_BYTES = AT_KEYS * ROW_BYTES;       // K or V of a stage
    // Q stays in shared memory only where its fragments do not fit registers
    // (two row tiles at 128, 64 rows at 256); otherwise it passes through the
    // last stage before that stage's first tile.
    static constexpr int Q_BYTES = DP == 64 ? 0 : DP == 128 ? 32 * ROW_BYTES : 64 * ROW_BYTES;
    static constexpr int OFF_STAGE = Q_BYTES;
    static constexpr int OFF_Q_PASS = OFF_STAGE + (STAGES - 1) * 2 * TILE_BYTES;
    static constexpr int OFF_ROW = OFF_STAGE + STAGES * 2 * TILE_BYTES;
    static constexpr int OFF_RED = OFF_ROW + AT_RING * AT_KEYS * 8;  // warps' (m, l): 4 x 32 x 8
    static constexpr int SMEM = OFF_RED + 1024;
};

template <typename T>
struct Mma;
template <>
struct Mma<__half> {
    static __device__ __forceinline__ void run(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ unsigned pack(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const unsigned *>(&h);
    }
};
template <>
struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void run(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
    {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ unsigned pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const unsigned *>(&h);
    }
};

__device__ __forceinline__ void ldsm4(unsigned (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(unsigned (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// 16 bytes global -> shared; zeros where !take (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte offset of 16-byte chunk c of row r in a tile.
template <int DP>
__device__ __forceinline__ uint32_t tile_off(int r, int c)
{
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// Cache row of key j of a page table in elements from the cache's base; -1
// for a page that is not there (recorded).
__device__ __forceinline__ long long key_row(const AttnParams &p, const int32_t *table, int j)
{
    const int page = __ldg(table + (j >> p.page_shift));
    if (page < 0 || page >= p.n_pages) {
        atomicCAS(p.status, 0u, ST_BAD_ID);
        return -1;
    }
    return static_cast<long long>(page) * p.page_stride +
           static_cast<long long>(j & ((1 << p.page_shift) - 1)) * p.row_stride;
}

// The suffix rows that every query of a sequence sees: all but the last
// n_q - 1 (never negative).
__device__ __forceinline__ int suffix_length(const AttnParams &p, int b)
{
    const int n = __ldg(p.suffix_len + b);
    return n < 0 ? 0 : n > p.max_suffix ? p.max_suffix : n;
}

// One warp's work on one stage: MT row tiles of 16 (Q at q_smem, row 16 *
// m0), 16 * NK keys from key k0 of the stage.  s_rowoff tells absent keys.
template <typename T, int DP, int MT, int NK, bool QREG>
struct WarpTile {
    float o[MT][DP / 8][4];
    float m[MT][2], l[MT][2];
    unsigned qf[QREG ? MT : 1][QREG ? DP / 16 : 1][4];

    __device__ __forceinline__ void load_q(unsigned (&f)[4], uint32_t q_s, int row0, int ks, int lane)
    {
        // a0: rows 0-7 k 0-7, a1: rows 8-15 k 0-7, a2: rows 0-7 k 8-15, a3: rows 8-15 k 8-15
        ldsm4(f, q_s + tile_off<DP>(row0 + (lane & 15), 2 * ks + (lane >> 4)));
    }

    __device__ __forceinline__ void init(uint32_t q_s, int m0, int lane)
    {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
            m[i][0] = m[i][1] = AT_NEG;
            l[i][0] = l[i][1] = 0.0f;
            if constexpr (QREG) {
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) load_q(qf[i][ks], q_s, 16 * (m0 + i), ks, lane);
            }
        }
    }

    __device__ __forceinline__ void step(uint32_t q_s, uint32_t k_s, uint32_t v_s, int m0, int k0,
                                         const long long *rowoff, bool masked, float scale_log2, int lane)
    {
        float s[MT][2 * NK][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][n][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            unsigned a[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if constexpr (QREG) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[i][e] = qf[i][ks][e];
                } else {
                    load_q(a[i], q_s, 16 * (m0 + i), ks, lane);
                }
            }
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                unsigned b[4];  // keys 0-7: d 0-7, d 8-15; keys 8-15: d 0-7, d 8-15
                ldsm4(b, k_s + tile_off<DP>(k0 + 16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    Mma<T>::run(s[i][2 * n], a[i], b[0], b[1]);
                    Mma<T>::run(s[i][2 * n + 1], a[i], b[2], b[3]);
                }
            }
        }
        if (masked) {
#pragma unroll
            for (int n = 0; n < 2 * NK; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (rowoff[k0 + 8 * n + 2 * (lane & 3) + e] < 0) {
#pragma unroll
                        for (int i = 0; i < MT; ++i) s[i][n][e] = s[i][n][e + 2] = -INFINITY;
                    }
        }
        unsigned pf[MT][NK][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {  // rows lane / 4 and lane / 4 + 8
                float mx = AT_NEG;
#pragma unroll
                for (int n = 0; n < 2 * NK; ++n) mx = fmaxf(mx, fmaxf(s[i][n][2 * hh], s[i][n][2 * hh + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                const float mn = fmaxf(m[i][hh], mx * scale_log2);
                const float c = ex2(m[i][hh] - mn);
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < 2 * NK; ++n) {
                    const float w0 = ex2(fmaf(s[i][n][2 * hh], scale_log2, -mn));
                    const float w1 = ex2(fmaf(s[i][n][2 * hh + 1], scale_log2, -mn));
                    sum += w0 + w1;
                    // The weights enter the product with v as its type's operands, off by
                    // half a unit of it at most (the largest, 1, by nothing): as much as
                    // one value of v.  The sum keeps them whole, so lse loses nothing.
                    pf[i][n >> 1][2 * (n & 1) + hh] = Mma<T>::pack(w0, w1);
                }
                m[i][hh] = mn;
                l[i][hh] = l[i][hh] * c + sum;  // this lane's keys; the quad's lanes are added at the end
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[i][n][2 * hh] *= c;
                    o[i][n][2 * hh + 1] *= c;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NK; ++n) {
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                unsigned b[4];  // d 0-7: keys 0-7, keys 8-15; d 8-15: keys 0-7, keys 8-15
                ldsm4t(b, v_s + tile_off<DP>(k0 + 16 * n + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    Mma<T>::run(o[i][2 * c], pf[i][n], b[0], b[1]);
                    Mma<T>::run(o[i][2 * c + 1], pf[i][n], b[2], b[3]);
                }
            }
        }
    }

    __device__ __forceinline__ void finish_l()
    {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                l[i][hh] += __shfl_xor_sync(0xFFFFFFFFu, l[i][hh], 1);
                l[i][hh] += __shfl_xor_sync(0xFFFFFFFFu, l[i][hh], 2);
            }
    }
};

// What a block works on.
struct Part {
    const int32_t *table;  // page table of the keys
    int k0, k1;            // keys [k0, k1) of it
    int row0, nrows;       // rows [row0, row0 + nrows) of the cache head
    int head;              // cache head
    int slot;
};

template <typename T, int DP>
struct Block {
    using C = AttnCfg<DP>;
    const AttnParams &p;
    const Part &w;
    uint8_t *smem;
    long long *rowoff;  // [AT_RING][AT_KEYS]
    int tiles;

    __device__ __forceinline__ uint32_t k_stage(int t) const
    {
        return smem_addr(smem + C::OFF_STAGE + (t % C::STAGES) * 2 * C::TILE_BYTES);
    }

    // Row offsets of tile t: one key a thread; keys past the range are absent.
    __device__ __forceinline__ long long find_row(int t) const
    {
        const int j = w.k0 + t * AT_KEYS + static_cast<int>(threadIdx.x);
        return j < w.k1 ? key_row(p, w.table, j) : -1;
    }

    __device__ __forceinline__ void issue(int t) const
    {
        constexpr int CH = DP / 8;
        const T *kb = static_cast<const T *>(p.k) + static_cast<long long>(w.head) * p.head_stride;
        const T *vb = static_cast<const T *>(p.v) + static_cast<long long>(w.head) * p.head_stride;
        const uint32_t ks = k_stage(t), vs = ks + C::TILE_BYTES;
        const long long *ro = rowoff + (t % AT_RING) * AT_KEYS;
        const int c = static_cast<int>(threadIdx.x) % CH;
#pragma unroll
        for (int i = 0; i < AT_KEYS * CH / AT_THREADS; ++i) {
            const int r = static_cast<int>(threadIdx.x) / CH + i * (AT_THREADS / CH);
            const long long off = ro[r];
            const bool take = off >= 0 && c * 8 < p.d;
            const long long at = take ? off + c * 8 : 0;
            const uint32_t d = tile_off<DP>(r, c);
            cp16(ks + d, kb + at, take);
            cp16(vs + d, vb + at, take);
        }
    }

    // Q rows of the tile into shared memory (zeros past the rows).
    __device__ __forceinline__ void load_q(uint32_t q_s, int rows_pad) const
    {
        constexpr int CH = DP / 8;
        for (int i = threadIdx.x; i < rows_pad * CH; i += AT_THREADS) {
            const int r = i / CH, c = i % CH;
            const bool take = r < w.nrows && c * 8 < p.d;
            long long at = 0;
            if (take) {
                const int row = w.row0 + r, tok = row / p.group, g = row - tok * p.group;
                at = tok * p.q_token_stride + (static_cast<long long>(w.head) * p.group + g) * p.q_head_stride + c * 8;
            }
            cp16(q_s + tile_off<DP>(r, c), static_cast<const T *>(p.q) + at, take);
        }
    }

    // The pipeline: init() once Q is there, body(k, v, row offsets, masked) per tile.
    template <typename Init, typename Body>
    __device__ __forceinline__ void run(uint32_t q_s, int rows_pad, Init init, Body body) const
    {
        constexpr int S = C::STAGES;
        __shared__ int s_absent;
        const int tid = threadIdx.x;
        if (tid == 0) s_absent = 0;
        for (int t = 0; t < S; ++t)
            if (tid < AT_KEYS) rowoff[t * AT_KEYS + tid] = find_row(t);
        load_q(q_s, rows_pad);
        asm volatile("cp.async.commit_group;" ::: "memory");
        __syncthreads();
        // a page of the first tiles that is not there (past the range does not count)
        for (int t = 0; t < S; ++t)
            if (tid < AT_KEYS && w.k0 + t * AT_KEYS + tid < w.k1 && rowoff[t * AT_KEYS + tid] < 0) s_absent = 1;
#pragma unroll
        for (int t = 0; t < S - 1; ++t) {
            if (t < tiles) issue(t);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");  // Q
        __syncthreads();
        init();  // read before the first barrier below, after which Q's stage may be filled
        for (int t = 0; t < tiles; ++t) {
            const long long next = tid < AT_KEYS ? find_row(t + S) : 0;
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncthreads();  // tile t is there for all, and stage (t - 1) % S has been read by all
            if (t + S - 1 < tiles) issue(t + S - 1);
            asm volatile("cp.async.commit_group;" ::: "memory");
            const uint32_t ks = k_stage(t);
            const bool masked = s_absent != 0 || w.k0 + (t + 1) * AT_KEYS > w.k1;
            body(ks, ks + C::TILE_BYTES, rowoff + (t % AT_RING) * AT_KEYS, masked);
            if (tid < AT_KEYS) {
                rowoff[((t + S) % AT_RING) * AT_KEYS + tid] = next;
                if (next < 0 && w.k0 + (t + S) * AT_KEYS + tid < w.k1) s_absent = 1;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }

    __device__ __forceinline__ long long out_row(int row) const
    {
        return (static_cast<long long>(w.slot) * p.hkv + w.head) * p.rows + row;
    }

    // Tall tiles: warp i has rows 16 i ..
    __device__ __forceinline__ void by_rows() const
    {
        constexpr bool QREG = DP <= 128;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const uint32_t q_s = smem_addr(smem + (QREG ? C::OFF_Q_PASS : 0));
        WarpTile<T, DP, 1, 4, QREG> a;
        const bool active = 16 * warp < w.nrows;
        run(q_s, 64, [&] { a.init(q_s, warp, lane); },
            [&](uint32_t ks, uint32_t vs, const long long *ro, bool masked) {
                if (active) a.step(q_s, ks, vs, warp, 0, ro, masked, p.scale_log2, lane);
            });
        a.finish_l();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = 16 * warp + (lane >> 2) + 8 * hh;
            if (r >= w.nrows) continue;
            const long long row = out_row(w.row0 + r);
            if ((lane & 3) == 0) p.part_ml[row] = make_float2(a.m[0][hh], a.l[0][hh]);
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) {
                const int c = 8 * n + 2 * (lane & 3);
                if (c < p.d)
                    *reinterpret_cast<float2 *>(p.part_o + row * p.d + c) =
                        make_float2(a.o[0][n][2 * hh], a.o[0][n][2 * hh + 1]);
            }
        }
    }

    // Low tiles: warp i has keys 16 i .. of every stage; the warps' results merge in shared memory.
    template <int MT>
    __device__ __forceinline__ void by_keys() const
    {
        constexpr bool QREG = MT * DP <= 128;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const uint32_t q_s = smem_addr(smem + (QREG ? C::OFF_Q_PASS : 0));
        WarpTile<T, DP, MT, 1, QREG> a;
        run(q_s, 16 * MT, [&] { a.init(q_s, 0, lane); },
            [&](uint32_t ks, uint32_t vs, const long long *ro, bool masked) {
                a.step(q_s, ks, vs, 0, 16 * warp, ro, masked, p.scale_log2, lane);
            });
        a.finish_l();
        float2 *red = reinterpret_cast<float2 *>(smem + C::OFF_RED);  // [4][32]
        float *acc = reinterpret_cast<float *>(smem + C::OFF_STAGE);  // [4][16 MT][DP]
        if ((lane & 3) == 0) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    red[warp * 32 + 16 * i + (lane >> 2) + 8 * hh] = make_float2(a.m[i][hh], a.l[i][hh]);
        }
        __syncthreads();  // the stages have been read, too
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = 16 * i + (lane >> 2) + 8 * hh;
                float mx = red[r].x, l = 0.0f;
#pragma unroll
                for (int u = 1; u < 4; ++u) mx = fmaxf(mx, red[u * 32 + r].x);
#pragma unroll
                for (int u = 0; u < 4; ++u) l += red[u * 32 + r].y * ex2(red[u * 32 + r].x - mx);
                const float c = ex2(a.m[i][hh] - mx);
                if (warp == 0 && (lane & 3) == 0 && r < w.nrows)
                    p.part_ml[out_row(w.row0 + r)] = make_float2(mx, l);
#pragma unroll
                for (int n = 0; n < DP / 8; ++n)
                    *reinterpret_cast<float2 *>(acc + (warp * 16 * MT + r) * DP + 8 * n + 2 * (lane & 3)) =
                        make_float2(a.o[i][n][2 * hh] * c, a.o[i][n][2 * hh + 1] * c);
            }
        __syncthreads();
        for (int i = threadIdx.x; i < w.nrows * (DP / 4); i += AT_THREADS) {
            const int r = i / (DP / 4), c = i % (DP / 4) * 4;
            if (c >= p.d) continue;
            float4 v = *reinterpret_cast<const float4 *>(acc + r * DP + c);
#pragma unroll
            for (int u = 1; u < 4; ++u) {
                const float4 x = *reinterpret_cast<const float4 *>(acc + (u * 16 * MT + r) * DP + c);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            *reinterpret_cast<float4 *>(p.part_o + out_row(w.row0 + r) * p.d + c) = v;
        }
    }
};

template <typename T, int DP>
__global__ void __launch_bounds__(AT_THREADS, DP == 256 ? 1 : 2) attn_part_kernel(const __grid_constant__ AttnParams p)
{
    using C = AttnCfg<DP>;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_wait();
    // Only now: the prefix kernel on tcgen05, launched next, does not wait
    // for this one, so it must not start before what this one waited for.
    pdl_launch_dependents();
    Part w;
    int id = blockIdx.x, tile_rows;
    if (id < p.p_blocks) {  // row tiles innermost: blocks that run together share their keys in L2
        const int rt = id % p.p_tiles;
        id /= p.p_tiles;
        w.head = id % p.hkv;
        const int split = id / p.hkv;
        w.slot = p.p_first + split;
        w.row0 = rt * p.p_tile;
        w.nrows = min(p.p_tile, p.rows - w.row0);
        w.table = p.prefix_pages;
        w.k0 = p.t_len + split * p.p_keys;
        w.k1 = min(p.prefix_len, w.k0 + p.p_keys);
        tile_rows = p.p_tile;
    } else {
        id -= p.p_blocks;
        const int rt = id % p.s_tiles;
        id /= p.s_tiles;
        w.head = id % p.hkv;
        id /= p.hkv;
        const int b = id % p.n_seqs, chunk = id / p.n_seqs;
        w.slot = p.p_first + p.p_splits + chunk;
        const int per = p.n_q * p.group;
        w.row0 = b * per + rt * p.s_tile;
        w.nrows = min(p.s_tile, per - rt * p.s_tile);
        w.table = p.suffix_pages + b * p.suffix_pages_stride;
        w.k0 = chunk * p.s_keys;
        w.k1 = min(suffix_length(p, b) - p.n_q + 1, w.k0 + p.s_keys);
        if (w.k1 <= w.k0) return;
        tile_rows = p.s_tile;
    }
    const Block<T, DP> blk{p, w, smem, reinterpret_cast<long long *>(smem + C::OFF_ROW), (w.k1 - w.k0 + AT_KEYS - 1) / AT_KEYS};
    if (tile_rows == 16)
        blk.template by_keys<1>();
    else if (tile_rows == 32) {
        if constexpr (DP <= 128) blk.template by_keys<2>();
    } else
        blk.by_rows();
}

// ------------------------------------------------------------- combining

__device__ __forceinline__ void put(float *o, float v) { *o = v; }
__device__ __forceinline__ void put(__half *o, float v) { *o = __float2half_rn(v); }
__device__ __forceinline__ void put(__nv_bfloat16 *o, float v) { *o = __float2bfloat16_rn(v); }
__device__ __forceinline__ float get(const __half *v) { return __half2float(*v); }
__device__ __forceinline__ float get(const __nv_bfloat16 *v) { return __bfloat162float(*v); }

constexpr int CB_WARPS = 8;   // warps of a combining block
constexpr int CB_BATCH = 4;   // parts whose loads are in flight per warp

// W warps per row, 8 / W rows per block.  A row's warp w takes every W-th
// part, CB_BATCH of them in flight; a lane has four adjacent elements of each
// 128 (E in all).  Few rows: the latency of the parts' loads bounds it, so a
// row has all eight warps.  Many rows: the parts' bytes (from L2) do, and one
// warp a row saves the merge through shared memory.
template <typename T, typename TO, int W, int E>
__global__ void __launch_bounds__(CB_WARPS * 32) attn_combine_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float s_o[W > 1 ? W : 1][W > 1 ? 32 * E : 1];
    __shared__ float2 s_ml[W];
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = W > 1 ? threadIdx.x >> 5 : 0;
    const int out_row = W > 1 ? blockIdx.x : blockIdx.x * CB_WARPS + (threadIdx.x >> 5);
    if (out_row >= p.n_seqs * p.n_q * p.hq) return;  // W == 1 only: no barrier follows
    const int tok = out_row / p.hq, h = out_row - tok * p.hq;
    const int g = h / p.group, b = tok / p.n_q, i = tok - b * p.n_q;
    const int row = tok * p.group + (h - g * p.group);
    pdl_wait();
    const int len = suffix_length(p, b);
    const int shared_by_all = max(0, len - p.n_q + 1);
    const int parts = p.p_first + p.p_splits + (shared_by_all + p.s_keys - 1) / p.s_keys;
    if (h == 0 && i == 0 && warp == 0 && lane == 0 && __ldg(p.suffix_len + b) != len) atomicCAS(p.status, 0u, ST_BAD_ID);
    float m = AT_NEG, l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;

    auto add = [&](float mp, float lp, const float (&op)[E]) {
        const float mn = fmaxf(m, mp), c = ex2(m - mn), cp = ex2(mp - mn);
        m = mn;
        l = l * c + lp * cp;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + op[e] * cp;
    };
    // element e of this lane is at lane 4 + 128 (e / 4) + e % 4
    const long long stride = static_cast<long long>(p.hkv) * p.rows, first = static_cast<long long>(g) * p.rows + row;
    for (int s0 = warp; s0 < parts; s0 += W * CB_BATCH) {
        float2 ml[CB_BATCH];
        float op[CB_BATCH][E];
#pragma unroll
        for (int u = 0; u < CB_BATCH; ++u) {
            const int s = s0 + u * W;
            ml[u] = make_float2(AT_NEG, 0.0f);
#pragma unroll
            for (int e = 0; e < E; ++e) op[u][e] = 0.0f;
            if (s < parts) {
                const long long at = first + s * stride;
                ml[u] = p.part_ml[at];
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const int c = 4 * lane + 32 * e;
                    if (c < p.d) {
                        const float4 v = *reinterpret_cast<const float4 *>(p.part_o + at * p.d + c);
                        op[u][e] = v.x, op[u][e + 1] = v.y, op[u][e + 2] = v.z, op[u][e + 3] = v.w;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < CB_BATCH; ++u) add(ml[u].x, ml[u].y, op[u]);
    }
    // the suffix rows that only the later queries see, one a step
    const T *q = static_cast<const T *>(p.q) + tok * p.q_token_stride + h * p.q_head_stride;
    const int32_t *table = p.suffix_pages + b * p.suffix_pages_stride;
    for (int j = shared_by_all + warp; j <= len - p.n_q + i; j += W) {
        const long long off = key_row(p, table, j);
        if (off < 0) continue;
        const T *k = static_cast<const T *>(p.k) + off + g * p.head_stride;
        const T *v = static_cast<const T *>(p.v) + off + g * p.head_stride;
        float dot = 0.0f, op[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = 4 * lane + 128 * (e / 4) + e % 4;
            op[e] = 0.0f;
            if (c < p.d) {
                dot = fmaf(get(q + c), get(k + c), dot);
                op[e] = get(v + c);
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
        add(dot * p.scale_log2, 1.0f, op);
    }
    TO *out = static_cast<TO *>(p.o) + tok * p.o_token_stride + h * p.o_head_stride;
    float mx = m, total = l;
    if constexpr (W == 1) {
        const float inv = 1.0f / total;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = 4 * lane + 128 * (e / 4) + e % 4;
            if (c < p.d) put(out + c, total == 0.0f ? 0.0f : o[e] * inv);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4 *>(&s_o[warp][4 * lane + 32 * e]) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        float c[W];
        mx = s_ml[0].x;
        total = 0.0f;
#pragma unroll
        for (int u = 1; u < W; ++u) mx = fmaxf(mx, s_ml[u].x);
#pragma unroll
        for (int u = 0; u < W; ++u) {
            c[u] = ex2(s_ml[u].x - mx);
            total += s_ml[u].y * c[u];
        }
        const int e = threadIdx.x;
        if (e < p.d) {
            float v = 0.0f;
#pragma unroll
            for (int u = 0; u < W; ++u) v = fmaf(s_o[u][e], c[u], v);
            put(out + e, total == 0.0f ? 0.0f : v * (1.0f / total));
        }
    }
    if (p.lse && warp == 0 && lane == 0)
        p.lse[static_cast<long long>(tok) * p.hq + h] =
            total != 0.0f ? (mx + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, typename TO>
cudaError_t launch_combine(const AttnParams &p, cudaStream_t st)
{
    const unsigned rows = static_cast<unsigned>(p.n_seqs * p.n_q * p.hq);
    // eight warps a row up to four waves of blocks (152 multiprocessors, eight blocks each)
    if (rows <= 608)
        return p.d <= 128 ? launch_pdl(attn_combine_kernel<T, TO, 8, 4>, dim3(rows), CB_WARPS * 32, 0, st, p)
                          : launch_pdl(attn_combine_kernel<T, TO, 8, 8>, dim3(rows), CB_WARPS * 32, 0, st, p);
    const dim3 grid((rows + CB_WARPS - 1) / CB_WARPS);
    return p.d <= 128 ? launch_pdl(attn_combine_kernel<T, TO, 1, 4>, grid, CB_WARPS * 32, 0, st, p)
                      : launch_pdl(attn_combine_kernel<T, TO, 1, 8>, grid, CB_WARPS * 32, 0, st, p);
}

template <typename T, int DP>
cudaError_t launch_part(const AttnParams &p, cudaStream_t st)
{
    const long long blocks = p.p_blocks + static_cast<long long>(p.n_seqs) * p.hkv * p.s_tiles * p.s_splits;
    if (blocks == 0) return cudaSuccess;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void *>(attn_part_kernel<T, DP>), AttnCfg<DP>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_part_kernel<T, DP>, dim3(static_cast<unsigned>(blocks)), AT_THREADS, AttnCfg<DP>::SMEM, st, p);
}

template <typename T>
cudaError_t launch_type(const AttnParams &p, qgemv_dtype o_type, cudaStream_t st)
{
    const cudaError_t e = p.d <= 64 ? launch_part<T, 64>(p, st) : p.d <= 128 ? launch_part<T, 128>(p, st)
                                                                             : launch_part<T, 256>(p, st);
    if (e != cudaSuccess) return e;
    if (p.t_mode) {
        const cudaError_t t = launch_attn_tc(p, std::is_same<T, __half>::value ? QGEMV_F16 : QGEMV_BF16, st);
        if (t != cudaSuccess) return t;
    }
    return o_type == QGEMV_F32 ? launch_combine<T, float>(p, st) : launch_combine<T, T>(p, st);
}

}  // namespace

int attn_tile_rows(int rows, int d) { return rows <= 16 ? 16 : rows <= 32 && d <= 128 ? 32 : 64; }

cudaError_t launch_attn(const AttnParams &p, qgemv_dtype type, qgemv_dtype o_type, cudaStream_t st)
{
    return type == QGEMV_F16 ? launch_type<__half>(p, o_type, st) : launch_type<__nv_bfloat16>(p, o_type, st);
}

}  // namespace qg
