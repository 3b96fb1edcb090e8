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
// rows) give each warp 16 rows.  Tall batches over long prefixes are attn_tc.cu's.
//
// What bounds it: memory for long suffixes (64 sequences of up to 2048 own
// keys, 8 heads of 128: 269 MB in 52 us, 5.2 TB/s, the SMs idle for a fifth of
// it at the end, where the next launch starts); the chain length, page, key,
// products, part, and then the combining launch, for small batches (two
// sequences on 160 keys 5.5 us, eight on 4096 9.1 us, 16 of up to 1500 own keys
// of 2 heads of 64 7.4 us, of which 3.8 are the combining launch on its own).
// So parts are single tiles of 64 keys as long as they fit the slots: with two
// at least, the first two took 6.5 and 10.4 us.
#include <type_traits>

#include "decode_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int AT_THREADS = 128;
constexpr int AT_KEYS = 64;    // keys of a stage
constexpr int AT_RING = 8;     // row-offset ring (tiles)
constexpr float AT_NEG = -1e30f;  // below every finite score; differences of it stay finite

// Weights are taken 2^AT_LIFT times as large where they enter the product with
// v as f16, which has no exponents below 2^-24: the largest is 1024 instead of 1,
// and what is 2^-35 of it still counts, not 2^-25 (a part of 1024 keys may hold one
// that stands that far above the others).  m holds the reference, so sums and
// parts know nothing of it.  bf16 has fp32's exponents.
template <typename T>
constexpr float AT_LIFT = std::is_same<T, __half>::value ? 10.0f : 0.0f;

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

// A sequence's suffix length within its bounds.  All its queries see all but
// the last n_q - 1 of these rows.
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
                // rounded up, so that no weight exceeds 2^AT_LIFT however large the scores
                const float mn = fmaxf(m[i][hh], __fadd_ru(__fmul_ru(mx, scale_log2), -AT_LIFT<T>));
                const float c = ex2(m[i][hh] - mn);
                float sum = 0.0f;
#pragma unroll
                for (int n = 0; n < 2 * NK; ++n) {
                    const float w0 = ex2(fmaf(s[i][n][2 * hh], scale_log2, -mn));
                    const float w1 = ex2(fmaf(s[i][n][2 * hh + 1], scale_log2, -mn));
                    sum += w0 + w1;
                    // The weights enter the product with v as its type's operands, off by
                    // half a unit of it at most (the largest, a power of two, by nothing):
                    // as much as one value of v, with an fp32 output too.  The sum keeps
                    // them whole, so lse loses nothing.
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

    // Place of a row's (m, l); of its elements 4 c4 .. of the sums.
    __device__ __forceinline__ long long ml_at(int row) const
    {
        return (static_cast<long long>(w.slot) * p.hkv + w.head) * p.rows + row;
    }
    __device__ __forceinline__ float4 *o_at(int row, int c4) const
    {
        return p.part_o + (static_cast<long long>(w.slot) * p.hkv + w.head) * p.rows * (p.d >> 2) + row * p.o_row +
               c4 * p.o_four;
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
            if ((lane & 3) == 0) p.part_ml[ml_at(w.row0 + r)] = make_float2(a.m[0][hh], a.l[0][hh]);
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                if (8 * n < p.d)
                    reinterpret_cast<float2 *>(o_at(w.row0 + r, 2 * n + ((lane & 2) >> 1)))[lane & 1] =
                        make_float2(a.o[0][n][2 * hh], a.o[0][n][2 * hh + 1]);
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
                    p.part_ml[ml_at(w.row0 + r)] = make_float2(mx, l);
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
            *o_at(w.row0 + r, c >> 2) = v;
        }
    }
};

// Heads of up to 64 leave room for a third block on a multiprocessor: 47
// sequences of 4 queries on 2057 keys take 18.3 us instead of 20.5, 64 of one on
// 3700 12.4 instead of 15.9 (15 of 4 on 777: 11.1 instead of 10.3).  The plan
// still counts two, so that the third has room for what the ranges leave over:
// with ranges for 420 blocks the second of these takes 15.9 again.
template <typename T, int DP>
__global__ void __launch_bounds__(AT_THREADS, DP == 256 ? 1 : DP == 64 ? 3 : 2) attn_part_kernel(const __grid_constant__ AttnParams p)
{
    using C = AttnCfg<DP>;
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_wait();
    // Only now: the prefix kernel on tcgen05, launched next, does not wait for
    // this one, so it must not start before what this one waited for.  The
    // combining launch comes in as these blocks end: let in here, its blocks take
    // their issue slots (eight samples: 10.3 us a call in a stream instead of
    // 9.4; let in after the last product 10.0).
    if (p.t_mode) pdl_launch_dependents();
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

__device__ __forceinline__ void put4(float *o, float4 v)
{
    if ((reinterpret_cast<uintptr_t>(o) & 15) == 0) {
        *reinterpret_cast<float4 *>(o) = v;
    } else {
        o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
    }
}
template <typename TO>
__device__ __forceinline__ void put4(TO *o, float4 v)
{
    const unsigned a = Mma<TO>::pack(v.x, v.y), b = Mma<TO>::pack(v.z, v.w);
    if ((reinterpret_cast<uintptr_t>(o) & 7) == 0) {
        *reinterpret_cast<uint2 *>(o) = make_uint2(a, b);
    } else {
        unsigned short *h = reinterpret_cast<unsigned short *>(o);
        h[0] = static_cast<unsigned short>(a), h[1] = static_cast<unsigned short>(a >> 16);
        h[2] = static_cast<unsigned short>(b), h[3] = static_cast<unsigned short>(b >> 16);
    }
}

constexpr int CB_BATCH = 4;   // parts whose loads are in flight per thread

__device__ __forceinline__ float4 get4(const __half *v)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(v);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 get4(const __nv_bfloat16 *v)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(v);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}

// A block combines ROWS rows of a cache head.
//   ROWS = 1: a warp has 128 elements of the row and every splits-th part,
//     eight warps in all: for few rows, where the loads' latency bounds it.
//   ROWS = 8: lane % 8 is the row, a lane has one group of four elements, a
//     warp 16 elements of the head, the block one warp per 16 elements.  For
//     many rows, where the parts' bytes (from L2) do: after the tcgen05
//     kernel, which has a row a thread, the parts lie with the rows innermost,
//     so that it writes and this reads runs of 128 bytes and more.
template <typename T, typename TO, int ROWS>
__global__ void __launch_bounds__(ROWS == 1 ? 512 : 1024) attn_combine_kernel(const __grid_constant__ AttnParams p)
{
    constexpr int ZONE = 7;            // suffix rows that only the later queries see
    constexpr int FOURS = 32 / ROWS;   // groups of four elements per warp
    __shared__ float s_score[ZONE][ROWS];
    __shared__ long long s_off[ZONE][ROWS];
    extern __shared__ __align__(16) float4 s_acc[];  // [splits - 1][groups][32] sums, then as many (m, l)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int groups = ((p.d >> 2) + FOURS - 1) / FOURS, splits = warps / groups;
    const int cg = warp % groups, part0 = warp / groups;
    const int g = blockIdx.y, row0 = blockIdx.x * ROWS;
    const int rl = lane % ROWS, row = row0 + rl, c4 = FOURS * cg + lane / ROWS;
    const bool live = row < p.rows, mine = live && 4 * c4 < p.d;
    // the lane's row: token, query of its sequence, query head
    auto shape = [&](int r, int &tok, int &i, int &h, int &len) {
        tok = r / p.group;
        h = g * p.group + r - tok * p.group;
        const int b = tok / p.n_q;
        i = tok - b * p.n_q;
        len = suffix_length(p, b);
    };
    pdl_wait();
    int tok = 0, i = 0, h = 0, len = 0;
    if (live) shape(row, tok, i, h, len);
    if (live && h == 0 && i == 0 && warp == 0 && lane < ROWS && __ldg(p.suffix_len + tok / p.n_q) != len)
        atomicCAS(p.status, 0u, ST_BAD_ID);

    const int shared_by_all = max(0, len - p.n_q + 1);
    const int parts = live ? p.p_first + p.p_splits + (shared_by_all + p.s_keys - 1) / p.s_keys : 0;
    const long long ml_stride = static_cast<long long>(p.hkv) * p.rows, ml0 = static_cast<long long>(g) * p.rows + row;
    const long long o_stride = ml_stride * (p.d >> 2);
    const long long o0 = static_cast<long long>(g) * p.rows * (p.d >> 2) + row * p.o_row + c4 * p.o_four;
    const int most = __reduce_max_sync(0xFFFFFFFFu, parts);
    float2 ml[CB_BATCH];
    float4 op[CB_BATCH];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int u = 0; u < CB_BATCH; ++u) {
            const int s = s0 + u * splits;
            ml[u] = make_float2(AT_NEG, 0.0f);
            op[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s < parts && mine) {
                ml[u] = p.part_ml[ml0 + s * ml_stride];
                op[u] = p.part_o[o0 + s * o_stride];
            }
        }
    };
    // Few rows: on their way during what follows.  (With eight rows a block the
    // registers that this takes spill, which costs more.)
    if (ROWS == 1) fetch(part0);

    // The rows that not all of a sequence's queries see: a warp per (key, row)
    // takes the score (a lane finds each of its keys first), the lanes add the
    // value below.
    if (p.n_q > 1) {
        const int count = (p.n_q - 1) * ROWS;
        for (int base = 0; warp + base * warps < count; base += 32) {  // 32 of the warp's at a time
            long long off = -1, q_at = 0;
            const int e0 = warp + (base + lane) * warps;
            if (e0 < count && row0 + e0 % ROWS < p.rows) {
                int rt, ri, rh, rn;
                shape(row0 + e0 % ROWS, rt, ri, rh, rn);
                const int j = max(0, rn - p.n_q + 1) + e0 / ROWS;
                if (j <= rn - p.n_q + ri) off = key_row(p, p.suffix_pages + rt / p.n_q * p.suffix_pages_stride, j);
                q_at = rt * p.q_token_stride + rh * p.q_head_stride;
            }
            for (int n = 0; n < 32 && warp + (base + n) * warps < count; n += 4) {
                float dot[4];
                long long oo[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    oo[u] = __shfl_sync(0xFFFFFFFFu, off, n + u);
                    const long long qq = __shfl_sync(0xFFFFFFFFu, q_at, n + u);
                    dot[u] = 0.0f;
                    if (oo[u] >= 0) {
                        const T *q = static_cast<const T *>(p.q) + qq;
                        const T *k = static_cast<const T *>(p.k) + oo[u] + g * p.head_stride;
                        for (int c = 4 * lane; c < p.d; c += 128) {
                            const float4 a = get4(q + c), b = get4(k + c);
                            dot[u] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, dot[u]))));
                        }
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1)
#pragma unroll
                    for (int u = 0; u < 4; ++u) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], d);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = warp + (base + n + u) * warps;
                    if (lane == 0 && e < count) {
                        s_score[e / ROWS][e % ROWS] = dot[u] * p.scale_log2;
                        s_off[e / ROWS][e % ROWS] = oo[u];
                    }
                }
            }
        }
        __syncthreads();
    }

    float m = AT_NEG, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float mp, float lp, float4 op) {
        const float mn = fmaxf(m, mp), c = ex2(m - mn), cp = ex2(mp - mn);
        m = mn;
        l = l * c + lp * cp;
        o.x = o.x * c + op.x * cp;
        o.y = o.y * c + op.y * cp;
        o.z = o.z * c + op.z * cp;
        o.w = o.w * c + op.w * cp;
    };
    for (int s0 = part0; s0 < most; s0 += splits * CB_BATCH) {
        if (ROWS != 1 || s0 != part0) fetch(s0);
#pragma unroll
        for (int u = 0; u < CB_BATCH; ++u) add(ml[u].x, ml[u].y, op[u]);
    }
    if (mine)
        for (int u = part0; u < p.n_q - 1; u += splits) {
            const long long off = s_off[u][rl];
            if (off >= 0)
                add(s_score[u][rl], 1.0f, get4(static_cast<const T *>(p.v) + off + g * p.head_stride + 4 * c4));
        }

    pdl_launch_dependents();  // the next kernel may come while the rows are written
    if (splits > 1) {
        float2 *s_ml = reinterpret_cast<float2 *>(s_acc + (splits - 1) * groups * 32);  // [splits - 1][groups][32]
        if (part0 > 0) {
            s_acc[((part0 - 1) * groups + cg) * 32 + lane] = o;
            s_ml[((part0 - 1) * groups + cg) * 32 + lane] = make_float2(m, l);
        }
        __syncthreads();
        if (part0 > 0) return;
        for (int u = 0; u < splits - 1; ++u) {
            const float2 ml = s_ml[(u * groups + cg) * 32 + lane];
            add(ml.x, ml.y, s_acc[(u * groups + cg) * 32 + lane]);
        }
    }
    if (mine) {
        TO *out = static_cast<TO *>(p.o) + tok * p.o_token_stride + h * p.o_head_stride + 4 * c4;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        put4(out, l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (p.lse && c4 == 0)
            p.lse[static_cast<long long>(tok) * p.hq + h] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <typename T, typename TO>
cudaError_t launch_combine(const AttnParams &p, cudaStream_t st)
{
    const unsigned rows = static_cast<unsigned>(p.rows), heads = static_cast<unsigned>(p.hkv);
    // a row a block up to seven blocks a multiprocessor, unless the rows are innermost
    const bool one = p.o_four == 1 && rows * heads <= 1024;
    const int groups = one ? (p.d + 127) / 128 : (p.d + 15) / 16;
    const dim3 grid(one ? rows : (rows + 7) / 8, heads);
    // warps that share a row's parts: as many as fill the multiprocessors about once
    const unsigned blocks = grid.x * grid.y;
    int splits = one ? 8 : blocks <= ATTN_SMS ? 4 : blocks <= 2 * ATTN_SMS ? 2 : 1;
    // but none without a batch of parts of its own, and past one wave of warps
    // (16 a multiprocessor) none with fewer than four batches: with eight warps
    // whatever the parts, 480 rows of 31 parts took 15.1 us a call instead of 13.5,
    // 960 of 20 parts 18.9 instead of 15.0, and two sequences on 160 keys 5.8
    // instead of 5.5.
    const int parts = p.p_first + p.p_splits + p.s_splits;
    const long long warps = one ? static_cast<long long>(rows) * heads * groups : 0;
    while (splits > 1 && splits / 2 * (warps * splits <= 16 * ATTN_SMS ? CB_BATCH : 4 * CB_BATCH) >= parts) splits /= 2;
    while (splits > 1 && groups * splits > 32) splits /= 2;
    const unsigned threads = static_cast<unsigned>(groups * splits * 32);
    const size_t smem = static_cast<size_t>((splits - 1) * groups * 32) * (sizeof(float4) + sizeof(float2));
    return one ? launch_pdl(attn_combine_kernel<T, TO, 1>, grid, threads, smem, st, p)
               : launch_pdl(attn_combine_kernel<T, TO, 8>, grid, threads, smem, st, p);
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
