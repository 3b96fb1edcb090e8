// kv8_attn.cuh -- attention over a paged cache of 8-bit codes with a scale for
// each block of rows and head, under a sliding window with first rows that stay
// visible (minfer README "How it works": GQA attention whose keys are split
// over blocks and whose partial results are combined).
//
//   s_j = scale ks_j (q . c_j),  o = sum_j 2^(s_j) vs_j d_j / sum_j 2^(s_j)
// with codes c_j of k and d_j of v, scales ks_j and vs_j of their blocks, and
// log2 e folded into scale.  Scales enter where a score or a weight is
// formed, never element by element: w_j = 2^(s_j + log2 vs_j - m) is the matrix
// operand of the product with d_j, with m a running reference near the largest
// s_j + log2 vs_j of the row, and l sums w_j / vs_j in fp32.  So a row's largest
// contribution has the operand's full precision however the scales differ.
// m is set by the first visible keys, 2^10 below their largest, and raised only when
// a weight would pass 2^14: after the first tiles almost never, which saves the
// shuffles of a maximum and the scaling of the sums for each tile.
//
// The products are transposed: scores = K Q^T and sums = V^T P^T, keys or
// elements of a head on the 16 rows of mma.sync, the few query rows of a cache head
// on its 8 columns, so that a group of up to 8 heads wastes nothing.  A thread's
// operands of K are 16 consecutive bytes of a row (the order of d in the
// contraction is free, Q's fragments have the same), of V 16 consecutive bytes of
// each of four rows, joined by byte permutations.  The weights pass from the one
// layout to the other by movmatrix.
//
// A warp streams tiles of 32 keys through a ring of its own in shared memory:
// TMA boxes of 16 rows (a page holds 16 at least, so a half of a tile lies in one),
// swizzled so that the 16-byte reads above meet no bank twice, an mbarrier a stage; the scales
// come by 4-byte copies.  No barrier of the block is met before the end.
//
// A unit is a sequence, cache head and tile of query rows; the warps of its block take its
// tiles in turn and merge once, through the ring.  Short sequences get a block a unit and
// one launch; where such blocks have a multiprocessor each, they have twice the
// warps.  Else ragged batches are balanced
// on the device: the sequences' tiles in one line are cut into as many equal ranges as
// the grid holds for each head and row tile, or, for few sequences, each sequence's
// into ranges of its own; a unit that is cut leaves its sums in the workspace, and a second
// launch joins them in the order of the ranges.  So nothing depends on which block runs when.
//
// What bounds it: up to 16 query rows a cache head the bytes where there are many (64
// sequences of up to 16384 keys, 32 + 8 heads of 128: 180 us, 6.0 TB/s, the copies alone 168;
// rings filled by 16-byte copies of the threads took 210 alone and 239 with the products);
// for few sequences the chain length, table, page, key, sums, join (8 of 256 / 4096 / 16384 keys,
// 16 + 2 heads: 7.0 / 9.3 / 18.7 us, the first 5 us whatever the length).  24 rows a cache head need 96 sums of a thread and
// leave one block of eight warps a multiprocessor, which wait for their own instructions
// most of the time; at 96 elements a head 72 sums and twelve warps, which spill a little
// (window of 4096 keys of 32 sequences, 24 + 4 heads of 96, four queries: 36.1 us; eight warps 40.2,
// as heads of 128 43.5, then in ranges 48.9, and 51.1 where the products of a tile's halves
// follow one another instead of taking turns).  16 keys at once instead of a whole tile
// spare registers and cost 13 to 40 % (32 rows a cache head).  More than 32 rows a cache head (16
// where a head has more than 128 elements) are tiles that stream all keys again, each its own unit: 8
// sequences of 16384 keys, 16 heads of 128 to one, 1 / 2 / 4 / 8 queries 15.1 / 20.7 / 30.4 / 50.4 us.
#pragma once

#include "f32x2.cuh"
#include "kv8_ops.h"
#include "qgemv_internal.cuh"
#include "tma.cuh"

namespace qg {
namespace {

constexpr int KC_THREADS = 256;    // of a block of the combining launch
constexpr float K8_NEG = -1e30f;   // below every finite score; differences of it stay finite
constexpr float K8_LIFT = 10.0f;   // a new reference lies so far below the largest score
constexpr float K8_SLACK = 14.0f;  // weights reach 2^14 before it moves (f16 ends at 2^16)

// DP: head_dim rounded up to 64, 96, 128 or 256; NT: tiles of 8 query rows; WIDE: one block of
// twice the warps a multiprocessor instead of two.
template <int DP, int NT, bool WIDE>
struct K8Cfg {
    static constexpr int KC = (DP + 63) / 64;             // 64-element chunks of a row of K, 96's second one of 32
    static constexpr int VB = DP <= 96 ? 8 : 16;          // bytes of a row of V that a thread takes at once
    static constexpr int VC = (DP + 8 * VB - 1) / (8 * VB);  // such pieces, 96's second one of half as many
    static constexpr int MT = DP / 16;                    // 16-row tiles of the sums
    static constexpr int ROW = DP == 64 ? 64 : 128;       // bytes of a row of a copied box
    static constexpr int BOX = KV8_KEYS * ROW;            // of a tile's box; K has ACROSS of them, then V
    static constexpr int ACROSS = (DP + ROW - 1) / ROW;
    static constexpr int TILE = 2 * ACROSS * BOX;
    static constexpr int BLOCKS = WIDE ? 1 : kv8_blocks(DP, NT);
    static constexpr int WARPS = kv8_warps(DP, NT) * (WIDE ? 2 : 1), THREADS = 32 * WARPS;
    static constexpr int STAGES = DP == 64 ? (NT > 2 ? 4 : 3) : DP <= 128 && NT > 2 ? (WARPS > 8 ? 2 : 3) : 2;
    static constexpr __device__ int k_steps(int c) { return DP == 96 && c ? 2 : 4; }       // of 16 elements in chunk c
    static constexpr __device__ int v_words(int c) { return DP == 96 && c ? 1 : VB / 4; }  // of piece c in a row
    static constexpr bool QREG = DP * NT <= 128;          // Q's fragments in registers
    static constexpr int OFF_META = WARPS * STAGES * TILE;               // per warp and stage: ks, vs of both halves
    static constexpr int OFF_Q = OFF_META + WARPS * STAGES * 16;
    static constexpr int OFF_QS = OFF_Q + 8 * NT * DP * 2;
    static constexpr int OFF_ML = OFF_QS + 8 * NT * 4;
    static constexpr int OFF_BAR = OFF_ML + WARPS * 8 * NT * 8;  // per warp and stage
    static constexpr int SMEM = OFF_BAR + WARPS * STAGES * 8 + 1024;  // boxes begin at 1024 bytes: the swizzle's period
    static_assert(2 * STAGES >= NT, "the warps' sums fit the ring");
    static_assert(BLOCKS * (SMEM + 2048) <= 228 * 1024, "the blocks fit a multiprocessor");
};

__device__ __forceinline__ void cp4_if(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0, unsigned b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from sums of zero.
__device__ __forceinline__ void mma0(float (&d)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0, unsigned b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ unsigned movm(unsigned a)
{
    unsigned d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ unsigned pack(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}

// Four codes as f16, exactly: bytes 0 and 1 to lo, 2 and 3 to hi.
template <int CODE>
__device__ __forceinline__ void cvt4(unsigned w, unsigned &lo, unsigned &hi)
{
    if constexpr (CODE == QGEMV_CODE_INT8) {
        w ^= 0x80808080u;  // 0..255; 0x6400 | b is 1024 + b
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        const unsigned x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&x), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&y), off);
        lo = *reinterpret_cast<const unsigned *>(&a), hi = *reinterpret_cast<const unsigned *>(&b);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}
__device__ __forceinline__ void lds64(uint32_t at, unsigned &x, unsigned &y)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at));
}
// e4m3's NaN codes (a row that no one has written may hold them) as 0.
__device__ __forceinline__ unsigned without_nan(unsigned w)
{
    return w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// Boxes lie in shared memory with the 16-byte chunks of a row swizzled (by the row's
// number, or its half with 64-byte rows).  The product's rows 0 .. 7 are these rows
// of a box's eight, so that neither the reads of K (a row for four lanes, four chunks of it,
// or two for four of 8 bytes) nor those of V (every second row, half of its chunks, or two) meet a
// bank twice.
template <int DP>
__device__ __forceinline__ int box_row(int k)
{
    return DP == 64 ? k ^ (k >> 1 & 1) : DP == 96 ? (k & 1) << 2 | (k & 2) | k >> 2 : (k & 1) << 2 | k >> 1;
}
// Byte offset of chunk c of row r.
template <int DP>
__device__ __forceinline__ int box_off(int r, int c)
{
    return DP == 64 ? r * 64 + ((c ^ (r >> 1 & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

// What a sequence's queries see of it, in tiles: the tiles of the first rows,
// then all from the earliest query's window on.
struct Seen {
    int n;      // rows
    int lead;   // tiles before the gap
    int gap;    // tiles left out
    int tiles;

    __device__ __forceinline__ Seen(const Kv8AttnParams &p, int len)
    {
        n = len < 0 ? 0 : len > p.max_len ? p.max_len : len;
        const int first = p.window ? max(0, n - p.n_q + 1 - p.window) : 0;
        lead = (min(p.sinks, first) + KV8_KEYS - 1) / KV8_KEYS;
        gap = max(0, first / KV8_KEYS - lead);
        tiles = (n + KV8_KEYS - 1) / KV8_KEYS - gap;
    }
    __device__ __forceinline__ int tile(int i) const { return i < lead ? i : i + gap; }
};

template <typename T>
__device__ __forceinline__ void put4(T *o, float4 v);
template <>
__device__ __forceinline__ void put4<float>(float *o, float4 v)
{
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
}
template <>
__device__ __forceinline__ void put4<__half>(__half *o, float4 v)
{
    o[0] = __float2half_rn(v.x), o[1] = __float2half_rn(v.y), o[2] = __float2half_rn(v.z), o[3] = __float2half_rn(v.w);
}
template <>
__device__ __forceinline__ void put4<__nv_bfloat16>(__nv_bfloat16 *o, float4 v)
{
    o[0] = __float2bfloat16_rn(v.x), o[1] = __float2bfloat16_rn(v.y);
    o[2] = __float2bfloat16_rn(v.z), o[3] = __float2bfloat16_rn(v.w);
}

// Query and head within the group of a row: its quotient and remainder by the group's heads
// (rows are below 2^15, so that half a row more times the fp32 reciprocal ends on the right side).
__device__ __forceinline__ int2 query_of(const Kv8AttnParams &p, int row)
{
    const int i = __float2int_rd((static_cast<float>(row) + 0.5f) * p.per_group);
    return make_int2(i, row - i * p.group);
}

// Four elements, from 4 * c on, of row `row` of sequence b and cache head h.
__device__ __forceinline__ void store_o(const Kv8AttnParams &p, int b, int h, int row, int c, float4 v)
{
    const int2 r = query_of(p, row);
    const long long token = static_cast<long long>(b) * p.n_q + r.x;
    const long long at = token * p.o_token_stride + (h * p.group + r.y) * p.o_head_stride + 4 * c;
    if (p.o_type == QGEMV_F32)
        put4(static_cast<float *>(p.o) + at, v);
    else if (p.o_type == QGEMV_F16)
        put4(static_cast<__half *>(p.o) + at, v);
    else
        put4(static_cast<__nv_bfloat16 *>(p.o) + at, v);
}
__device__ __forceinline__ void store_lse(const Kv8AttnParams &p, int b, int h, int row, float m, float l)
{
    if (!p.lse) return;
    const int2 r = query_of(p, row);
    const long long token = static_cast<long long>(b) * p.n_q + r.x;
    p.lse[token * p.hq + h * p.group + r.y] =
        l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// A sequence without rows: zeros for `rows` rows from row0 on of head h.
__device__ __forceinline__ void store_none(const Kv8AttnParams &p, int b, int h, int row0, int rows)
{
    const int quads = p.d / 4;
    for (int i = threadIdx.x; i < rows * quads; i += blockDim.x) {
        const int row = row0 + i / quads, c = i % quads;
        store_o(p, b, h, row, c, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        if (c == 0) store_lse(p, b, h, row, 0.0f, 0.0f);
    }
}

template <int CODE, int DP, int NT, bool WIDE>
__global__ void __launch_bounds__(K8Cfg<DP, NT, WIDE>::THREADS, K8Cfg<DP, NT, WIDE>::BLOCKS) kv8_attn_kernel(
    const __grid_constant__ Kv8AttnParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map)
{
    using C = K8Cfg<DP, NT, WIDE>;
    extern __shared__ __align__(16) uint8_t k8_raw[];
    __shared__ int s_abort;
    uint8_t *k8_smem = k8_raw + ((1024 - (smem_addr(k8_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t s_base = smem_addr(k8_smem);
    const uint32_t s_ring = s_base + warp * C::STAGES * C::TILE;
    const uint32_t s_meta = s_base + C::OFF_META + warp * C::STAGES * 16;
    float *s_qs = reinterpret_cast<float *>(k8_smem + C::OFF_QS);
    float2 *s_ml = reinterpret_cast<float2 *>(k8_smem + C::OFF_ML);

    uint64_t *full = reinterpret_cast<uint64_t *>(k8_smem + C::OFF_BAR) + warp * C::STAGES;
    volatile int *abort_flag = &s_abort;

    pdl_launch_dependents();
    if (lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(warp & 1 ? &v_map : &k_map) : "memory");
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    if (tid == 0) s_abort = 0;
    __syncthreads();
    pdl_wait();

    // The unit: cache head and tile of query rows.  Then the block's range [lo, hi) of
    // tiles, the sequence that it begins in and where that one's tiles begin: along the line of all
    // sequences' tiles, or (aligned, and a block for each unit) within the sequence.
    const int unit = blockIdx.x, per_seq = gridDim.x, no = static_cast<int>(blockIdx.y + blockIdx.z * gridDim.y);
    const int h = p.row_tiles == 1 ? unit : unit / p.row_tiles, row0 = (unit - h * p.row_tiles) * p.tile_rows;
    const int rows = min(p.tile_rows, p.rows - row0), id = no * per_seq + unit;
    int lo, hi, range = 0, seq_at = 0, b;  // in tiles: all of them fit 31 bits
    if (p.balanced) {
        bool mine;  // whether there is a range for this block
        if (p.aligned) {
            // up to 32 sequences, one for each lane, and whole ranges for each of them, so that no block has two
            const int n = lane < p.n_seqs ? __ldg(p.lens + lane) : 0, tiles = Seen(p, n).tiles;
            if ((n < 0 || n > p.max_len) && id == 0 && warp == 0) atomicCAS(p.status, 0u, ST_BAD_ID);
            const int total = __reduce_add_sync(0xFFFFFFFFu, tiles), spare = p.ranges - p.n_seqs;
            range = max(KV8_SPLIT_MIN, (total + spare - 1) / spare);
            const int own = (tiles + range - 1) / range;
            int upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const unsigned behind = __ballot_sync(0xFFFFFFFFu, upto > no);
            mine = behind;
            b = mine ? __ffs(behind) - 1 : 0;
            lo = (no - __shfl_sync(0xFFFFFFFFu, upto - own, b)) * range;
            hi = min(lo + range, __shfl_sync(0xFFFFFFFFu, tiles, b));
        } else {
            // every warp adds all sequences' tiles up, each lane a run of them
            const int run = (p.n_seqs + 31) / 32;
            int tiles = 0;
            for (int i = lane * run; i < min(p.n_seqs, (lane + 1) * run); ++i) {
                const int n = __ldg(p.lens + i);
                tiles += Seen(p, n).tiles;
                if ((n < 0 || n > p.max_len) && id == 0 && warp == 0) atomicCAS(p.status, 0u, ST_BAD_ID);
            }
            int upto = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const int total = __shfl_sync(0xFFFFFFFFu, upto, 31);
            range = max(KV8_SPLIT_MIN, (total + p.ranges - 1) / p.ranges);
            lo = no * range, hi = min(total, lo + range);
            mine = lo < total;
            // the first lane whose run ends behind lo walks its run
            const unsigned behind = __ballot_sync(0xFFFFFFFFu, upto > lo);
            const int owner = behind ? __ffs(behind) - 1 : 0;
            int at = lane * run;
            seq_at = upto - tiles;
            if (lane == owner && mine) {
                for (;; ++at) {
                    const int n = Seen(p, __ldg(p.lens + at)).tiles;
                    if (seq_at + n > lo) break;
                    seq_at += n;
                }
            }
            b = __shfl_sync(0xFFFFFFFFu, at, owner);
            seq_at = __shfl_sync(0xFFFFFFFFu, seq_at, owner);
        }
        for (int i = id; i < p.n_seqs; i += p.grid)
            if (Seen(p, __ldg(p.lens + i)).n == 0) {
                for (int k = 0; k < p.hkv; ++k) store_none(p, i, k, 0, p.rows);
                if (p.parts_by_unit)
                    for (int k = tid; k < per_seq; k += C::THREADS) p.parts[i * per_seq + k] = make_int4(0, 0, 0, 0);
            }
        if (!p.parts_by_unit && tid == 0) p.parts[id] = make_int4(0, 0, 0, 0);
        if (!mine) return;
    } else {
        b = no;
        if (b >= p.n_seqs) return;
        const int n = __ldg(p.lens + b);
        if ((n < 0 || n > p.max_len) && tid == 0) atomicCAS(p.status, 0u, ST_BAD_ID);
        const Seen seen(p, n);
        if (seen.n == 0) {
            store_none(p, b, h, row0, rows);
            return;
        }
        lo = 0, hi = seen.tiles;
    }

    Seen seen(p, __ldg(p.lens + b));
    int pos = lo;
    // where in a box the thread's bytes of K lie (of 64 elements each) and those of V (of two rows)
    const int pg = box_row<DP>(g);
    const uint32_t k_off0 = box_off<DP>(pg, t);
    const uint32_t k_off1 = DP == 96 ? box_off<DP>(pg, 4 + (t >> 1)) + 8 * (t & 1) : box_off<DP>(pg, 4 + t);
    const int v_unit = DP <= 96 ? g : pg;  // of VB elements of a head
    auto v_at = [&](int k) {
        return C::VB == 8 ? box_off<DP>(box_row<DP>(2 * t + k), g >> 1) + 8 * (g & 1) : box_off<DP>(box_row<DP>(2 * t + k), pg);
    };
    const uint32_t v_off0 = v_at(0), v_off1 = v_at(1);
    const uint32_t v_two0 = DP == 96 ? box_off<DP>(box_row<DP>(2 * t), 4 + (g >> 2)) + 4 * (g & 3) : 0;  // of the second piece
    const uint32_t v_two1 = DP == 96 ? box_off<DP>(box_row<DP>(2 * t + 1), 4 + (g >> 2)) + 4 * (g & 3) : 0;
    // the warp's ring: tiles on their way and taken, the next to write and to read, the
    // phases to wait for, and whether pages are there (a bit for each stage, and half of it)
    int sent = 0, taken = 0, slot = 0, rd = 0;
    unsigned phases = 0, absent = 0;
    bool ok = true;
    while (pos < hi) {
        const int i0 = pos - seq_at, i1 = min(seen.tiles, hi - seq_at);

        // ---- the warp's tiles i0 + warp, + WARPS, ... on their way
        const int32_t *table = p.pages + b * p.pages_stride;
        const float *st = (lane & 1 ? p.c.vs : p.c.ks) + h * p.c.scale_head;  // lanes 0 .. 3: k and v of the halves
        const bool split = p.c.page_shift == 4;  // a tile's halves lie on pages of their own
        auto page_of = [&](int i, int half) {
            const int j = seen.tile(i) * KV8_KEYS + 16 * half;
            return i < i1 && j < seen.n ? __ldg(table + (j >> p.c.page_shift)) : 0;
        };
        // a lane for each box: of K and V, of each 128 elements, of each half where it is split
        constexpr int ACROSS = C::ACROSS;
        const bool box_v = lane & 1;
        const int box_x = (lane >> 1) % ACROSS, box_half = (lane >> 1) / ACROSS;
        const bool boxes = lane < 2 * ACROSS * (split ? 2 : 1);
        const uint32_t box_to = s_ring + (box_v ? ACROSS * C::BOX : 0) + box_x * C::BOX + box_half * 16 * C::ROW;
        int ahead = i0 + warp;
        int page = page_of(ahead, 0), page1 = split ? page_of(ahead, 1) : page;
        auto issue = [&]() {
            if (ahead < i1 && ok) {
                const int j0 = seen.tile(ahead) * KV8_KEYS, in_page = j0 & ((1 << p.c.page_shift) - 1);
                const unsigned n_pages = static_cast<unsigned>(p.c.n_pages);
                const bool here = static_cast<unsigned>(page) < n_pages, here1 = static_cast<unsigned>(page1) < n_pages;
                absent = (absent & ~(3u << 2 * slot)) |
                         (static_cast<unsigned>(!here) | static_cast<unsigned>(!here1) << 1) << 2 * slot;
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + slot, C::TILE);
                    if (!here || !here1) atomicCAS(p.status, 0u, ST_BAD_ID);
                }
                __syncwarp();
                if (boxes) {  // a page that is not there reads as zeros: beyond the tensor
                    const int at = box_half ? here1 ? page1 : static_cast<int>(n_pages) : here ? page : static_cast<int>(n_pages);
                    tma_load4(box_to + slot * C::TILE, box_v ? &v_map : &k_map, box_x * C::ROW, in_page, h, at, full + slot);
                }
                if (lane < 4) {
                    const int row = split ? 0 : in_page + 16 * (lane >> 1), pg = lane & 2 ? page1 : page;
                    const bool take = j0 + 16 * (lane >> 1) < seen.n && (lane & 2 ? here1 : here);
                    const long long sc = pg * p.c.scale_page + (row >> p.c.block_shift) * p.c.scale_block;
                    cp4_if(s_meta + slot * 16 + lane * 4, st + (take ? sc : 0), take);
                }
                ++sent;
                slot = slot + 1 == C::STAGES ? 0 : slot + 1;
                ahead += C::WARPS;
                page = page_of(ahead, 0);
                page1 = split ? page_of(ahead, 1) : page;
            }
            cp_commit();
        };
        // the unit's queries on their way too
        constexpr int QR = (8 * NT + C::WARPS - 1) / C::WARPS;  // rows of a warp
        uint4 q_raw[QR];
#pragma unroll
        for (int k = 0; k < QR; ++k) {
            const int r = warp + k * C::WARPS, row = row0 + r;
            q_raw[k] = make_uint4(0, 0, 0, 0);
            if (r < rows && 8 * lane < p.d) {
                const int2 at = query_of(p, row);
                const long long token = static_cast<long long>(b) * p.n_q + at.x;
                q_raw[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + token * p.q_token_stride +
                                                                 (h * p.group + at.y) * p.q_head_stride + 8 * lane));
            }
        }
#pragma unroll 1
        for (int s = 0; s < C::STAGES - 1; ++s) issue();

        // ---- queries in f16; bf16 rows divided by a power of two
#pragma unroll
        for (int k = 0; k < QR; ++k) {
            const int r = warp + k * C::WARPS;
            if (r >= 8 * NT) break;
            uint4 w = q_raw[k];
            float qs = p.scale_log2;
            if (p.q_bf16) {
                unsigned u[4] = {w.x, w.y, w.z, w.w};
                unsigned top = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max(top, max((u[i] << 16) & 0x7FFFFFFFu, u[i] & 0x7FFF0000u));
                top = __reduce_max_sync(0xFFFFFFFFu, top);
                // the power of two of the row's largest value; infinities and NaN as they are
                int e = static_cast<int>(top >> 23);
                if (e == 255 || top == 0) e = 127;
                e = min(max(e, 2), 252);
                const float down = __uint_as_float(static_cast<unsigned>(254 - e) << 23);  // 2^(127 - e)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u[i] = pack(__uint_as_float(u[i] << 16) * down, __uint_as_float(u[i] & 0xFFFF0000u) * down);
                w = make_uint4(u[0], u[1], u[2], u[3]);
                qs *= __uint_as_float(static_cast<unsigned>(e) << 23);
            }
            // chunk c of a row lies at c ^ (row & 1): the fragments' reads meet no bank twice
            if (8 * lane < DP) *reinterpret_cast<uint4 *>(k8_smem + C::OFF_Q + r * DP * 2 + ((lane ^ (r & 1)) << 4)) = w;
            if (lane == 0) s_qs[r] = qs;
        }
        __syncthreads();

        const uint32_t q_at = s_base + C::OFF_Q + g * DP * 2 + 32 * t, q_x = (g & 1) << 4;
        auto load_q = [&](int j, int c, unsigned (&f)[8]) {  // 16 elements 64 c + 16 t .. of row 8 j + g
#pragma unroll
            for (int x = 0; x < C::k_steps(c) / 2; ++x) {
                const uint32_t at = DP == 96 && c ? s_base + C::OFF_Q + g * DP * 2 + 128 + (16 * t ^ q_x)
                                                  : q_at + (16 * x ^ q_x) + 128 * c;
                const uint4 v = lds128(at + 8 * j * DP * 2);
                f[4 * x] = v.x, f[4 * x + 1] = v.y, f[4 * x + 2] = v.z, f[4 * x + 3] = v.w;
            }
        };
        unsigned qf[C::QREG ? NT : 1][C::QREG ? C::KC : 1][8];
        if constexpr (C::QREG) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < C::KC; ++c) load_q(j, c, qf[j][c]);
        }
        // per thread, rows 8 j + 2 t and + 1: factor, minus the reference (0, and a bit of `unset`,
        // before the first visible key), sum of the weights over their scales, sums of v
        float2 qs[NT], nm[NT], l[NT];
        float o[NT][C::MT][4];
        unsigned unset = (1u << 2 * NT) - 1;
        bool fresh = true;  // a row of the warp is unset
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            qs[j] = *reinterpret_cast<const float2 *>(s_qs + 8 * j + 2 * t);
            nm[j] = l[j] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < C::MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][i][e] = 0.0f;
        }

        // The references that a tile with exponents s, relative to them (-infinity: not seen), asks for.
        auto raise = [&](float (&s)[2][NT][4]) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(fmaxf(s[0][j][e], s[0][j][2 + e]), fmaxf(s[1][j][e], s[1][j][2 + e]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
                    const unsigned bit = 1u << (2 * j + e);
                    if (unset & bit ? mx > K8_NEG : mx > K8_SLACK) {
                        const float up = mx - K8_LIFT, by = unset & bit ? 1.0f : ex2(-up);
                        unset &= ~bit;
                        (e ? nm[j].y : nm[j].x) -= up;
                        (e ? l[j].y : l[j].x) *= by;
#pragma unroll
                        for (int x = 0; x < 2; ++x) s[x][j][e] -= up, s[x][j][2 + e] -= up;
#pragma unroll
                        for (int i = 0; i < C::MT; ++i) o[j][i][e] *= by, o[j][i][2 + e] *= by;
                    }
                }
            fresh = __any_sync(0xFFFFFFFFu, unset);
        };

#pragma unroll 1
        for (int i = i0 + warp; i < i1; i += C::WARPS) {
            issue();
            cp_wait<C::STAGES - 1>();
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(full + rd, phases >> rd & 1, abort_flag, p.status, WAIT_LIMIT_NS)) && ok;
            if (!ok) break;
            __syncwarp();  // the scales came by copies of lanes 0 .. 3, which a vote orders for no other lane
            const uint32_t src = s_ring + rd * C::TILE;
            float ks[2], vs[2], lv[2], inv[2];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(ks[0]), "=f"(vs[0]), "=f"(ks[1]), "=f"(vs[1])
                         : "r"(s_meta + rd * 16));
            const unsigned gone = absent >> 2 * rd & 3;  // halves whose page is not there
            phases ^= 1u << rd;
            ++taken;
            rd = rd + 1 == C::STAGES ? 0 : rd + 1;
            const int j0 = seen.tile(i) * KV8_KEYS;
            const bool whole = j0 + KV8_KEYS - 1 <= seen.n - p.n_q && !gone &&
                               (!p.window || j0 > seen.n - 1 - p.window || j0 + KV8_KEYS - 1 < p.sinks);

            // ---- both sixteens at once
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // a block of zeros has scale 0: any other does for its codes
                vs[x] = vs[x] < 8.673617e-19f ? 8.673617e-19f : vs[x];  // 2^-60
                lv[x] = lg2(vs[x]), inv[x] = rcp(vs[x]);
            }
            // scores
            float s[2][NT][4];
#pragma unroll
            for (int c = 0; c < C::KC; ++c) {
                unsigned a[2][4][4];
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    const uint32_t at =
                        src + (DP == 64 ? 0 : c >> 1) * C::BOX + 16 * h2 * C::ROW + ((c & 1) ? k_off1 : k_off0);
                    unsigned xw[4], yw[4];
                    if (C::k_steps(c) == 4) {
                        const uint4 x = lds128(at), y = lds128(at + 8 * C::ROW);
                        xw[0] = x.x, xw[1] = x.y, xw[2] = x.z, xw[3] = x.w;
                        yw[0] = y.x, yw[1] = y.y, yw[2] = y.z, yw[3] = y.w;
                    } else {
                        lds64(at, xw[0], xw[1]), lds64(at + 8 * C::ROW, yw[0], yw[1]);
                    }
#pragma unroll
                    for (int k = 0; k < C::k_steps(c); ++k) {
                        cvt4<CODE>(xw[k], a[h2][k][0], a[h2][k][2]);
                        cvt4<CODE>(yw[k], a[h2][k][1], a[h2][k][3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    unsigned f[8];
                    if constexpr (C::QREG) {
#pragma unroll
                        for (int k = 0; k < 2 * C::k_steps(c); ++k) f[k] = qf[j][c][k];
                    } else {
                        load_q(j, c, f);
                    }
#pragma unroll
                    for (int k = 0; k < C::k_steps(c); ++k)
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2) {
                            const unsigned(&w)[4] = a[h2][k];
                            if (c == 0 && k == 0)
                                mma0(s[h2][j], w[0], w[1], w[2], w[3], f[2 * k], f[2 * k + 1]);
                            else
                                mma(s[h2][j], w[0], w[1], w[2], w[3], f[2 * k], f[2 * k + 1]);
                        }
                }
            }
            // exponents relative to the references in place of the sums
            float top = -INFINITY;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float2 k2 = make_float2(ks[x], ks[x]);
                const float2 v2 = make_float2(lv[x], lv[x]);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float2 f = mul2(k2, qs[j]), at = add2(v2, nm[j]);
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const float2 a = fma2(make_float2(s[x][j][k], s[x][j][k + 1]), f, at);
                        s[x][j][k] = a.x, s[x][j][k + 1] = a.y;
                        top = fmaxf(top, fmaxf(a.x, a.y));
                    }
                }
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int q_pos = seen.n - p.n_q + query_of(p, row0 + 8 * j + 2 * t + e).x;
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int key = j0 + 16 * x + pg + 8 * k;
                                const bool sees = key <= q_pos && (!p.window || key > q_pos - p.window || key < p.sinks) &&
                                                  !(gone >> x & 1);
                                if (!sees) s[x][j][2 * k + e] = -INFINITY;
                            }
                    }
            }
            if (__any_sync(0xFFFFFFFFu, top > K8_SLACK) || fresh || !whole) raise(s);
            unsigned pb[2][NT][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float2 a = make_float2(ex2(s[x][j][0]), ex2(s[x][j][1]));
                    const float2 b = make_float2(ex2(s[x][j][2]), ex2(s[x][j][3]));
                    float2 sum = add2(a, b);
                    const float2 i2 = make_float2(inv[x], inv[x]);
                    if (whole) {
                        l[j] = fma2(sum, i2, l[j]);
                    } else {  // a row that sees none of the half takes nothing from its scale either
                        if (sum.x != 0.0f) l[j].x = fmaf(sum.x, i2.x, l[j].x);
                        if (sum.y != 0.0f) l[j].y = fmaf(sum.y, i2.y, l[j].y);
                    }
                    // The weights are operands in f16: off by half a unit of it.  l keeps them whole.
                    pb[x][j][0] = movm(pack(a.x, a.y));
                    pb[x][j][1] = movm(pack(b.x, b.y));
                }

            // weighted sums of v
#pragma unroll
            for (int c = 0; c < C::VC; ++c)
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    constexpr int W = C::VB / 4;
                    const bool two = DP == 96 && c;
                    unsigned v[4][W];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t at = src + (C::ACROSS + (DP == 96 ? 0 : c)) * C::BOX +
                                            (16 * h2 + 8 * (r >> 1)) * C::ROW +
                                            (two ? r & 1 ? v_two1 : v_two0 : r & 1 ? v_off1 : v_off0);
                        if constexpr (W == 4) {
                            const uint4 x = lds128(at);
                            v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                        } else if (two) {
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[r][0]) : "r"(at));
                        } else {
                            lds64(at, v[r][0], v[r][1]);
                        }
                    }
                    if (CODE == QGEMV_CODE_E4M3 && !whole) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int k = 0; k < C::v_words(c); ++k) v[r][k] = without_nan(v[r][k]);
                    }
#pragma unroll
                    for (int k = 0; k < C::v_words(c); ++k)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            // elements 4 k + 2 x and + 1 of keys 2 t, 2 t + 1 and of 2 t + 8, 2 t + 9
                            unsigned a0, a1, a2, a3;
                            cvt4<CODE>(__byte_perm(v[0][k], v[1][k], x ? 0x7362 : 0x5140), a0, a1);
                            cvt4<CODE>(__byte_perm(v[2][k], v[3][k], x ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma(o[j][(C::VB / 2) * c + 2 * k + x], a0, a1, a2, a3, pb[h2][j][0], pb[h2][j][1]);
                        }
                }
            __syncwarp();
        }

        // ---- the warps' sums through the ring
        cp_wait<0>();
        // after a wait that ran out: the copies in flight end, bounded, before the ring is anything else
        for (; taken < sent; ++taken) {
            mbar_drain(full + rd, phases >> rd & 1);
            phases ^= 1u << rd;
            rd = rd + 1 == C::STAGES ? 0 : rd + 1;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = e ? l[j].y : l[j].x;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                const int r = 8 * j + 2 * t + e;
                const float m = unset >> (2 * j + e) & 1 ? K8_NEG : e ? -nm[j].y : -nm[j].x;
                if (g == 0) s_ml[warp * 8 * NT + r] = make_float2(m, sum);
                // elements of its unit of the row, in quads; quad c of a row lies at c ^ t: no bank twice
                float4 *to = reinterpret_cast<float4 *>(k8_smem) + (warp * 8 * NT + r) * (DP / 4);
#pragma unroll
                for (int c = 0; c < C::VC; ++c)
#pragma unroll
                    for (int k = 0; k < C::v_words(c); ++k) {
                        const int i = (C::VB / 2) * c + 2 * k;
                        to[(2 * C::VB * c + C::v_words(c) * v_unit + k) ^ t] =
                            make_float4(o[j][i][e], o[j][i][2 + e], o[j][i + 1][e], o[j][i + 1][2 + e]);
                    }
            }
        __syncthreads();
        const bool whole_unit = i0 == 0 && i1 == seen.tiles;
        const int part = 2 * id + (pos != lo);
        for (int x = tid; x < rows * (DP / 4); x += C::THREADS) {
            const int r = x / (DP / 4), c = x % (DP / 4);
            float top = K8_NEG;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) top = fmaxf(top, s_ml[w * 8 * NT + r].x);
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float total = 0.0f;
#pragma unroll
            for (int w = 0; w < C::WARPS; ++w) {
                const float2 ml = s_ml[w * 8 * NT + r];
                const float by = ex2(ml.x - top);
                const float4 v = reinterpret_cast<const float4 *>(k8_smem)[(w * 8 * NT + r) * (DP / 4) + (c ^ ((r >> 1) & 3))];
                total = fmaf(ml.y, by, total);
                sum.x = fmaf(v.x, by, sum.x), sum.y = fmaf(v.y, by, sum.y);
                sum.z = fmaf(v.z, by, sum.z), sum.w = fmaf(v.w, by, sum.w);
            }
            if (4 * c >= p.d) continue;
            if (whole_unit) {
                const float by = total == 0.0f ? 0.0f : 1.0f / total;
                store_o(p, b, h, row0 + r, c, make_float4(sum.x * by, sum.y * by, sum.z * by, sum.w * by));
                if (c == 0) store_lse(p, b, h, row0 + r, top, total);
            } else {
                const long long at = static_cast<long long>(part) * 8 * NT + r;
                *reinterpret_cast<float4 *>(p.part_o + at * p.d + 4 * c) = sum;
                if (c == 0) p.part_ml[at] = make_float2(top, total);
            }
        }
        // the sequence begins here: its parts, if it ends in a later block's range
        if (tid == 0 && p.balanced && i0 == 0 && (p.parts_by_unit || i1 < seen.tiles)) {
            const int n = (seq_at + seen.tiles - 1) / range - (p.aligned ? 0 : no) + 1;
            p.parts[p.parts_by_unit ? b * per_seq + unit : id] = make_int4(b, unit, part, i1 < seen.tiles ? n : 0);
        }
        pos = seq_at + i1;
        if (pos >= hi) break;
        fence_proxy_async_smem();
        __syncthreads();  // the ring is free again, for copies too
        seq_at += seen.tiles;
        do {
            seen = Seen(p, __ldg(p.lens + ++b));  // one with rows follows, as pos < hi
        } while (seen.tiles == 0);
    }
}

// Joins the parts of the units that the ranges cut: block x those of unit x, or, where
// there are more units than blocks, of the one that block x of the launch before
// left to its successors (which hold it as their first).  Eight threads take 32
// elements of a row from every so many parts; `lanes` such groups, a power of two, share
// a row's 32 elements, so that even 150 parts are a few loads one behind the other.
__global__ void __launch_bounds__(KC_THREADS) kv8_combine_kernel(const __grid_constant__ Kv8AttnParams p, int tile_pad)
{
    __shared__ float4 s_o[KC_THREADS];
    __shared__ float2 s_ml[KC_THREADS];
    const int lanes = p.combine_lanes, group = threadIdx.x >> 3, c = threadIdx.x & 7, mine = group & (lanes - 1);
    const int chunks = (p.d + 31) / 32, item = (blockIdx.y * (KC_THREADS / 8) + group) / lanes;
    const int r = item / chunks, at4 = (item - r * chunks) * 32 + 4 * c;  // row, element
    pdl_launch_dependents();
    pdl_wait();
    const int4 u = p.parts[blockIdx.x];
    if (u.w == 0) return;
    const int per_seq = p.hkv * p.row_tiles;
    const int h = p.row_tiles == 1 ? u.y : u.y / p.row_tiles, row0 = (u.y - h * p.row_tiles) * p.tile_rows;
    const bool there = r < min(p.tile_rows, p.rows - row0) && at4 < p.d;
    float top = K8_NEG, total = 0.0f;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float m, float l, const float4 &v) {
        const float mn = fmaxf(top, m), old = ex2(top - mn), by = ex2(m - mn);
        top = mn;
        total = fmaf(l, by, total * old);
        sum.x = fmaf(v.x, by, sum.x * old), sum.y = fmaf(v.y, by, sum.y * old);
        sum.z = fmaf(v.z, by, sum.z * old), sum.w = fmaf(v.w, by, sum.w * old);
    };
    if (there) {
        constexpr int U = 4;
        for (int i0 = mine; i0 < u.w; i0 += U * lanes) {
            float2 ml[U];
            float4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int i = i0 + k * lanes;
                if (i < u.w) {
                    const long long a = static_cast<long long>(i == 0 ? u.z : 2 * ((u.z >> 1) + i * per_seq)) * tile_pad + r;
                    ml[k] = p.part_ml[a];
                    v[k] = *reinterpret_cast<const float4 *>(p.part_o + a * p.d + at4);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * lanes < u.w) add(ml[k].x, ml[k].y, v[k]);
        }
    }
    if (lanes > 1) {
        s_o[threadIdx.x] = sum;
        s_ml[threadIdx.x] = make_float2(top, total);
        for (int o = lanes >> 1; o; o >>= 1) {
            __syncthreads();
            if (mine < o) {
                const float2 ml = s_ml[threadIdx.x + 8 * o];
                add(ml.x, ml.y, s_o[threadIdx.x + 8 * o]);
                s_o[threadIdx.x] = sum;
                s_ml[threadIdx.x] = make_float2(top, total);
            }
        }
    }
    if (!there || mine) return;
    const float by = total == 0.0f ? 0.0f : 1.0f / total;
    store_o(p, u.x, h, row0 + r, at4 / 4, make_float4(sum.x * by, sum.y * by, sum.z * by, sum.w * by));
    if (at4 == 0) store_lse(p, u.x, h, row0 + r, top, total);
}

// A cache's codes as [page][head][row][element], boxes of up to 32 rows of 128 elements.
bool encode(CUtensorMap *map, const Kv8AttnParams &p, const void *base)
{
    const auto fn = map_encoder();
    if (!fn) return false;
    const cuuint32_t rows = 1u << p.c.page_shift;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.d), rows, static_cast<cuuint64_t>(p.hkv),
                                static_cast<cuuint64_t>(p.c.n_pages)};
    // a stride that nothing is reached by may be any
    const auto stride = [](long long s, long long n) { return static_cast<cuuint64_t>(n > 1 ? s : 16); };
    const cuuint64_t strides[3] = {stride(p.c.row_stride, rows), stride(p.c.head_stride, p.hkv), stride(p.c.page_stride, p.c.n_pages)};
    const cuuint32_t box[4] = {p.d <= 64 ? 64u : 128u, rows < KV8_KEYS ? rows : KV8_KEYS, 1, 1}, ones[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, p.d <= 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CODE, int DP, int NT, bool WIDE>
cudaError_t launch_wide(const Kv8AttnParams &p, cudaStream_t st)
{
    using C = K8Cfg<DP, NT, WIDE>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(kv8_attn_kernel<CODE, DP, NT, WIDE>), C::SMEM, done);
    if (e != cudaSuccess) return e;
    CUtensorMap k_map, v_map;
    if (!encode(&k_map, p, p.c.k) || !encode(&v_map, p, p.c.v)) return cudaErrorInvalidValue;
    // (units of a sequence, ranges) or, with a block for each unit, (units, sequences in two dimensions)
    const unsigned units = static_cast<unsigned>(p.hkv * p.row_tiles), n = static_cast<unsigned>(p.balanced ? p.ranges : p.n_seqs);
    const unsigned ny = n < 32768 ? n : 32768;
    const dim3 grid(units, ny, (n + ny - 1) / ny);
    e = launch_pdl(kv8_attn_kernel<CODE, DP, NT, WIDE>, grid, C::THREADS, C::SMEM, st, p, k_map, v_map);
    if (e != cudaSuccess || !p.balanced) return e;
    const int items = KC_THREADS / 8 / p.combine_lanes, all = p.tile_rows * ((p.d + 31) / 32);  // of a block, of a unit
    const int blocks = p.parts_by_unit ? p.n_seqs * p.hkv * p.row_tiles : p.grid;
    return launch_pdl(kv8_combine_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((all + items - 1) / items)),
                      KC_THREADS, 0, st, p, 8 * NT);
}

template <int CODE, int DP, int NT>
cudaError_t launch_nt(const Kv8AttnParams &p, cudaStream_t st)
{
    if constexpr (kv8_blocks(DP, NT) == 2) {
        if (p.wide) return launch_wide<CODE, DP, NT, true>(p, st);
    }
    return launch_wide<CODE, DP, NT, false>(p, st);
}

template <int CODE, int DP>
cudaError_t launch_dp(const Kv8AttnParams &p, cudaStream_t st)
{
    const int nt = (p.tile_rows + 7) / 8;
    if constexpr (DP < 256) {
        if (nt == 4) return launch_nt<CODE, DP, 4>(p, st);
        if (nt == 3) return launch_nt<CODE, DP, 3>(p, st);
    }
    return nt == 2 ? launch_nt<CODE, DP, 2>(p, st) : launch_nt<CODE, DP, 1>(p, st);
}

template <int CODE>
cudaError_t launch_code(const Kv8AttnParams &p, cudaStream_t st)
{
    if (p.d > 128) return launch_dp<CODE, 256>(p, st);
    return p.d <= 64 ? launch_dp<CODE, 64>(p, st) : p.d <= 96 ? launch_dp<CODE, 96>(p, st) : launch_dp<CODE, 128>(p, st);
}

}  // namespace

}  // namespace qg
