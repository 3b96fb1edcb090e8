// attn_tc.cu -- the prefix part of the shared-prefix attention on the
// fifth-generation tensor cores, for batches with many rows per cache head
// (see attn_prefix.cu for the parts and how they are combined).
//
// With R rows per cache head the prefix takes 4 R d operations per key
// against 4 d bytes read: from a few hundred rows on the matrix products
// bound it, at a rate that mma.sync reaches a quarter of.
//
// A block (one per multiprocessor) takes a range of keys of one cache head
// and two "streams" of 128 rows, each with its own scores S and weighted sum
// O in tensor memory (128 columns each):
//   rows mode: the streams are two row tiles over the same keys;
//   keys mode (at most 128 rows): one row tile, and the streams take
//   alternate key tiles and leave two parts.
// Per stream and tile of 128 keys:
//   S = Q K^T (tcgen05.mma, both operands from shared memory), read back row
//   by row: thread i of the stream's four warps owns row i, so maxima and
//   sums need no shuffles; P = 2^(S scale - m), rounded to the cache's type,
//   goes over S's own columns (two elements a column); O += P V with P from
//   tensor memory and V from shared memory.
// One warp issues the products, alternating between the streams, so that one
// stream's products run while the other's weights are computed; a stream's
// weights go over in two halves, and the sums of the first start while the
// second forms.
//
// Measured: 1024 rows x 8 heads x 65536 keys of 128 elements 186 us, 1.48
// PFLOP/s (0.76 of the measured bf16 burst rate, 0.87 of the sustained one),
// products 64 % of the time; 320 rows x 2 heads x 32749 keys 20 us.  A pair of tiles of 128 keys takes 2850
// cycles, the products' own 2048: the rest is handing over between the row
// threads and the products, twice a tile and stream.  A block of few tiles
// spends 3 us before its first scores (tensor memory, page table, first keys)
// and 2 on its part.
// Tried and slower at the first size: scores of 64 keys, double-buffered (274
// against 239 us then: with N = 64 a product takes 49 cycles instead of 32,
// bound by its operands' shared-memory reads, and the waits double); a warp
// per stream for the products (250); one lane polling a barrier for its warp.
//
// The reference m of a row is its running maximum, but follows it only when
// that rises by more than 2^8: O is rescaled (in tensor memory, by the row's
// own thread) in few tiles instead of all, and the weights stay below 2^8 (f16:
// 2^14), exact in scale.  They enter the product with v rounded to the cache's
// type; l sums the unrounded weights in fp32.
//
// K and V tiles share a ring of buffers in the 128-byte-swizzled layout the
// products read: rows of 64 elements, halves of the head side by side.  K is
// the K-major operand of S, V the same bytes as the MN-major operand of O.
// One warp fills the ring with TMA copies of a page's rows (or of 128 of
// them), through tensor maps of the cache; a page that is not there is a
// coordinate past the tensor, which reads as zeros.  The range is whole tiles:
// what a prefix has beyond them goes to attn_prefix.cu's blocks.  (Filled by
// four warps with 16-byte cp.async copies the ring cost a third of the
// instructions of the kernel.)
//
// Registers: the launch has 384 threads of 168; the row threads take 208,
// the other warps 88: 256 * 208 + 128 * 88 = 384 * 168.
//
// Every wait is bounded: a block that gives up records QGEMV_ERR_TIMEOUT and
// frees its tensor memory.  Every block first waits (bounded) for its copies and
// products in flight, in their warps, which have nothing else to do by then.
#include <type_traits>

#include "decode_ops.h"
#include "qgemv_internal.cuh"
#include "tc_ptx.cuh"
#include "tma.cuh"

namespace qg {
namespace {

constexpr int AC_THREADS = 384;   // warps 0-3, 4-7: rows of streams 0, 1; 8: products; 9: keys and values
constexpr int AC_KEYS = 128;      // keys of a tile
constexpr int AC_ROWS = 128;      // rows of a stream
constexpr int AC_MASKS = 8;       // tiles whose presence masks are kept, per stream: the ring holds fewer
constexpr float AC_RISE = 8.0f;   // rise of the maximum (base 2) that moves the reference
constexpr float AC_NEG = -1e30f;
// f16 weights lie 2^6 times as high, below 2^14 with the rise (see AT_LIFT in
// attn_prefix.cu): what is 2^-31 of the largest or more counts.
template <typename T>
constexpr float AC_LIFT = std::is_same<T, __half>::value ? 6.0f : 0.0f;

template <int DP>
struct TcCfg {
    static constexpr int HALF = AC_KEYS * 128;            // 64 elements of 128 rows
    static constexpr int TILE = HALF * DP / 64;           // a K or V tile; also 128 rows of Q
    static constexpr int NBUF = DP == 64 ? 8 : 5;
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_BAR = OFF_RING + NBUF * TILE;
    static constexpr int NBAR = 2 * NBUF + 10;
    static constexpr int OFF_MASK = OFF_BAR + 8 * NBAR;   // [stream][AC_MASKS][4] words
    static constexpr int SMEM = (OFF_MASK + 2 * AC_MASKS * 16 + 15) / 16 * 16 + 1024;  // aligned up to 1024 at run time
};
static_assert(TcCfg<128>::SMEM <= 227 * 1024, "shared memory of the prefix kernel");

// Tensor-memory columns of a stream's scores (weights over their first half) and sums.
__device__ __forceinline__ constexpr uint32_t col_s(int s) { return 128u * s; }
__device__ __forceinline__ constexpr uint32_t col_o(int s) { return 256u + 128u * s; }

// Four products D = A x B [+ D] along K: A and B in shared memory, 32 bytes a
// step apart (64 elements, one swizzled row), or A in tensor memory, 8
// columns a step apart, and B 16 rows of 128 bytes.  The whole warp runs the
// issuing loop and one elected lane issues all four: the operands are then
// known to be uniform, and the steps cost an addition each.  (Issued one by
// one, from a branch of one lane, each product took about 130 cycles.)
__device__ __forceinline__ void tc_mma4_ss(uint32_t d_t, uint64_t adesc, uint64_t bdesc, uint32_t idesc, int accumulate)
{
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_t),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma4_ts(uint32_t d_t, uint32_t a_t, uint64_t bdesc, uint32_t idesc, int accumulate)
{
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d_t),
        "r"(a_t), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of a 128-byte-swizzled operand: groups of 8 rows 1024 bytes
// apart (stride byte offset); `lead` separates the 64-element halves of an
// MN-major operand (unused by a K-major one).
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr, uint32_t lead)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tc_ld32(uint32_t taddr, float *d)
{
    unsigned r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) d[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const unsigned *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ac_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a * b + c and a + b on pairs (two IEEE operations each).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tadd.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

template <typename T>
__device__ __forceinline__ unsigned pack2(float lo, float hi);
template <>
__device__ __forceinline__ unsigned pack2<__half>(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}
template <>
__device__ __forceinline__ unsigned pack2<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&h);
}

__device__ __forceinline__ void ac_cp16(uint32_t dst, const void *src, bool take)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

// Byte offset of 16-byte chunk c of row r: halves of 8 chunks, 128-byte rows, swizzled.
__device__ __forceinline__ uint32_t ac_off(int r, int c)
{
    return static_cast<uint32_t>((c >> 3) * (AC_KEYS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Bounded wait of a converged warp.
__device__ __forceinline__ bool ac_wait(uint64_t *bar, unsigned parity, volatile int *abort_flag, unsigned *status)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort_flag, status, WAIT_LIMIT_NS)) != 0;
}

// A block's work, the same for all roles.
struct TcWork {
    int head, k0;
    int tiles;       // key tiles of the range
    int n[2];        // tiles of each stream
    int row0[2];     // first row
    int nrows;       // rows from row0[0] on that exist (both streams together in rows mode)
    bool by_keys;
    // key tile of a stream's i-th step
    __device__ __forceinline__ int tile(int s, int i) const { return by_keys ? 2 * i + s : i; }
};

template <typename T, int DP>
__global__ void __launch_bounds__(AC_THREADS, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap)
{
    using C = TcCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ int s_absent;
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + C::NBUF;
    uint64_t *s_full = empty + C::NBUF, *p_full = s_full + 2, *pv_done = p_full + 4,  // [stream]; [stream][half]; [stream]
             *q_full = pv_done + 2, *drained = q_full + 1;
    unsigned *masks = reinterpret_cast<unsigned *>(smem + C::OFF_MASK);
    volatile int *abort_flag = &s_abort;

    if (warp == 9 && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &vmap : &kmap) : "memory");
    if (tid == 0) {
        s_abort = 0;
        s_absent = 0;
        for (int i = 0; i < C::NBUF; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_full, 2 * AC_ROWS);
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    TcWork w;
    {
        int id = blockIdx.x;
        const int rt = id % p.t_tiles;
        id /= p.t_tiles;
        w.head = id % p.hkv;
        const int split = id / p.hkv;
        w.by_keys = p.t_mode == 2;
        w.k0 = split * p.t_keys;
        w.tiles = (min(p.t_len, w.k0 + p.t_keys) - w.k0) / AC_KEYS;
        w.row0[0] = rt * (w.by_keys ? AC_ROWS : 2 * AC_ROWS);
        w.row0[1] = w.row0[0] + (w.by_keys ? 0 : AC_ROWS);
        w.nrows = min(p.rows - w.row0[0], w.by_keys ? AC_ROWS : 2 * AC_ROWS);
        w.n[0] = w.by_keys ? (w.tiles + 1) / 2 : w.tiles;
        w.n[1] = w.by_keys ? w.tiles / 2 : w.nrows > AC_ROWS ? w.tiles : 0;
    }
    if (p.t_wait) pdl_wait();
    pdl_launch_dependents();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 9) {
            // ------------------------------------------------ keys and values
            // A tile is boxes of `box` rows (a page, or the tile), 64 elements wide;
            // lane i copies box i % boxes of half i / boxes.
            const int box = min(1 << p.page_shift, AC_KEYS), boxes = AC_KEYS / box;
            const bool copies = lane < boxes * (DP / 64);
            const int half = lane / boxes, mine = lane - half * boxes;
            const uint32_t dst = half * C::HALF + mine * box * 128;
            // this lane's page of key tile t, n_pages (beyond the tensor: zeros) when it is not there
            auto find = [&](int t) -> int {
                const int page = __ldg(p.prefix_pages + ((w.k0 + t * AC_KEYS + (mine & (boxes - 1)) * box) >> p.page_shift));
                return page >= 0 && page < p.n_pages ? page : static_cast<int>(p.n_pages);
            };
            int n = 0;  // buffers issued
            bool ok = true;
            auto fill = [&](const CUtensorMap *map, int t, int page) {
                const int b = n % C::NBUF;
                if (n >= C::NBUF) ok = ac_wait(&empty[b], static_cast<unsigned>((n / C::NBUF - 1) & 1), abort_flag, p.status);
                if (!ok) return;
                if (lane == 0) mbar_arrive_expect_tx(&full[b], C::TILE);
                __syncwarp();
                if (copies)
                    tma_load4(smem_addr(smem + C::OFF_RING) + b * C::TILE + dst, map, 64 * half,
                              (w.k0 + t * AC_KEYS) & ((1 << p.page_shift) - 1), w.head, page, &full[b]);
                ++n;
            };
            // which keys of a tile are there, for the row threads
            auto present = [&](int s, int i, int page) {
                const unsigned there = __ballot_sync(0xFFFFFFFFu, page < p.n_pages);
                if (there != 0xFFFFFFFFu && lane == 0) {
                    atomicCAS(p.status, 0u, ST_BAD_ID);
                    *static_cast<volatile int *>(&s_absent) = 1;
                }
                if (lane < 4) {
                    unsigned bits = 0;
                    for (int e = 0; e < 32; ++e) bits |= (there >> ((32 * lane + e) / box) & 1u) << e;
                    masks[(s * AC_MASKS + (i & (AC_MASKS - 1))) * 4 + lane] = bits;
                }
                __syncwarp();
            };
            const bool two = w.by_keys;  // the streams have keys of their own
            int cur[2], nxt[2];          // pages of the streams' tiles i and i + 1
            cur[0] = find(w.tile(0, 0));
            cur[1] = two && w.n[1] > 0 ? find(w.tile(1, 0)) : 0;
            present(0, 0, cur[0]);
            if (!two) present(1, 0, cur[0]);
            if (two && w.n[1] > 0) present(1, 0, cur[1]);
            fill(&kmap, w.tile(0, 0), cur[0]);
            if (two && w.n[1] > 0) fill(&kmap, w.tile(1, 0), cur[1]);
            nxt[0] = w.n[0] > 1 ? find(w.tile(0, 1)) : 0;
            nxt[1] = two && w.n[1] > 1 ? find(w.tile(1, 1)) : 0;
            for (int i = 0; i < w.n[0] && ok; ++i) {
    #pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s == 1 && !two) break;
                    const int after = i + 2 < w.n[s] ? find(w.tile(s, i + 2)) : 0;  // on its way meanwhile
                    if (i < w.n[s]) fill(&vmap, w.tile(s, i), cur[s]);
                    if (i + 1 < w.n[s] && ok) {
                        present(s, i + 1, nxt[s]);
                        if (!two) present(1, i + 1, nxt[s]);
                        fill(&kmap, w.tile(s, i + 1), nxt[s]);
                    }
                    cur[s] = nxt[s];
                    nxt[s] = after;
                }
            }
            // The copies in flight end before the block does (bounded), also where
            // another warp gives up after this one is done.  A buffer's earlier fills
            // were complete before it was filled again.
            if (lane == 0)
                for (int b = n > C::NBUF ? n - C::NBUF : 0; b < n; ++b)
                    mbar_drain(&full[b % C::NBUF], static_cast<unsigned>((b / C::NBUF) & 1));
            __syncwarp();
        } else if (warp == 8) {
            // ------------------------------------------------ products
            {
                constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
                constexpr uint32_t IDESC = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 4) << 24);
                constexpr uint32_t IDESC_S = IDESC | ((AC_KEYS / 8u) << 17);
                constexpr uint32_t IDESC_O = IDESC | (1u << 16) | ((DP / 8u) << 17);  // B is MN-major
                const uint32_t q_s = smem_addr(smem), ring = smem_addr(smem + C::OFF_RING);
                int pos = 0;
                bool ok = true;
                auto acquire = [&]() -> int {  // the next buffer, once it is full
                    const int b = pos % C::NBUF;
                    ok = ok && ac_wait(&full[b], static_cast<unsigned>((pos / C::NBUF) & 1), abort_flag, p.status);
                    tc_fence_after();
                    ++pos;
                    return __shfl_sync(0xFFFFFFFFu, b, 0);
                };
                auto scores = [&](int s, int b) {
                    const uint32_t qa = q_s + (w.by_keys ? 0 : s * C::TILE), ka = ring + b * C::TILE;
    #pragma unroll
                    for (int hf = 0; hf < DP / 64; ++hf)
                        tc_mma4_ss(tm + col_s(s), tc_desc(qa + hf * C::HALF, 16), tc_desc(ka + hf * C::HALF, 16), IDESC_S, hf);
                    tc_commit_elect(&s_full[s]);
                };
                auto sums = [&](int s, int i, int b) {
                    const uint32_t va = ring + b * C::TILE;
    #pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        ok = ok && ac_wait(&p_full[2 * s + hf], static_cast<unsigned>(i & 1), abort_flag, p.status);
                        if (!ok) return;
                        tc_fence_after();
                        tc_mma4_ts(tm + col_o(s), tm + col_s(s) + 32 * hf, tc_desc(va + hf * AC_KEYS / 2 * 128, C::HALF), IDESC_O,
                                   i > 0 || hf > 0);
                    }
                    if (i == w.n[s] - 1) tc_commit_elect(&pv_done[s]);
                };
                int kbuf = 0, vbuf = 0;                      // the current buffers
                // One stream's products of tile i: the sums with its weights, then the
                // scores of the next tile over the columns that those weights leave.
                // i = -1: the first scores.
                auto turn = [&](int s, int i) {
                    const bool own = w.by_keys || s == 0;                  // takes its buffers itself
                    const bool last = w.by_keys || s == 1 || w.n[1] == 0;  // and is their last reader
                    if (i >= 0 && i < w.n[s]) {
                        if (own) vbuf = acquire();
                        if (ok) sums(s, i, vbuf);
                        if (!ok) return;
                        if (last) tc_commit_elect(&empty[vbuf]);
                    }
                    if (i + 1 < w.n[s]) {
                        if (own) kbuf = acquire();
                        if (!ok) return;
                        scores(s, kbuf);
                        if (last) tc_commit_elect(&empty[kbuf]);
                    }
                };
                ok = ac_wait(q_full, 0, abort_flag, p.status);
                for (int i = -1; i < w.n[0] && ok; ++i) {
                    turn(0, i);
                    if (ok) turn(1, i);
                }
                // The products in flight end before the block does, by a commit of its
                // own (bounded): after an abort, half of a tile's sums, or sums that no
                // scores follow yet, have no other.
                tc_commit_elect(drained);
                if (lane == 0) mbar_drain(drained, 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------ rows
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int s = warp >> 2, wq = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t to = tm + col_o(s) + lanes;
        const int r = (w.by_keys ? 0 : s * AC_ROWS) + 32 * wq + lane;  // row of the block
        // Q: the stream's warps copy its tile, 32 rows each; rows past the batch are zeros
        if (!(s && w.by_keys)) {
            constexpr int CH = DP / 8, RPI = 32 / CH;  // chunks of a row, rows per instruction
            long long off = -1;
            if (r < w.nrows) {
                const int row = w.row0[0] + r, tok = row / p.group, g = row - tok * p.group;
                off = tok * p.q_token_stride + (static_cast<long long>(w.head) * p.group + g) * p.q_head_stride;
            }
            const int c = lane % CH;
#pragma unroll 4
            for (int i = 0; i < 32 / RPI; ++i) {
                const int rr = i * RPI + lane / CH;
                const long long o = __shfl_sync(0xFFFFFFFFu, off, rr);
                const bool take = o >= 0 && c * 8 < p.d;
                ac_cp16(smem_addr(smem) + s * C::TILE + ac_off(32 * wq + rr, c),
                        static_cast<const T *>(p.q) + (take ? o + c * 8 : 0), take);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
        }
        mbar_arrive(q_full);
        float m = AC_NEG;
        float2 l2 = make_float2(0.0f, 0.0f);
        bool ok = true;
        for (int i = 0; i < w.n[s] && ok; ++i) {
            ok = ac_wait(&s_full[s], static_cast<unsigned>(i & 1), abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t ts = tm + col_s(s) + lanes;
            float x[AC_KEYS];
#pragma unroll
            for (int c = 0; c < AC_KEYS; c += 32) tc_ld32(ts + c, x + c);
            tc_wait_ld();
            if (*static_cast<volatile int *>(&s_absent)) {
                const unsigned *mk = masks + (s * AC_MASKS + (i & (AC_MASKS - 1))) * 4;
#pragma unroll
                for (int c = 0; c < AC_KEYS; c += 32) {
                    const unsigned bits = mk[c >> 5];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(bits >> e & 1)) x[c + e] = -INFINITY;
                }
            }
            float mm[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mm[e] = fmaxf(x[2 * e], x[2 * e + 1]);
#pragma unroll
            for (int c = 8; c < AC_KEYS; c += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) mm[e] = fmaxf(mm[e], fmaxf(x[c + 2 * e], x[c + 2 * e + 1]));
            // rounded up, and the rise's bound down, so that the weights stay below 2^(rise + lift) for scores of any size
            const float top = fmaxf(fmaxf(mm[0], mm[1]), fmaxf(mm[2], mm[3]));
            const float mx = __fadd_ru(fmaxf(__fmul_ru(top, p.scale_log2), AC_NEG), -AC_LIFT<T>);
            if (i == 0) {
                m = mx;
            } else {
                const bool rise = mx > __fadd_rd(m, AC_RISE);
                if (__any_sync(0xFFFFFFFFu, rise)) {
                    // O holds the sums of the tiles before; they are complete: the
                    // scores of this tile were issued after them
                    const float f = rise ? ac_ex2(m - mx) : 1.0f;
                    if (rise) m = mx;
                    l2.x *= f;
                    l2.y *= f;
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        float o[32];
                        tc_ld32(to + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tc_st32(to + c, reinterpret_cast<const unsigned *>(o));
                    }
                    tc_wait_st();
                }
            }
            const float2 sc = make_float2(p.scale_log2, p.scale_log2), nm = make_float2(-m, -m);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // the first half's sums start while the second half's weights form
                unsigned pk[32];
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float2 a = fma2(make_float2(x[64 * hf + c], x[64 * hf + c + 1]), sc, nm);
                    const float2 e = make_float2(ac_ex2(a.x), ac_ex2(a.y));
                    l2 = add2(l2, e);
                    pk[c / 2] = pack2<T>(e.x, e.y);
                }
                tc_st32(ts + 32 * hf, pk);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * s + hf]);
            }
        }
        // the part: a row a lane, 16 bytes each
        const bool have = w.n[s] > 0;
        if (have && ok) {
            ok = ac_wait(&pv_done[s], 0, abort_flag, p.status);
            tc_fence_after();
        }
        const int split = blockIdx.x / (p.t_tiles * p.hkv);
        const int slot = w.by_keys ? 2 * split + s : split;
        const bool mine = r < w.nrows;
        const long long slab = static_cast<long long>(slot) * p.hkv + w.head;
        const int row = w.row0[0] + r;
        if (ok && (have || w.by_keys)) {  // a stream without keys leaves an empty part
            if (mine) p.part_ml[slab * p.rows + row] = make_float2(have ? m : AC_NEG, l2.x + l2.y);
#pragma unroll
            for (int c = 0; c < DP; c += 32) {
                float o[32];
                if (have) {
                    tc_ld32(to + c, o);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    if (mine && c + e < p.d)
                        p.part_o[(slab * (p.d >> 2) + ((c + e) >> 2)) * p.rows + row] =
                            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
    // The part launch may still be running: this one, which the combining launch
    // waits for, ends after it (see launch_pdl).
    pdl_wait();
}

// The cache as [page][head][row][element], boxes of up to 128 rows of 64 elements.
bool encode(CUtensorMap *map, const AttnParams &p, const void *base, qgemv_dtype type)
{
    const auto fn = map_encoder();
    if (!fn) return false;
    const cuuint32_t rows = 1u << p.page_shift;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.d), rows, static_cast<cuuint64_t>(p.hkv),
                                static_cast<cuuint64_t>(p.n_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(2 * p.row_stride), static_cast<cuuint64_t>(2 * p.head_stride),
                                   static_cast<cuuint64_t>(2 * p.page_stride)};
    const cuuint32_t box[4] = {64, rows < AC_KEYS ? rows : AC_KEYS, 1, 1}, ones[4] = {1, 1, 1, 1};
    return fn(map, type == QGEMV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
cudaError_t launch_t(const AttnParams &p, qgemv_dtype type, cudaStream_t st)
{
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(attn_tc_kernel<T, DP>), TcCfg<DP>::SMEM, done);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap, vmap;
    if (!encode(&kmap, p, p.k, type) || !encode(&vmap, p, p.v, type)) return cudaErrorInvalidValue;
    return launch_pdl(attn_tc_kernel<T, DP>, dim3(static_cast<unsigned>(p.t_blocks)), AC_THREADS, TcCfg<DP>::SMEM, st, p,
                      kmap, vmap);
}

// A stride that a tensor map takes: positive, a multiple of 16 bytes, below 2^40.
inline bool map_stride(long long elements) { return elements > 0 && elements % 8 == 0 && 2 * elements < (1ll << 40); }

}  // namespace

bool attn_tc_takes(const qgemv_kv_cache &c)
{
    return c.head_dim <= 128 && c.page_size >= 8 && map_stride(c.row_stride) && map_stride(c.head_stride) &&
           map_stride(c.page_stride);
}

cudaError_t launch_attn_tc(const AttnParams &p, qgemv_dtype type, cudaStream_t st)
{
    if (type == QGEMV_F16) return p.d <= 64 ? launch_t<__half, 64>(p, type, st) : launch_t<__half, 128>(p, type, st);
    return p.d <= 64 ? launch_t<__nv_bfloat16, 64>(p, type, st) : launch_t<__nv_bfloat16, 128>(p, type, st);
}

}  // namespace qg
