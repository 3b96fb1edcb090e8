// fork_pages.cu -- sequences of a paged cache reordered by parent: table rows
// gathered, and the partly filled page of each copied to a page of its own, in all
// layers' caches at once.
//
// What bounds it: memory where many rows are copied (read and written once), else
// the chain of dependent loads parent, length, page, rows.  A block takes one
// sequence and walks the arrays (k and v of each cache) in steps of the grid, so
// that this chain is paid once for several copies.  256 sequences, 36 caches: 46 us, 6.4 TB/s,
// with blocks for 32 a multiprocessor (for 8 a one 55, 16 51, 128 46); eight of 28 caches 2.5 us.
#include "kv8_ops.h"
#include "qgemv_internal.cuh"

namespace qg {
namespace {

constexpr int FK_THREADS = 128, FK_UNROLL = 4;

__global__ void __launch_bounds__(FK_THREADS) fork_kernel(const __grid_constant__ ForkParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, i = blockIdx.x;
    const bool tell = tid == 0 && blockIdx.y == 0;
    const int parent = __ldg(p.f.parents + i);
    if (parent < 0 || parent >= p.f.n_in) {
        if (parent != -1 && tell) atomicCAS(p.status, 0u, ST_BAD_ID);
        return;
    }
    const int page_size = 1 << p.page_shift;
    const long long most = static_cast<long long>(p.f.n_columns) << p.page_shift;
    const int len = __ldg(p.f.lens + parent);
    int fresh = __ldg(p.f.fresh + i);
    const int n = len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
    if (n != len && tell) atomicCAS(p.status, 0u, ST_BAD_ID);
    if (fresh < -1 || fresh >= p.n_pages) {
        if (tell) atomicCAS(p.status, 0u, ST_BAD_ID);
        fresh = -1;
    }
    const int full = n >> p.page_shift, rows = n & (page_size - 1);
    const int32_t *from = p.f.pages + parent * p.f.pages_stride;
    if (blockIdx.y == 0 && p.first) {
        int32_t *to = p.f.pages_out + i * p.f.out_stride;
        for (int j = tid; j < full; j += FK_THREADS) to[j] = __ldg(from + j);
        if (tid == 0) {
            if (full < p.f.n_columns) {
                if (fresh >= 0)
                    to[full] = fresh;
                else if (rows)
                    to[full] = __ldg(from + full);
            }
            p.f.lens_out[i] = n;
        }
    }
    if (rows == 0 || fresh < 0) return;
    const int page = __ldg(from + full);
    if (page < 0 || page >= p.n_pages) {
        if (tell) atomicCAS(p.status, 0u, ST_BAD_ID);
        return;
    }
    if (page == fresh) return;

    const int chunks = p.head_bytes >> 4, per_row = p.heads * chunks, total = rows * per_row;
    for (int a = blockIdx.y; a < p.n_arrays; a += gridDim.y) {
        const int c = a >> 1;
        const uint8_t *src = static_cast<const uint8_t *>(p.base[a]) + page * p.page_stride[c];
        uint8_t *dst = static_cast<uint8_t *>(p.base[a]) + fresh * p.page_stride[c];
        // whole rows that lie one behind the other are one run of 16-byte chunks
        const bool run = p.head_stride[c] == p.head_bytes && p.row_stride[c] == static_cast<long long>(p.heads) * p.head_bytes;
        auto at = [&](int x) -> long long {
            if (run) return 16ll * x;
            const int row = x / per_row, y = x - row * per_row, h = y / chunks;
            return row * p.row_stride[c] + h * p.head_stride[c] + 16ll * (y - h * chunks);
        };
        for (int x0 = tid; x0 < total; x0 += FK_THREADS * FK_UNROLL) {
            uint4 v[FK_UNROLL];
#pragma unroll
            for (int u = 0; u < FK_UNROLL; ++u)
                if (x0 + u * FK_THREADS < total) v[u] = *reinterpret_cast<const uint4 *>(src + at(x0 + u * FK_THREADS));
#pragma unroll
            for (int u = 0; u < FK_UNROLL; ++u)
                if (x0 + u * FK_THREADS < total) *reinterpret_cast<uint4 *>(dst + at(x0 + u * FK_THREADS)) = v[u];
        }
        if (p.block_shift >= 0) {
            const int blocks = (rows + (1 << p.block_shift) - 1) >> p.block_shift;
            const float *ss = p.scale[a] + page * p.scale_page[c];
            float *sd = p.scale[a] + fresh * p.scale_page[c];
            for (int x = tid; x < blocks * p.heads; x += FK_THREADS) {
                const long long o = x / p.heads * p.scale_block[c] + x % p.heads * p.scale_head[c];
                sd[o] = ss[o];
            }
        }
    }
}

}  // namespace

cudaError_t launch_fork(const ForkParams &p, int sms, cudaStream_t st)
{
    // Blocks that share a sequence until there are 32 for each multiprocessor: 256 sequences of 72
    // arrays take 46 us; 16 for each 51, 8 for each 55, as many as there are arrays 46.
    const long long want = (32ll * sms + p.f.n_out - 1) / p.f.n_out;
    const unsigned ny = static_cast<unsigned>(want < p.n_arrays ? want : p.n_arrays);
    return launch_pdl(fork_kernel, dim3(static_cast<unsigned>(p.f.n_out), ny), FK_THREADS, 0, st, p);
}

}  // namespace qg
