// decode_ops.h -- internal interface between the C ABI of the decode step's
// operators between its GEMVs (decode_api.cu) and their kernels: rotary
// positions with the cache write (rope_kv.cu), attention over a cache whose
// prefix the batch shares (attn_prefix.cu) and the rules on logits
// (logits_rules.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qgemv.h"

namespace qg {

// Multiprocessors and the status word of the current device (qgemv_api.cu).
qgemv_status device_props(int *sms, unsigned **status);

// Allow a kernel `bytes` of dynamic shared memory, once per device (`done`:
// one bit per device, a static of the caller's; a second setting is harmless).
inline cudaError_t allow_smem(const void *kernel, size_t bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Launch with programmatic dependent launch: the kernel may start while the
// preceding one drains and touches memory only after its griddepcontrol.wait.
// The one exception, the prefix kernel behind the attention's part launch
// (attn_tc.cu), rests on two conditions: that launch lets it in only after its
// own wait, so what came before is complete, and the prefix kernel waits before it
// ends, so that its successor's wait covers both.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st,
                              Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// ---------------------------------------------------------------- rotary

struct RopeParams {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const int32_t *pos, *slots;
    void *q_out;
    long long q_out_stride;
    void *ck, *cv;
    long long page_stride, row_stride, head_stride;
    long long n_slots;
    int page_shift;
    int hq, hkv, d, rot;
    int heads_per_block;     // heads that the block's threads cover at once
    float mscale;
    unsigned *status;
    unsigned long long turns[128];
};
// vec: every address and stride suits 16-byte accesses.
cudaError_t launch_rope(RopeParams &p, qgemv_dtype in, qgemv_dtype q_out, qgemv_dtype cache, bool half_layout, bool vec,
                        long long n_tokens, int sms, cudaStream_t st);

// ---------------------------------------------------------------- logits

struct LogitsParams {
    const void *x;
    void *out;
    long long x_stride, out_stride;
    long long vocab;
    const long long *hist;
    long long hist_stride;
    const int32_t *hist_len;
    int max_hist;
    const float *rep, *freq, *pres;
    const long long *bias_ids;
    const float *bias;
    long long bias_stride;
    const int32_t *bias_len;
    int max_bias;
    const uint32_t *mask;
    long long mask_stride;
    long long *idx;
    float *val;
    unsigned long long *keys;  // [rows] running maxima, zero between launches
    unsigned *cnt;             // [rows] arrivals, zero between launches
    unsigned *status;
    int slice;                 // tokens per block: a multiple of 32
};
constexpr int LOGITS_ROWS = 1024;      // rows per launch: keys and arrivals fit the counter area
constexpr int LOGITS_KEYS_BYTES = 8 * LOGITS_ROWS;
cudaError_t launch_logits(LogitsParams &p, qgemv_dtype type, int rows, int sms, cudaStream_t st);

// ------------------------------------------------------------- attention

// One launch of the split attention.  A "row" of cache head g is one query
// of one token, R = token * group + (head within the group); the rows of a
// cache head share its keys.
struct AttnParams {
    const void *q;
    long long q_token_stride, q_head_stride;
    const void *k, *v;
    long long page_stride, row_stride, head_stride;
    long long n_pages;
    int page_shift;
    int d;                     // head_dim
    const int32_t *prefix_pages, *suffix_pages, *suffix_len;
    long long suffix_pages_stride;
    int n_seqs, n_q, hq, hkv, group;
    int rows;                  // n_seqs * n_q * group
    int prefix_len, max_suffix;
    float scale, scale_log2;   // of the scores; times log2(e)
    // parts: the prefix in p_splits ranges of p_keys keys for row tiles of
    // p_tile rows, every suffix in ranges of s_keys keys for tiles of s_tile
    int p_tile, p_tiles, p_splits, p_keys;
    int p_first;               // slots before the prefix part's own: the tcgen05 kernel's
    int s_tile, s_tiles, s_splits, s_keys;
    int p_blocks;              // blocks of the prefix part
    // the prefix's whole tiles of 128 keys on tcgen05 (attn_tc.cu), the blocks
    // above take what is left of it; mode 1: pairs of 128-row tiles, one slot per
    // split; 2: one row tile, two slots per split; 0: not used
    int t_mode, t_tiles, t_splits, t_keys, t_blocks;
    int t_len;                 // keys that it takes
    int t_wait;                // no launch of this call precedes it (no rest, no suffix)
    float4 *part_o;            // [slot][hkv] sums weighted with 2^(score - m), a row's elements 4 c .. at
                               //   row * o_row + c * o_four: rows innermost after the tcgen05 kernel, else outermost
    long long o_row, o_four;
    float2 *part_ml;           // [slot][hkv][rows] (m, l)
    void *o;
    long long o_token_stride, o_head_stride;
    float *lse;
    unsigned *status;
};
// Multiprocessors that the attention's splits are made for (a GB300's).  Not the
// device's own count: the workspace query knows no device, and the order in
// which a row's parts are added, so its bits, follows from the sizes alone.
constexpr int ATTN_SMS = 152;

// Rows of a tile for a part with `rows` rows per cache head (attn_prefix.cu).
int attn_tile_rows(int rows, int d);
bool attn_tc_takes(const qgemv_kv_cache &c);  // whether a cache's layout suits it
cudaError_t launch_attn_tc(const AttnParams &p, qgemv_dtype type, cudaStream_t st);
cudaError_t launch_attn(const AttnParams &p, qgemv_dtype type, qgemv_dtype o_type, cudaStream_t st);

}  // namespace qg
