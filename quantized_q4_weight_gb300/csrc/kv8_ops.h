// kv8_ops.h -- internal interface between the C ABI (kv8_api.cu) and the
// kernels of a step over an 8-bit cache and of beam search: norms with the
// rotation (norm_rope.cu), the cache write (kv8_append.cu), attention over the
// cache (kv8_attn.cuh), the beams' best continuations (beam_select.cu) and the
// reordering of pages (fork_pages.cu).
#pragma once

#include "decode_ops.h"

namespace qg {

// ------------------------------------------------------- norm and rotation

struct NormRopeParams {
    RopeParams r;             // without a cache: slots null, ck = k_out, page_shift -1, row_stride = k_out_stride
    const float *q_weight, *k_weight;
    float eps;
    int v_heads;              // hkv, or 0 without a cache
};
cudaError_t launch_norm_rope(NormRopeParams &p, qgemv_dtype in, qgemv_dtype q_out, qgemv_dtype k_out, bool half_layout,
                             bool vec, long long n_tokens, int sms, cudaStream_t st);

// ------------------------------------------------------------ 8-bit cache

// Where a row's codes and a block's scale lie.
struct Kv8Layout {
    uint8_t *k, *v;
    float *ks, *vs;
    long long page_stride, row_stride, head_stride;     // bytes
    long long scale_page, scale_block, scale_head;      // floats
    long long n_pages;
    int page_shift, block_shift;
};

struct Kv8AppendParams {
    Kv8Layout c;
    const void *k, *v;
    int k_stride, v_stride, code_row;     // elements between tokens, bytes between a page's rows
    long long n_tokens;
    const int32_t *first, *lens, *pages;
    long long pages_stride;
    int n_new, max_new, max_len, blocks;  // n_new: without `first`; blocks: that max_new rows can touch
    int n_seqs, hkv, d;
    int pieces;                           // threads' pieces of 8 elements a row: d / 8
    int per_piece;                        // 65536 / pieces, rounded up
    int items;                            // heads of k and v that a block takes (kv8_append.cu)
    unsigned *status;
};
cudaError_t launch_kv8_append(const Kv8AppendParams &p, qgemv_dtype in, qgemv_code_type code, bool vec, cudaStream_t st);

struct Kv8AttnParams {
    Kv8Layout c;
    const void *q;
    long long q_token_stride, q_head_stride;
    int q_bf16;
    const int32_t *lens, *pages;
    long long pages_stride;
    int n_seqs, n_q, hq, hkv, group, d;
    int max_len, window, sinks;
    int rows, row_tiles, tile_rows;  // of a sequence and cache head: n_q * group, in row_tiles of tile_rows
    float scale_log2;
    float per_group;                 // 1 / group
    int balanced, ranges, grid;      // `ranges` of all tiles over `grid` blocks, or a block for each unit
    int aligned;                     // ranges begin with their sequence: there are eight times as many as sequences
    int wide;                        // blocks of twice the warps (kv8_attn.cuh)
    int parts_by_unit;               // there are no more units than blocks
    int4 *parts;                     // of each unit, or block: sequence, unit, first part, parts (0: none)
    float *part_o;                   // [2 grid][tile rows, padded][d]
    float2 *part_ml;                 // [2 grid][tile rows, padded]
    int combine_lanes;               // groups that share a row's elements in the combining launch: 1 .. 32
    void *o;
    int o_type;                      // qgemv_dtype
    long long o_token_stride, o_head_stride;
    float *lse;
    unsigned *status;
};
constexpr int KV8_KEYS = 32;         // keys of a tile
constexpr int KV8_SPLIT_MIN = 6;     // tiles of a range at least: one for each warp of the narrowest blocks
// Rows of a tile at most, and, for tiles of 8 nt rows, blocks a multiprocessor
// and warps a block.
constexpr int kv8_tile_rows(int d) { return d <= 128 ? 32 : 16; }
constexpr int kv8_blocks(int d, int nt) { return d > 128 || (d > 64 && nt > 2) || nt > 3 ? 1 : 2; }
constexpr int kv8_warps(int d, int nt)
{
    if (d > 128) return 6;
    return d > 64 && d <= 96 && nt == 3 ? 12 : nt == 4 || (d > 64 && nt == 3) || (d <= 64 && nt <= 2) ? 8 : 6;
}
// One translation unit for each type of codes (kv8_attn.cuh).
cudaError_t launch_kv8_attn_int8(const Kv8AttnParams &p, cudaStream_t st);
cudaError_t launch_kv8_attn_e4m3(const Kv8AttnParams &p, cudaStream_t st);

// ------------------------------------------------------------------- beams

struct BeamParams {
    const void *x;
    long long x_stride, vocab;
    const float *scores;
    const int32_t *done;
    float *score;
    long long *token;
    int32_t *parent;
    int beams, n_best, row0;      // row0: of the launch's first group (parents are rows of all groups)
    int slices, slice;            // of a row; elements of one, a multiple of 2048
    unsigned *cnt;                // [groups] arrivals, zero between launches
    float2 *part_ml;              // [rows][slices] maximum, sum of exponentials
    unsigned long long *part;     // [rows][slices][n_best] keys, best first; 0: none
};
constexpr int BEAM_GROUPS = 4080;  // groups of a launch: their arrivals fit the counter area before its last 64 bytes
int beam_slices(long long rows, long long vocab);  // slices of a row
cudaError_t launch_beam(const BeamParams &p, qgemv_dtype type, int groups, cudaStream_t st);

// ------------------------------------------------------------------- pages

// One array of pages of all caches of a launch: codes or elements, or scales.
struct ForkParams {
    qgemv_fork f;
    int n_arrays, page_shift, block_shift;      // block_shift -1: no scales
    int heads, head_bytes;                      // a multiple of 16
    long long n_pages;
    long long page_stride[64], row_stride[64], head_stride[64];    // bytes, of each cache
    void *base[128];                            // k and v of each cache
    float *scale[128];
    long long scale_page[64], scale_block[64], scale_head[64];
    int first;                                  // this launch writes tables and lengths
    unsigned *status;
};
constexpr int FORK_CACHES = 64;
cudaError_t launch_fork(const ForkParams &p, int sms, cudaStream_t st);

}  // namespace qg
