// Internal interface between the C-ABI layer (api.cpp) and the kernels of the
// operations beside the whole-warp fused kernels: the half-warp fused kernel
// (qnorm_rope_kv_insert_half.cu), the KV-row kernel for calls with no q
// (kv_rows.cu), the MXFP8 activation quantiser (gemma_rmsnorm_mxfp8.cu), the
// indexer-K insert and gather (indexer_k.cu), the check of the bounded waits
// (wait_check.cu) and the 4-bit cache's operators (fp4_*.cu).
// Not installed; not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsv4kv.h"
#include "launch.h"

namespace dsv4 {

// KV rows with no q, one row per quarter-warp (kv_rows.cu); the grid is capped at max_ctas.
int kv_rows_ctas_per_sm(int *ctas_per_sm);
int kv_rows_per_warp();
int launch_kv_rows(int store_mode, const LaunchArgs &a, int64_t max_ctas, cudaStream_t stream);

// Warps per CTA of the FP8 cache reader (dequant_gather.cu; its other entry points
// are in launch.h).
int gather_warps_per_cta();

// The fused step with one row per half-warp (qnorm_rope_kv_insert_half.cu).
int half_ctas_per_sm(int *ctas_per_sm);
int half_q_rows_per_warp();
int launch_half(int store_mode, const LaunchArgs &a, int64_t ctas, cudaStream_t stream);

// Residual add + Gemma RMSNorm + MXFP8 rows.
int launch_gemma_rmsnorm_mxfp8(const uint16_t *x, const uint16_t *residual, const uint16_t *gamma,
                               int64_t m, int32_t n, float eps, uint16_t *residual_out,
                               uint8_t *codes, uint8_t *scales, cudaStream_t stream);

// Indexer-K quant-insert and gather; grids are capped at max_ctas.
int indexer_ctas_per_sm(int *ctas_per_sm, bool gather);
int launch_indexer_insert(const uint16_t *k, const int64_t *slots, uint8_t *cache,
                          int64_t num_blocks, int32_t block_size, int64_t rows, int32_t *err,
                          int64_t max_ctas, cudaStream_t stream);
int launch_indexer_gather(const uint8_t *cache, int64_t num_blocks, int32_t block_size,
                          const int64_t *slots, int64_t rows, uint8_t *k_out, float *scale_out,
                          int32_t *err, int64_t max_ctas, cudaStream_t stream);

// One warp waits on an mbarrier nothing completes, for at most max_cycles SM
// cycles (clamped to the kernels' own limit), then flags DSV4_DEVERR_TIMEOUT.
int launch_wait_check(int64_t max_cycles, int32_t *err, cudaStream_t stream);

// What the operators over the paged caches have in common: B requests, their pages by a
// block table, and Q new tokens each.
struct PagedBatch {
    const uint8_t *cache;
    int64_t num_blocks;
    int32_t block_size;
    const int32_t *table;   // [batch] rows of `width` entries, `table_stride` apart
    int64_t table_stride;
    int32_t width;
    const int32_t *lens;    // [batch], the new tokens included
    int32_t batch;
    int32_t *err;
};

// Positions that a row tile with keys may take on the line that is dealt to the CTAs,
// beside one for each of its tiles of keys (fp4_tiles.cuh).
constexpr int kFp4StartCost = 2;

struct AttentionArgs {
    PagedBatch b;
    const uint16_t *q;      // [batch, q_len, heads, 512]
    int32_t q_len;
    int32_t heads;
    float scale;
    int32_t window;         // 0: none
    const uint64_t *tree;   // [batch, q_len] or null: the drafted keys that each drafted token sees
    const float *sinks;     // [heads] or null
    uint16_t *out;
    float *lse;             // [batch, q_len, heads]: written by the attention, read by the weights
    float *weights;         // [batch] rows, weights_stride apart
    int64_t weights_stride;
    int32_t weights_width;
};

constexpr int kFp4MoveRows = 64;  // kept rows that a CTA of the eviction moves

struct Fp4EvictArgs {
    PagedBatch b;             // b.cache is written too
    const float *weights;
    int64_t weights_stride;
    int32_t weights_width;
    int32_t budget;
    int32_t recent;
    const int32_t *new_table;
    int64_t new_table_stride;
    int32_t new_width;
    int32_t *kept;          // [batch, budget]
    int32_t *new_lens;      // [batch]
    float *new_weights;     // [batch, budget]
};

// Keys in a tile of the attention over the FP8 and bf16 caches, and the positions that
// beginning a row tile takes on its line: with 0, 2, 3, 4, 6 and 8 of them 48 requests of up to 4096
// FP8 keys take (in a graph) 45.8, 38.4, 38.7, 37.9, 38.9 and 39.4 us, 128 of up to 8192 266, 253, 251, 253,
// 255 and 256, 32 with 16 drafted tokens 339, 293, 289, 290, 297 and 302, and wide trees over bf16 rows
// 590, 596, 597, 598, 600 and 603.
constexpr int kLatentTileKeys = 64;
constexpr int kLatentStartCost = 4;

// latent_attention.cu; the workspace holds latent_attention_workspace() bytes
size_t latent_attention_workspace();
int launch_latent_attention(int store_mode, const AttentionArgs &a, void *workspace, cudaStream_t stream);

// Drafted tokens of a request: a token's ancestors are bits of one word.
constexpr int kMaxDrafted = 64;

struct TreeKeepArgs {
    PagedBatch b;              // b.cache is written too
    int32_t q_len;
    const int32_t *path;       // [batch, q_len]
    const int32_t *path_lens;  // [batch]
    int32_t *new_lens;         // [batch]
};

// tree_keep.cu
int launch_tree_keep(int store_mode, const TreeKeepArgs &a, cudaStream_t stream);

constexpr int kMaxRopeDim = 256;

struct RopeTableArgs {
    const double *frequencies;  // host, [rope_dim / 2]
    int32_t rope_dim;
    double magnitude;
    const int64_t *positions;   // [count] or null: first, first + 1, ...
    int64_t first, count;
    float *out;                 // [count, rope_dim]
    int32_t sms;
    int32_t *err;
};

// rope_table.cu
int launch_rope_table(const RopeTableArgs &a, cudaStream_t stream);

struct RopeRowsArgs {
    const uint8_t *x;
    uint8_t *out;               // x itself, with the same strides, or apart from it
    int32_t type;
    int64_t tokens;
    int32_t heads, width;
    int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride;  // elements
    int32_t offset, rope_dim, layout;
    bool inverse;
    const int64_t *positions;   // [tokens]
    const float *cos_sin;       // [max_position, rope_dim]
    int64_t max_position;
    int32_t sms;
    int32_t *err;
};

// rope_rows.cu
int launch_rope_rows(const RopeRowsArgs &a, cudaStream_t stream);

// fp4_gather.cu; the grid is capped at max_ctas
int fp4_gather_ctas_per_sm(int *ctas_per_sm);
int launch_fp4_gather(const uint8_t *cache, int64_t num_blocks, int32_t block_size,
                      const int64_t *slots, int64_t rows, uint16_t *out, int32_t *err,
                      int64_t max_ctas, cudaStream_t stream);
// fp4_attention.cu; the workspace holds fp4_attention_workspace() bytes
size_t fp4_attention_workspace();
int launch_fp4_attention(const AttentionArgs &a, void *workspace, cudaStream_t stream);
// fp4_weights.cu
int launch_fp4_weights(const AttentionArgs &a, cudaStream_t stream);
// fp4_evict.cu
int launch_fp4_evict(const Fp4EvictArgs &a, cudaStream_t stream);

// The checked build's record of skipped accesses, one reader per kernel file
// (DSV4_BOUNDS_FLAG_READER of bounds.cuh); -1 in the release build.
int bounds_flag_fused(int reset);
int bounds_flag_half(int reset);
int bounds_flag_kv_rows(int reset);
int bounds_flag_gather(int reset);
int bounds_flag_indexer(int reset);
int bounds_flag_mxfp8(int reset);
int bounds_flag_fp4_gather(int reset);
int bounds_flag_fp4_attention(int reset);
int bounds_flag_fp4_weights(int reset);
int bounds_flag_fp4_evict(int reset);
int bounds_flag_latent_attention(int reset);
int bounds_flag_tree_keep(int reset);
int bounds_flag_rope_table(int reset);
int bounds_flag_rope_rows(int reset);

}  // namespace dsv4
