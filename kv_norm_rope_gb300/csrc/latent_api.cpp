// C-ABI entry points of the attention over the FP8 and bf16 caches and of the move that keeps
// an accepted path: argument checks on the host, before anything is enqueued, then the launches.

#include <cuda_runtime.h>

#include <cstdint>

#include "dsv4kv.h"
#include "hostcheck.h"
#include "ops.h"

namespace {

using dsv4::aligned;
using dsv4::PagedBatch;

// the alignment of a cache with this store
uintptr_t cache_alignment(int store_mode)
{
    return store_mode == DSV4_STORE_FP8 ? 8 : store_mode == DSV4_STORE_INDEXER ? 4 : 16;
}

}  // namespace

extern "C" {

size_t dsv4_latent_attention_workspace_bytes(void)
{
    return dsv4::latent_attention_workspace();
}

int dsv4_latent_attention(int store_mode, const void *q, const void *kv_cache, int64_t num_blocks,
                          int32_t block_size, const int32_t *block_table, int64_t table_stride,
                          int32_t table_width, const int32_t *seq_lens, int32_t batch, int32_t q_len,
                          int32_t num_heads, float scale, int32_t window, const uint64_t *tree,
                          const float *sinks, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, int32_t *device_error, void *stream)
{
    if (store_mode != DSV4_STORE_FP8 && store_mode != DSV4_STORE_BF16)
        return DSV4_ERR_VALUE;
    int st = dsv4::check_sizes(num_blocks, block_size, table_stride, table_width, batch);
    if (st == DSV4_OK)
        st = dsv4::check_attention(q_len, num_heads, batch, scale, window, int64_t(table_width) * block_size,
                                   dsv4::kLatentTileKeys, dsv4::kLatentStartCost);
    if (st != DSV4_OK)
        return st;
    if (workspace_bytes < dsv4_latent_attention_workspace_bytes())
        return DSV4_ERR_SHAPE;
    // drafted tokens are bits of a word, and a window holds all of them
    if (tree && (q_len > dsv4::kMaxDrafted || (window > 0 && window < q_len)))
        return DSV4_ERR_SHAPE;
    if (batch == 0)
        return DSV4_OK;
    if (!q || !kv_cache || !block_table || !seq_lens || !out || !workspace)
        return DSV4_ERR_NULL;
    if (!aligned(q, 16) || !aligned(kv_cache, cache_alignment(store_mode)) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(tree, 8) || !aligned(sinks, 4) || !aligned(lse, 4) || !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::AttentionArgs a = {};
    a.b = PagedBatch{static_cast<const uint8_t *>(kv_cache), num_blocks, block_size, block_table, table_stride,
                     table_width, seq_lens, batch, device_error};
    a.q = static_cast<const uint16_t *>(q);
    a.q_len = q_len;
    a.heads = num_heads;
    a.scale = scale;
    a.window = window < int64_t(table_width) * block_size ? window : 0;
    a.tree = tree;
    a.sinks = sinks;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    return dsv4::launch_latent_attention(store_mode, a, workspace, static_cast<cudaStream_t>(stream));
}

int dsv4_tree_keep(int store_mode, void *kv_cache, int64_t num_blocks, int32_t block_size,
                   const int32_t *block_table, int64_t table_stride, int32_t table_width,
                   const int32_t *seq_lens, int32_t batch, int32_t q_len, const int32_t *path,
                   const int32_t *path_lens, int32_t *new_seq_lens, int32_t *device_error, void *stream)
{
    if (store_mode != DSV4_STORE_FP8 && store_mode != DSV4_STORE_BF16 && store_mode != DSV4_STORE_FP4 &&
        store_mode != DSV4_STORE_INDEXER)
        return DSV4_ERR_VALUE;
    const int st = dsv4::check_sizes(num_blocks, block_size, table_stride, table_width, batch);
    if (st != DSV4_OK)
        return st;
    if (q_len < 1 || q_len > dsv4::kMaxDrafted)
        return DSV4_ERR_SHAPE;
    if (batch == 0)
        return DSV4_OK;
    if (!kv_cache || !block_table || !seq_lens || !path || !path_lens || !new_seq_lens)
        return DSV4_ERR_NULL;
    if (!aligned(kv_cache, cache_alignment(store_mode)) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(path, 4) || !aligned(path_lens, 4) || !aligned(new_seq_lens, 4) || !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::TreeKeepArgs a = {};
    a.b = PagedBatch{static_cast<const uint8_t *>(kv_cache), num_blocks, block_size, block_table, table_stride,
                     table_width, seq_lens, batch, device_error};
    a.q_len = q_len;
    a.path = path;
    a.path_lens = path_lens;
    a.new_lens = new_seq_lens;
    return dsv4::launch_tree_keep(store_mode, a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
