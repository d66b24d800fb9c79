// C-ABI entry points of the 4-bit cache's operators: argument checks on the
// host, before anything is enqueued, then the launches.  The 4-bit insert is in
// api.cpp, beside the stores it shares its arguments with.

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "dsv4kv.h"
#include "hostcheck.h"
#include "ops.h"

namespace {

using dsv4::aligned;
using dsv4::check_sizes;
using dsv4::PagedBatch;
using dsv4::too_many_slots;

// tiles of 128 keys
int check_attention(int32_t q_len, int32_t num_heads, int32_t batch, float scale, int32_t window,
                    int64_t most_keys)
{
    return dsv4::check_attention(q_len, num_heads, batch, scale, window, most_keys, 128,
                                 dsv4::kFp4StartCost);
}

// SM count times CTAs per SM of the reader, per device (bit-identical values
// from any thread, so a race only repeats the queries)
constexpr int kMaxDevices = 64;
std::atomic<int64_t> g_resident[kMaxDevices];

int resident_readers(int64_t *resident)
{
    int dev = 0, sms = 0, per = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return DSV4_ERR_CUDA;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    *resident = cached ? g_resident[dev].load(std::memory_order_relaxed) : 0;
    if (*resident > 0)
        return DSV4_OK;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1 ||
        dsv4::fp4_gather_ctas_per_sm(&per) != DSV4_OK || per < 1)
        return DSV4_ERR_CUDA;
    *resident = int64_t(sms) * per;
    if (cached)
        g_resident[dev].store(*resident, std::memory_order_relaxed);
    return DSV4_OK;
}

}  // namespace

extern "C" {

size_t dsv4_fp4_cache_bytes(int64_t num_blocks, int32_t block_size)
{
    if (num_blocks < 1 || block_size < 1)
        return 0;
    return size_t(num_blocks) * size_t(block_size) * DSV4_FP4_SLOT_BYTES;
}

int dsv4_fp4_dequant_gather(const uint8_t *kv_cache, int64_t num_blocks, int32_t block_size,
                            const int64_t *slots, int64_t num_rows, void *out,
                            int32_t *device_error, void *stream)
{
    if (num_rows < 0 || num_blocks < 1 || block_size < 1)
        return DSV4_ERR_SHAPE;
    if (too_many_slots(num_blocks, block_size) || num_rows > INT64_MAX / 4096)
        return DSV4_ERR_SHAPE;
    if (num_rows == 0)
        return DSV4_OK;
    if (!kv_cache || !slots || !out)
        return DSV4_ERR_NULL;
    if (!aligned(kv_cache, 16) || !aligned(slots, 8) || !aligned(out, 16) ||
        !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    int64_t resident = 0;
    if (resident_readers(&resident) != DSV4_OK)
        return DSV4_ERR_CUDA;
    return dsv4::launch_fp4_gather(kv_cache, num_blocks, block_size, slots, num_rows,
                                   static_cast<uint16_t *>(out), device_error, resident,
                                   static_cast<cudaStream_t>(stream));
}

size_t dsv4_fp4_attention_workspace_bytes(void)
{
    return dsv4::fp4_attention_workspace();
}

int dsv4_fp4_attention(const void *q, const uint8_t *kv_cache, int64_t num_blocks,
                       int32_t block_size, const int32_t *block_table, int64_t table_stride,
                       int32_t table_width, const int32_t *seq_lens, int32_t batch,
                       int32_t q_len, int32_t num_heads, float scale, int32_t window,
                       const float *sinks, void *out, float *lse, void *workspace,
                       size_t workspace_bytes, int32_t *device_error, void *stream)
{
    int st = check_sizes(num_blocks, block_size, table_stride, table_width, batch);
    if (st == DSV4_OK)
        st = check_attention(q_len, num_heads, batch, scale, window,
                             int64_t(table_width) * block_size);
    if (st != DSV4_OK)
        return st;
    if (workspace_bytes < dsv4_fp4_attention_workspace_bytes())
        return DSV4_ERR_SHAPE;
    if (batch == 0)
        return DSV4_OK;
    if (!q || !kv_cache || !block_table || !seq_lens || !out || !workspace)
        return DSV4_ERR_NULL;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(sinks, 4) ||
        !aligned(lse, 4) || !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::AttentionArgs a = {};
    a.b = PagedBatch{kv_cache, num_blocks, block_size, block_table, table_stride,
                   table_width, seq_lens, batch, device_error};
    a.q = static_cast<const uint16_t *>(q);
    a.q_len = q_len;
    a.heads = num_heads;
    a.scale = scale;
    a.window = window < int64_t(table_width) * block_size ? window : 0;
    a.sinks = sinks;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    return dsv4::launch_fp4_attention(a, workspace, static_cast<cudaStream_t>(stream));
}

int dsv4_fp4_attention_weights(const void *q, const uint8_t *kv_cache, int64_t num_blocks,
                               int32_t block_size, const int32_t *block_table,
                               int64_t table_stride, int32_t table_width,
                               const int32_t *seq_lens, int32_t batch, int32_t q_len,
                               int32_t num_heads, float scale, int32_t window, const float *lse,
                               float *weights, int64_t weights_stride, int32_t weights_width,
                               int32_t *device_error, void *stream)
{
    int st = check_sizes(num_blocks, block_size, table_stride, table_width, batch);
    if (st == DSV4_OK)
        st = check_attention(q_len, num_heads, batch, scale, window,
                             int64_t(table_width) * block_size);
    if (st != DSV4_OK)
        return st;
    if (weights_width < 0 || weights_stride < weights_width ||
        weights_stride > INT64_MAX / 4096 / 65536)
        return DSV4_ERR_SHAPE;
    if (batch == 0)
        return DSV4_OK;
    if (!q || !kv_cache || !block_table || !seq_lens || !lse || !weights)
        return DSV4_ERR_NULL;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(weights, 4) ||
        !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::AttentionArgs a = {};
    a.b = PagedBatch{kv_cache, num_blocks, block_size, block_table, table_stride,
                   table_width, seq_lens, batch, device_error};
    a.q = static_cast<const uint16_t *>(q);
    a.q_len = q_len;
    a.heads = num_heads;
    a.scale = scale;
    a.window = window < int64_t(table_width) * block_size ? window : 0;
    a.lse = const_cast<float *>(lse);
    a.weights = weights;
    a.weights_stride = weights_stride;
    a.weights_width = weights_width;
    return dsv4::launch_fp4_weights(a, static_cast<cudaStream_t>(stream));
}

int dsv4_fp4_evict(uint8_t *kv_cache, int64_t num_blocks, int32_t block_size,
                   const int32_t *block_table, int64_t table_stride, int32_t table_width,
                   const int32_t *seq_lens, int32_t batch, const float *weights,
                   int64_t weights_stride, int32_t weights_width, int32_t budget,
                   int32_t recent, const int32_t *new_block_table, int64_t new_table_stride,
                   int32_t new_table_width, int32_t *kept, int32_t *new_seq_lens,
                   float *new_weights, int32_t *device_error, void *stream)
{
    const int st = check_sizes(num_blocks, block_size, table_stride, table_width, batch);
    if (st != DSV4_OK)
        return st;
    if (weights_width < 0 || weights_stride < weights_width ||
        weights_stride > INT64_MAX / 4096 / 65536 || budget < 1 || recent < 0 || recent > budget ||
        new_table_width < 1 || new_table_stride < new_table_width ||
        new_table_stride > INT64_MAX / 4096 / 65536 ||
        int64_t(new_table_width) * block_size < budget ||
        int64_t(batch) * budget > int64_t(INT32_MAX) * dsv4::kFp4MoveRows)  // a grid's CTAs
        return DSV4_ERR_SHAPE;
    if (batch == 0)
        return DSV4_OK;
    if (!kv_cache || !block_table || !seq_lens || !weights || !new_block_table || !kept ||
        !new_seq_lens || !new_weights)
        return DSV4_ERR_NULL;
    if (!aligned(kv_cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(weights, 4) || !aligned(new_block_table, 4) || !aligned(kept, 4) ||
        !aligned(new_seq_lens, 4) || !aligned(new_weights, 4) || !aligned(device_error, 4))
        return DSV4_ERR_ALIGN;
    dsv4::Fp4EvictArgs a = {};
    a.b = PagedBatch{kv_cache, num_blocks, block_size, block_table, table_stride,
                   table_width, seq_lens, batch, device_error};
    a.weights = weights;
    a.weights_stride = weights_stride;
    a.weights_width = weights_width;
    a.budget = budget;
    a.recent = recent;
    a.new_table = new_block_table;
    a.new_table_stride = new_table_stride;
    a.new_width = new_table_width;
    a.kept = kept;
    a.new_lens = new_seq_lens;
    a.new_weights = new_weights;
    return dsv4::launch_fp4_evict(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
