// Eviction from the 4-bit cache by accumulated attention weight: select, then move.
//
// A weight becomes an unsigned key that orders as the number does (NaN as
// -infinity, -0 as 0).  The threshold T is the `need`-th highest key of the
// candidates, found by radix selection in three passes of 11, 11 and 10 bits: a
// histogram of the keys that agree with T's bits so far says which bits come
// next.  A row is then kept when it is recent, when its key is above T, or when it
// equals T and is among the first of those that are still needed; positions come
// from counts in index order, so ties go to the lower index and nothing depends
// on the order in which threads run.
//
// A request is selected by one CTA, a long one by a cluster of up to 16, each with an
// equal run of the candidates: the CTAs add their counts (the bins that are not
// empty) to the first one's through distributed shared memory, and that one tells
// them the bits.  A warp has a contiguous span; its weights are read five times, from
// L1 after the first.  What bounds the selection is the latency of its passes, not
// bytes: 262144 weights take 471 us with one CTA, 57 with 8 that read each other's
// histograms whole, 37 with 16 that exchange what is not empty; requests of up to 8192
// take 16 us with one CTA, 15 with two and 25 with four, so a CTA gets 16384.
//
// The move is bound by memory, 368 bytes read and written a row: a CTA looks up where
// 64 rows are and go, then copies them 16 bytes a thread with all its loads in flight
// (98304 rows: 14 us, 5.2 TB/s, in a list of launches; a warp a row took 25); it is launched while the
// selection ends.

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fp4.cuh"
#include "launch_status.h"
#include "ops.h"

namespace dsv4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
namespace cg = cooperative_groups;

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMaxCluster = 16;  // more than the portable 8, where the device allows it
constexpr int kWeightsPerCta = 16384;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = kFp4MoveRows;    // of a CTA
constexpr int kPieces = kFp4Slot / 16;     // of a row: 22 of data, one of scales
constexpr int kMovePieces = (kMoveRows * kPieces + kMoveThreads - 1) / kMoveThreads;

struct EParams {
    Fp4EvictArgs a;
    uint64_t block_div;
};

__device__ __forceinline__ void flag(int32_t *err, int bit)
{
    if (err != nullptr)
        atomicOr(err, bit);
}

__device__ __forceinline__ Span weights_span(const Fp4EvictArgs &a)
{
    return Span{a.weights, (uint64_t(a.b.batch - 1) * a.weights_stride + a.weights_width) * 4u};
}
__device__ __forceinline__ Span kept_span(const Fp4EvictArgs &a)
{
    return Span{a.kept, uint64_t(a.b.batch) * uint32_t(a.budget) * 4u};
}

__device__ __forceinline__ uint32_t order_key(float w)
{
    if (w != w)
        w = -INFINITY;
    const uint32_t b = __float_as_uint(w + 0.0f);  // -0 + 0 = 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// inclusive prefix sum of a value a thread over the CTA
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto warp_scan = [&](uint32_t x) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(kFull, x, d);
            if (lane >= d)
                x += o;
        }
        return x;
    };
    v = warp_scan(v);
    __syncthreads();
    if (lane == 31)
        warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0)
        warp_sums[lane] = warp_scan(warp_sums[lane]);
    __syncthreads();
    return v + (warp > 0 ? warp_sums[warp - 1] : 0u);
}

struct SelectShared {
    uint32_t hist[kBins];      // this CTA's counts
    uint32_t total[3][kBins];  // of the first CTA: the cluster's, a pass each
    uint32_t warp_sums[32];
    uint32_t digit, need;
    uint32_t above[kSelectWarps], equal[kSelectWarps];  // a warp's counts, then those before it
    uint32_t cta_above, cta_equal;
};

__global__ void __launch_bounds__(kSelectThreads) fp4_select_kernel(const EParams p)
{
    __shared__ SelectShared s;
    const Fp4EvictArgs &a = p.a;
    cg::cluster_group cluster = cg::this_cluster();
    let_kernel_after_begin();
    const int ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x / ctas;
    int64_t limit = int64_t(a.b.width) * a.b.block_size;
    limit = limit < a.weights_width ? limit : a.weights_width;
    int n = int(ldg4_in(a.b.lens + r, Span{a.b.lens, uint64_t(a.b.batch) * 4u}, a.b.err));
    cluster.sync();  // new_lens may be lens
    if (n > limit) {
        if (tid == 0 && rank == 0)
            flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
        n = int(limit);
    }
    n = n < 0 ? 0 : n;
    const int keep = n < a.budget ? n : a.budget;
    int32_t *kept = a.kept + int64_t(r) * a.budget;
    if (tid == 0 && rank == 0)
        st_i32_in(a.new_lens + r, keep, Span{a.new_lens, uint64_t(a.b.batch) * 4u}, a.b.err);
    // the recent rows, or all there are
    const int candidates = n <= a.budget ? 0 : n - a.recent;
    const int chosen = n <= a.budget ? 0 : a.budget - a.recent;
    // (in 64 bits: a budget may be less than a step below 2^31)
    for (int64_t i = rank * kSelectThreads + tid; i < a.budget - chosen; i += ctas * kSelectThreads)
        st_i32_in(kept + chosen + i, i < n - candidates ? candidates + int(i) : -1, kept_span(a), a.b.err);
    if (chosen == 0)
        return;  // the same in every CTA of the cluster

    // this CTA's candidates [begin, end), this warp's [from, to)
    const float *w = a.weights + r * a.weights_stride;
    const int per_cta = ((candidates + ctas - 1) / ctas + 31) & ~31;
    const int64_t begin64 = int64_t(rank) * per_cta;
    const int begin = begin64 < candidates ? int(begin64) : candidates;
    const int end = candidates - begin < per_cta ? candidates : begin + per_cta;
    const int per_warp = ((end - begin + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
    const int from = begin + warp * per_warp < end ? begin + warp * per_warp : end;
    const int to = end - from < per_warp ? end : from + per_warp;
    const auto key_at = [&](int i) {
        return i < to ? order_key(ldg_f32_in(w + i, weights_span(a), a.b.err)) : 0u;
    };
    // f(key, whether there is one, index) for the span in order, 32 at a time
    const auto span = [&](auto f) {
#pragma unroll 8
        for (int i = from + lane; i - lane < to; i += 32)
            f(key_at(i), i < to, i);
    };
    uint32_t need = uint32_t(chosen), prefix = 0u;
    for (int i = tid; i < kBins; i += kSelectThreads)
        s.hist[i] = s.total[0][i] = s.total[1][i] = s.total[2][i] = 0u;
    SelectShared *lead = cluster.map_shared_rank(&s, 0);
    cluster.sync();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        uint32_t *hist = ctas > 1 ? s.hist : s.total[pass];
        span([&](uint32_t k, bool there, int) {
            if (there && (pass == 0 || ((k ^ prefix) >> (pass == 1 ? 21 : 10)) == 0u))
                atomicAdd(&hist[(k >> shift) & mask], 1u);
        });
        __syncthreads();
        if (ctas > 1) {
            for (int i = tid; i < kBins; i += kSelectThreads) {
                if (s.hist[i] != 0u)
                    atomicAdd(&lead->total[pass][i], s.hist[i]);
                s.hist[i] = 0u;
            }
            cluster.sync();
        }
        if (rank == 0) {
            // thread i holds the bins that are 2i and 2i + 1 from the top
            const uint32_t first = s.total[pass][kBins - 1 - 2 * tid];
            const uint32_t second = s.total[pass][kBins - 2 - 2 * tid];
            const uint32_t upto = cta_scan(first + second, s.warp_sums);
            const uint32_t before = upto - first - second;
            if (upto >= need && before < need) {
                const bool one = before + first >= need;
                const uint32_t digit = uint32_t(kBins - 1 - 2 * tid) - (one ? 0u : 1u);
                for (int c = 0; c < ctas; ++c) {
                    SelectShared *to = cluster.map_shared_rank(&s, c);
                    to->digit = digit;
                    to->need = need - before - (one ? 0u : first);
                }
            }
        }
        if (ctas > 1)
            cluster.sync();
        else
            __syncthreads();
        prefix |= s.digit << shift;
        need = s.need;
        __syncthreads();
    }
    // `need` rows whose key is the threshold `prefix` are kept, the first ones.  A
    // span's counts, and those of the warps and CTAs before it.
    uint32_t above = 0u, equal = 0u;
    span([&](uint32_t k, bool there, int) {
        above += __popc(__ballot_sync(kFull, there && k > prefix));
        equal += __popc(__ballot_sync(kFull, there && k == prefix));
    });
    if (lane == 0) {
        s.above[warp] = above;
        s.equal[warp] = equal;
    }
    __syncthreads();
    if (warp == 0) {
        // exclusive counts of the warps, and the CTA's
        const uint32_t mine_above = s.above[lane], mine_equal = s.equal[lane];
        uint32_t x = mine_above, y = mine_equal;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t ox = __shfl_up_sync(kFull, x, d), oy = __shfl_up_sync(kFull, y, d);
            if (lane >= d) {
                x += ox;
                y += oy;
            }
        }
        s.above[lane] = x - mine_above;
        s.equal[lane] = y - mine_equal;
        if (lane == 31) {
            s.cta_above = x;
            s.cta_equal = y;
        }
    }
    cluster.sync();
    above = s.above[warp];
    equal = s.equal[warp];
    for (int c = 0; c < rank; ++c) {
        above += *cluster.map_shared_rank(&s.cta_above, c);
        equal += *cluster.map_shared_rank(&s.cta_equal, c);
    }
    cluster.sync();  // no CTA leaves while its counts are read
    const uint32_t lower = (1u << lane) - 1u;
    span([&](uint32_t k, bool there, int i) {
        const uint32_t is_above = __ballot_sync(kFull, there && k > prefix);
        const uint32_t is_equal = __ballot_sync(kFull, there && k == prefix);
        const uint32_t rank_equal = equal + __popc(is_equal & lower);
        const bool take = ((is_above >> lane) & 1u) || (((is_equal >> lane) & 1u) && rank_equal < need);
        const uint32_t at = above + __popc(is_above & lower) + (rank_equal < need ? rank_equal : need);
        if (take)
            st_i32_in(kept + at, i, kept_span(a), a.b.err);
        above += __popc(is_above);
        equal += __popc(is_equal);
    });
}

// CTA b moves the kept rows kMoveRows b.. of the batch.
__global__ void __launch_bounds__(kMoveThreads) fp4_move_kernel(const EParams p)
{
    __shared__ Fp4Row from_s[kMoveRows], to_s[kMoveRows];
    const Fp4EvictArgs &a = p.a;
    const int tid = threadIdx.x;
    const int64_t rows = int64_t(a.b.batch) * a.budget, row0 = int64_t(blockIdx.x) * kMoveRows;
    const uint32_t bs = uint32_t(a.b.block_size);
    uint8_t *cache = const_cast<uint8_t *>(a.b.cache);
    const Span cs{cache, uint64_t(a.b.num_blocks) * bs * kFp4Slot};
    wait_for_kernel_before();
    if (tid < kMoveRows) {
        Fp4Row from_at{nullptr, nullptr}, to_at{nullptr, nullptr};
        const int64_t i = row0 + tid;
        if (i < rows) {
            const int64_t r = i / a.budget;
            const uint32_t to = uint32_t(i - r * a.budget);
            // through L2: the selection wrote it, perhaps after this kernel began
            const int from = int(ld4_in(a.kept + i, kept_span(a), a.b.err));
            float weight = 0.0f;
            if (from >= 0) {
                const Span old_span{a.b.table, (uint64_t(a.b.batch - 1) * a.b.table_stride + a.b.width) * 4u};
                const Span new_span{a.new_table,
                                    (uint64_t(a.b.batch - 1) * a.new_table_stride + a.new_width) * 4u};
                const uint32_t f = fastdiv(uint32_t(from), p.block_div), t = fastdiv(to, p.block_div);
                const uint32_t src = ldg4_in(a.b.table + r * a.b.table_stride + f, old_span, a.b.err);
                const uint32_t dst = ldg4_in(a.new_table + r * a.new_table_stride + t, new_span, a.b.err);
                weight = ldg_f32_in(a.weights + r * a.weights_stride + from, weights_span(a), a.b.err);
                if (int64_t(src) < a.b.num_blocks && int64_t(dst) < a.b.num_blocks) {
                    from_at = fp4_row(cache, src, uint32_t(from) - f * bs, bs);
                    to_at = fp4_row(cache, dst, to - t * bs, bs);
                } else {
                    flag(a.b.err, DSV4_DEVERR_SLOT_RANGE);
                }
            }
            st_f32_in(a.new_weights + i, weight, Span{a.new_weights, uint64_t(rows) * 4u}, a.b.err);
        }
        from_s[tid] = from_at;
        to_s[tid] = to_at;
    }
    __syncthreads();
    uint4 v[kMovePieces];
    uint8_t *put[kMovePieces];
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k) {
        const int u = tid + k * kMoveThreads, row = u / kPieces, piece = u % kPieces;
        put[k] = nullptr;
        if (row < kMoveRows && from_s[row].data != nullptr) {
            const bool data = piece < kPieces - 1;
            v[k] = ldg16_in(data ? from_s[row].data + 16 * piece : from_s[row].scale, cs, a.b.err);
            put[k] = const_cast<uint8_t *>(data ? to_s[row].data + 16 * piece : to_s[row].scale);
        }
    }
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k)
        if (put[k] != nullptr)
            st16_in(put[k], v[k], cs, a.b.err);
}

// the largest cluster of the selection: 16 CTAs where the device takes them, else 8
int largest_cluster()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 8;
    const bool cached = dev >= 0 && dev < 64;
    int size = cached ? known[dev].load(std::memory_order_relaxed) : 0;
    if (size > 0)
        return size;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kMaxCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(kMaxCluster);
    config.blockDim = dim3(kSelectThreads);
    config.attrs = &attr;
    config.numAttrs = 1;
    int clusters = 0;
    size = cudaFuncSetAttribute(fp4_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                       cudaSuccess &&
                   cudaOccupancyMaxActiveClusters(&clusters, fp4_select_kernel, &config) == cudaSuccess &&
                   clusters > 0
               ? kMaxCluster
               : 8;
    if (cached)
        known[dev].store(size, std::memory_order_relaxed);
    return size;
}

}  // namespace

int launch_fp4_evict(const Fp4EvictArgs &a, cudaStream_t stream)
{
    EParams p{a, fastdiv_magic(uint32_t(a.b.block_size))};
    int64_t most = int64_t(a.b.width) * a.b.block_size;
    most = most < a.weights_width ? most : a.weights_width;
    const unsigned largest = unsigned(largest_cluster());
    unsigned cluster = 1;
    while (cluster < largest && int64_t(cluster) * kWeightsPerCta < most)
        cluster *= 2;
    const int st = launch_cluster(fp4_select_kernel, dim3(unsigned(a.b.batch) * cluster),
                                  dim3(kSelectThreads), cluster, stream, p);
    if (st != DSV4_OK)
        return st;
    const int64_t ctas = (int64_t(a.b.batch) * a.budget + kMoveRows - 1) / kMoveRows;
    return launch_after(fp4_move_kernel, dim3(unsigned(ctas)), dim3(kMoveThreads), stream, p);
}

}  // namespace dsv4

DSV4_BOUNDS_FLAG_READER(bounds_flag_fp4_evict)
