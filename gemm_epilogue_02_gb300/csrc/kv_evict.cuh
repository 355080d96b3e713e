// Eviction from the paged cache by accumulated attention weight.  Of sequence
// b's n = lengths[b] positions, each head keeps k = min(n, keep): the last
// r = min(recent, k), and of the n - r before them the k - r of largest weight
// (ties to the lowest position; a NaN counts as less than any number).  The kept
// rows are copied in order to positions 0 .. k - 1 of other pages, with their
// scales and weights.
//
// Two kernels: kv_select_kernel finds the positions, kv_gather_kernel copies
// the rows.
//
// Selection reads 4 bytes a position and is bound by latency: a cluster of
// blocks shares one sequence and head, each block a slice of its positions.  A
// weight becomes a 32-bit key of the same order, which stays in shared memory;
// kv_rank() finds the largest ones.
#pragma once
#include <cooperative_groups.h>

#include "kv_cache.cuh"
#include "kv_rank.cuh"

namespace tgemm {

constexpr int kSelectMaxCached = 48 * 1024;           // keys of a slice in shared memory (192 KiB); of longer ones none

struct EvictParams {
    KvView from, to;
    KvTable table, to_table;       // to_table.lengths is not used
    KvWeights weights, to_weights;
    int *kept;                     // [batch, heads, keep]
    int *to_lengths;
    int keep, recent;
    int cached;                    // keys that the selection's blocks have room for
    unsigned int *status;
};

// Grid: (cluster size, heads, batch), a cluster along x.  kAlone: of one block.
template <int kThreads, bool kAlone>
__global__ void __launch_bounds__(kThreads, 2) kv_select_kernel(const EvictParams p) {
    extern __shared__ uint32_t keys[];
    __shared__ RankShared<kThreads> sh;
    __shared__ int s_n;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = kAlone ? 1 : static_cast<int>(cluster.num_blocks()), rank = kAlone ? 0 : static_cast<int>(cluster.block_rank());
    const int head = blockIdx.y, b = blockIdx.z;
    kv_rank_clear(sh);
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        bool bad = false;
        int length = kv_length(p.table.lengths[b], p.table.width, p.from.page_size, &bad);
        if (length > p.weights.width) {
            length = p.weights.width;
            bad = true;
        }
        if (bad && rank == 0) record_status(p.status, kStatusCache);
        s_n = length;
    }
    __syncthreads();                             // the histograms are zero
    const int n = s_n, k = min(n, p.keep), r = min(p.recent, k);
    const float *w = p.weights.base + b * p.weights.batch_stride + head * p.weights.head_stride;
    float *to_w = p.to_weights.base + b * p.to_weights.batch_stride + head * p.to_weights.head_stride;
    int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    if (head == 0 && rank == 0 && threadIdx.x == 0) p.to_lengths[b] = k;
    const int first = n - r, best = k - r;       // of the first `first` positions, `best` stay
    const int slice = (first + blocks - 1) / blocks, lo = min(first, rank * slice);
    const float *const mine = w + lo;
    const bool some = best > 0 && best < first;
    const int size = some ? min(first, lo + slice) - lo : 0;
    const bool cached = size <= p.cached;
    auto key_at = [&](int i) { return cached ? keys[i] : kv_weight_key(__float_as_uint(mine[i])); };
    if (some && cached) {
#pragma unroll 8
        for (int i = threadIdx.x; i < size; i += kThreads) keys[i] = kv_weight_key(__float_as_uint(mine[i]));
    }
    // What follows the best: the recent ones, and -1 past k.
    for (int i = best + rank * kThreads + threadIdx.x; i < p.keep; i += blocks * kThreads) {
        const int j = first + i - best;
        kept[i] = i < k ? j : -1;
        to_w[i] = i < k ? w[j] : 0.0f;
    }
    if (!some) {
        if (best > 0)                            // nothing is evicted
            for (int j = rank * kThreads + threadIdx.x; j < first; j += blocks * kThreads) {
                kept[j] = j;
                to_w[j] = w[j];
            }
        if (kAlone) return;
        // The blocks of a cluster go on together to every barrier, whatever length each of them has read.
    }
    __syncthreads();                             // the keys are there

    kv_rank<kAlone ? RankBy::kBlock : RankBy::kCluster>(
        sh, size, best, p.status, key_at,
        [&](int at, int i) {
            kept[at] = lo + i;
            to_w[at] = mine[i];
        });
}

// Copying the kept rows: as in kv_append_kernel a block first finds the places
// of a chunk of rows and then streams them, keys and values, all requested
// before the first is stored.  Grid: (heads * batch, chunks at most).
constexpr int kGatherThreads = 256;

template <bool kE4m3, int kLanes, int kUnroll>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const EvictParams p) {
    constexpr int kPass = kGatherThreads / kLanes, kRows = kPass * kUnroll;
    __shared__ long long s_src[kRows], s_dst[kRows];
    __shared__ int s_n;
    const int b = static_cast<int>(blockIdx.x) / p.from.heads, head = static_cast<int>(blockIdx.x) - b * p.from.heads;
    const int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    griddep_wait();
    if (threadIdx.x == 0) {
        bool bad = false;
        s_n = min(kv_length(p.table.lengths[b], p.table.width, p.from.page_size, &bad), p.weights.width);
    }
    __syncthreads();
    const int n = s_n, k = min(n, p.keep), best = k - min(p.recent, k), shift = n - k;
    const int piece = threadIdx.x % kLanes, in_pass = threadIdx.x / kLanes;
    const bool inside = piece * 16 < p.from.row_bytes;
    for (int i0 = static_cast<int>(blockIdx.y) * kRows; i0 < k; i0 += static_cast<int>(gridDim.y) * kRows) {
        const int row = i0 + static_cast<int>(threadIdx.x);
        if (threadIdx.x < kRows) {
            long long src = 0, dst = -1;
            if (row < k) {
                int page, slot, to_page, to_slot;
                // (kept[row] < n, unless another stream has changed a length or a weight meanwhile)
                const int from = shift > 0 && row < best ? kept[row] : row + shift;
                if (static_cast<unsigned>(from) >= static_cast<unsigned>(n) ||
                    row >= static_cast<long long>(p.to_table.width) * p.to.page_size ||
                    !kv_row(p.table.pages + b * p.table.stride, from, p.from.page_size, p.from.pages, &page, &slot) ||
                    !kv_row(p.to_table.pages + b * p.to_table.stride, row, p.to.page_size, p.to.pages, &to_page,
                            &to_slot)) {
                    record_status(p.status, kStatusCache);
                } else {
                    src = kv_offset(p.from, page, slot, head);
                    dst = kv_offset(p.to, to_page, to_slot, head);
                    if (!TGEMM_CHECK(dst + p.to.row_bytes <= p.to.dbg_bytes, kChkKvRow, p.status)) dst = -1;
                    if (kE4m3) {
                        const long long s = kv_scale_offset(p.from, page, slot, head);
                        const long long d = kv_scale_offset(p.to, to_page, to_slot, head);
                        p.to.k_scale[d] = p.from.k_scale[s];
                        p.to.v_scale[d] = p.from.v_scale[s];
                    }
                }
            }
            s_src[threadIdx.x] = src;
            s_dst[threadIdx.x] = dst;
        }
        __syncthreads();
        uint4 x[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kPass + in_pass;
            if (s_dst[i] >= 0 && inside) {
                x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(p.from.k + s_src[i]) + piece);
                x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(p.from.v + s_src[i]) + piece);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kPass + in_pass;
            if (s_dst[i] >= 0 && inside) {
                *(reinterpret_cast<uint4 *>(p.to.k + s_dst[i]) + piece) = x[u][0];
                *(reinterpret_cast<uint4 *>(p.to.v + s_dst[i]) + piece) = x[u][1];
            }
        }
        __syncthreads();
    }
}

}  // namespace tgemm
