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
// weight becomes a 32-bit key of the same order; the key of rank k - r is found
// 11 bits at a time (11 + 11 + 10) from histograms of the keys that share the
// bits found so far, which the blocks add up through distributed shared memory;
// then every larger key is kept, and of the equal ones the first few in order of
// position.  A slice stays in the block's L1 between its five passes.
#pragma once
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace tgemm {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectBins = 2048;

struct EvictParams {
    KvView from, to;
    KvTable table, to_table;       // to_table.lengths is not used
    KvWeights weights, to_weights;
    int *kept;                     // [batch, heads, keep]
    int *to_lengths;
    int keep, recent;
    unsigned int *status;
};

// A key of the same order as the weight: larger weight, larger key; -0 as +0;
// NaN below every number.
__host__ __device__ inline uint32_t kv_weight_key(uint32_t bits) {
    if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    if (bits == 0x80000000u) bits = 0u;
    return (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
}

// Grid: (cluster size, heads, batch), a cluster along x.
__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
    __shared__ int hist[kSelectBins];
    __shared__ int warp_sums[2][kSelectWarps];
    __shared__ int s_counts[2];                  // this block's larger and equal keys
    __shared__ int s_digit, s_need;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    griddep_wait();
    griddep_launch_dependents();
    const int head = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    int n = kv_length(p.table.lengths[b], p.table.width, p.from.page_size, &bad);
    if (n > p.weights.width) {
        n = p.weights.width;
        bad = true;
    }
    if (bad && rank == 0 && threadIdx.x == 0) record_status(p.status, kStatusCache);
    const int k = min(n, p.keep), r = min(p.recent, k);
    const float *w = p.weights.base + b * p.weights.batch_stride + head * p.weights.head_stride;
    float *to_w = p.to_weights.base + b * p.to_weights.batch_stride + head * p.to_weights.head_stride;
    int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    if (head == 0 && rank == 0 && threadIdx.x == 0) p.to_lengths[b] = k;
    const int first = n - r, best = k - r;       // of the first `first` positions, `best` stay
    // What follows them: the recent ones, and -1 past k.
    for (int i = best + rank * kSelectThreads + threadIdx.x; i < p.keep; i += blocks * kSelectThreads) {
        const int j = first + i - best;
        kept[i] = i < k ? j : -1;
        to_w[i] = i < k ? w[j] : 0.0f;
    }
    if (best == first) {                         // nothing is evicted
        for (int j = rank * kSelectThreads + threadIdx.x; j < first; j += blocks * kSelectThreads) {
            kept[j] = j;
            to_w[j] = w[j];
        }
        return;                                  // every block of the cluster
    }
    if (best == 0) return;
    const int slice = (first + blocks - 1) / blocks, lo = min(first, rank * slice), hi = min(first, lo + slice);

    uint32_t prefix = 0;
    int need = best;                             // rank of the limit among the keys with this prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        const uint32_t mask = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
        for (int i = threadIdx.x; i < kSelectBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = lo + threadIdx.x; j < hi; j += kSelectThreads) {
            const uint32_t key = kv_weight_key(__float_as_uint(w[j]));
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
        }
        cluster.sync();
        // Thread i: bins bins-1-2i and bins-2-2i of all blocks; the first whose running sum from the top
        // reaches `need` holds the limit.
        int c[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int bin = bins - 1 - 2 * static_cast<int>(threadIdx.x) - e;
            if (bin >= 0)
                for (int q = 0; q < blocks; ++q) c[e] += cluster.map_shared_rank(hist, q)[bin];
        }
        int sum = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        if (lane == 31) warp_sums[0][warp] = sum;
        __syncthreads();
        int before = 0;
        for (int q = 0; q < warp; ++q) before += warp_sums[0][q];
        sum += before;
        const int above = sum - c[0] - c[1];
        if (above < need && sum >= need) {       // one thread
            const bool second = above + c[0] < need;
            s_digit = bins - 1 - 2 * static_cast<int>(threadIdx.x) - (second ? 1 : 0);
            s_need = need - above - (second ? c[0] : 0);
        }
        cluster.sync();                          // every block has read the histograms
        prefix |= static_cast<uint32_t>(s_digit) << shift;
        need = s_need;
    }

    // Each warp takes a contiguous part of the slice: counted, then written.
    const int part = ((hi - lo + kSelectWarps - 1) / kSelectWarps + 31) / 32 * 32;
    const int from = min(hi, lo + warp * part), to = min(hi, from + part);
    int larger = 0, equal = 0;
#pragma unroll 4
    for (int j = from + lane; j < to; j += 32) {
        const uint32_t key = kv_weight_key(__float_as_uint(w[j]));
        larger += key > prefix;
        equal += key == prefix;
    }
    larger = __reduce_add_sync(0xffffffffu, larger);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        warp_sums[0][warp] = larger;
        warp_sums[1][warp] = equal;
    }
    __syncthreads();
    if (warp < 2) {
        const int total = __reduce_add_sync(0xffffffffu, warp_sums[warp][lane]);
        if (lane == 0) s_counts[warp] = total;
    }
    cluster.sync();
    int larger_before = 0, equal_before = 0;
    for (int q = 0; q < rank; ++q) {
        const int *other = cluster.map_shared_rank(s_counts, q);
        larger_before += other[0];
        equal_before += other[1];
    }
    for (int q = 0; q < warp; ++q) {
        larger_before += warp_sums[0][q];
        equal_before += warp_sums[1][q];
    }
    cluster.sync();                              // no block leaves while its counts are read
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int j0 = from; j0 < to; j0 += 32) {
        const int j = j0 + lane;
        const float x = j < to ? w[j] : 0.0f;
        const uint32_t key = j < to ? kv_weight_key(__float_as_uint(x)) : 0u;
        const bool is_larger = j < to && key > prefix, is_equal = j < to && key == prefix;
        const unsigned ml = __ballot_sync(0xffffffffu, is_larger), me = __ballot_sync(0xffffffffu, is_equal);
        const int ties = equal_before + __popc(me & below);
        const int at = larger_before + __popc(ml & below) + min(ties, need);
        if (is_larger || (is_equal && ties < need)) {
            kept[at] = j;
            to_w[at] = x;
        }
        larger_before += __popc(ml);
        equal_before += __popc(me);
    }
}

// Copying the kept rows: as in kv_append_kernel a block first finds the places
// of a chunk of rows and then streams them, keys and values, all requested
// before the first is stored.  Grid: (chunks, heads, batch).
constexpr int kGatherThreads = 256;

template <bool kE4m3, int kLanes, int kUnroll>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const EvictParams p) {
    constexpr int kPass = kGatherThreads / kLanes, kRows = kPass * kUnroll;
    __shared__ long long s_src[kRows], s_dst[kRows];
    griddep_wait();
    griddep_launch_dependents();
    const int head = blockIdx.y, b = blockIdx.z;
    const int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    const int k = p.to_lengths[b];
    const int piece = threadIdx.x % kLanes, in_pass = threadIdx.x / kLanes;
    const bool inside = piece * 16 < p.from.row_bytes;
    for (int i0 = blockIdx.x * kRows; i0 < k; i0 += gridDim.x * kRows) {
        const int row = i0 + threadIdx.x;
        if (threadIdx.x < kRows) {
            long long src = 0, dst = -1;
            if (row < k) {
                int page, slot, to_page, to_slot;
                if (row >= static_cast<long long>(p.to_table.width) * p.to.page_size ||
                    !kv_row(p.table.pages + b * p.table.stride, kept[row], p.from.page_size, p.from.pages, &page,
                            &slot) ||
                    !kv_row(p.to_table.pages + b * p.to_table.stride, row, p.to.page_size, p.to.pages, &to_page,
                            &to_slot)) {
                    record_status(p.status, kStatusCache);
                } else {
                    src = kv_offset(p.from, page, slot, head);
                    dst = kv_offset(p.to, to_page, to_slot, head);
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
