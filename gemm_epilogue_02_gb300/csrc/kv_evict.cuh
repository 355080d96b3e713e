// Eviction from the paged cache by accumulated attention weight.  Of sequence
// b's n = lengths[b] positions, each head keeps k = min(n, keep): the last
// r = min(recent, k), and of the n - r before them the k - r of largest weight
// (ties to the lowest position; a NaN counts as less than any number).  The kept
// rows are copied in order to positions 0 .. k - 1 of other pages, with their
// scales and weights.
//
// Two kernels: kv_select_kernel finds the positions (one block per sequence and
// head), kv_gather_kernel copies the rows.
//
// Selection: a weight becomes a 32-bit key of the same order; the key of rank
// k - r is found eight bits at a time from histograms of the keys that share
// the bits found so far; then every larger key is kept, and of the equal ones
// the first few in order of position.
#pragma once
#include "kv_cache.cuh"

namespace tgemm {

constexpr int kSelectThreads = 1024;
constexpr int kGatherThreads = 256;

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

// Inclusive sum over the block of one value per thread (kSelectThreads).
__device__ __forceinline__ int block_scan(int v, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    return v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelectThreads) kv_select_kernel(const EvictParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    griddep_wait();
    griddep_launch_dependents();
    const int head = blockIdx.x, b = blockIdx.y;
    bool bad = false;
    int n = kv_length(p.table.lengths[b], p.table.width, p.from.page_size, &bad);
    if (n > p.weights.width) {
        n = p.weights.width;
        bad = true;
    }
    if (bad && threadIdx.x == 0) record_status(p.status, kStatusCache);
    const int k = min(n, p.keep), r = min(p.recent, k);
    const float *w = p.weights.base + b * p.weights.batch_stride + head * p.weights.head_stride;
    float *to_w = p.to_weights.base + b * p.to_weights.batch_stride + head * p.to_weights.head_stride;
    int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    if (head == 0 && threadIdx.x == 0) p.to_lengths[b] = k;
    const int first = n - r;                  // positions that have to earn their place
    if (threadIdx.x == 0) {
        s_prefix = 0;
        s_need = k - r;
    }
    __syncthreads();
    if (k - r < first && k - r > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : ~0u << (shift + 8);
            for (int j = threadIdx.x; j < first; j += kSelectThreads) {
                const uint32_t key = kv_weight_key(__float_as_uint(w[j]));
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int need = s_need, d = 255;
                while (d > 0 && hist[d] < need) need -= hist[d--];
                s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
                s_need = need;
            }
            __syncthreads();
        }
    }
    const bool all = k - r >= first;          // nothing is evicted
    const uint32_t limit = s_prefix;
    const int equal = s_need;                 // how many of the keys equal to the limit stay
    int done = 0, ties = 0;
    for (int base = 0; base < first && done < k - r; base += kSelectThreads) {
        const int j = base + threadIdx.x;
        const uint32_t key = j < first ? kv_weight_key(__float_as_uint(w[j])) : 0u;
        const int tie = !all && j < first && key == limit;
        const int tie_rank = ties + block_scan(tie, warp_sums);
        const int tie_total = ties + warp_sums[31];
        const int take = j < first && (all || key > limit || (tie && tie_rank <= equal));
        const int rank = done + block_scan(take, warp_sums);
        const int total = done + warp_sums[31];
        if (take) {
            kept[rank - 1] = j;
            to_w[rank - 1] = w[j];
        }
        ties = tie_total;
        done = total;
        __syncthreads();
    }
    for (int i = threadIdx.x; i < p.keep - (k - r); i += kSelectThreads) {
        const int at = k - r + i;
        kept[at] = at < k ? first + i : -1;
        to_w[at] = at < k ? w[first + i] : 0.0f;
    }
}

// One warp per kept row pair.
template <bool kE4m3>
__global__ void __launch_bounds__(kGatherThreads) kv_gather_kernel(const EvictParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.y % p.from.heads, b = blockIdx.y / p.from.heads;
    const int *kept = p.kept + (static_cast<long long>(b) * p.from.heads + head) * p.keep;
    const int k = p.to_lengths[b];
    for (int i = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5); i < k;
         i += gridDim.x * (kGatherThreads / 32)) {
        int page, slot, to_page, to_slot;
        if (static_cast<long long>(i) >= static_cast<long long>(p.to_table.width) * p.to.page_size ||
            !kv_row(p.table.pages + b * p.table.stride, kept[i], p.from.page_size, p.from.pages, &page, &slot) ||
            !kv_row(p.to_table.pages + b * p.to_table.stride, i, p.to.page_size, p.to.pages, &to_page, &to_slot)) {
            if (lane == 0) record_status(p.status, kStatusCache);
            continue;
        }
        const long long src = kv_offset(p.from, page, slot, head), dst = kv_offset(p.to, to_page, to_slot, head);
        if (lane * 16 < p.from.row_bytes) {
            *reinterpret_cast<uint4 *>(p.to.k + dst + lane * 16) =
                *reinterpret_cast<const uint4 *>(p.from.k + src + lane * 16);
            *reinterpret_cast<uint4 *>(p.to.v + dst + lane * 16) =
                *reinterpret_cast<const uint4 *>(p.from.v + src + lane * 16);
        }
        if (kE4m3 && lane == 0) {
            const long long s = kv_scale_offset(p.from, page, slot, head);
            const long long d = kv_scale_offset(p.to, to_page, to_slot, head);
            p.to.k_scale[d] = p.from.k_scale[s];
            p.to.v_scale[d] = p.from.v_scale[s];
        }
    }
}

}  // namespace tgemm
