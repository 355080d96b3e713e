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
// the key of rank k - r is found 11 bits at a time (11 + 11 + 10) from
// histograms of the keys that share the bits found so far.  A block alone scans
// its bins; the blocks of a cluster add theirs up through distributed shared
// memory, whose reads are slow, so one warp of each reads the sums of 32 bins,
// finds the group and then reads its bins (131072 positions: 28 us; every block
// reading every bin 34 us).  Then every larger key is kept, and of the equal
// ones the first few in order of position.
#pragma once
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace tgemm {

constexpr int kSelectBins = 2048;
constexpr int kSelectMaxCached = 48 * 1024;           // keys of a slice in shared memory (192 KiB); of longer ones none
constexpr int kSelectMaxBlocks = 8;                   // of a cluster
constexpr int kSelectGroups = kSelectBins / 32;
static_assert(kSelectGroups == 64, "two groups a lane");

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

// A key of the same order as the weight: larger weight, larger key; -0 as +0;
// NaN below every number.
__host__ __device__ inline uint32_t kv_weight_key(uint32_t bits) {
    if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
    if (bits == 0x80000000u) bits = 0u;
    return (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
}

// Where a kept position goes among the `best`: after the larger keys before it and as many of the equal ones as are
// wanted; false where that is none of them (weights that another stream changes between the selection's passes leave
// it without a sound count).
__host__ __device__ inline bool kv_kept_place(int larger, int ties, int need, int best, int *at) {
    const unsigned place = static_cast<unsigned>(larger) + static_cast<unsigned>(ties < need ? ties : need);
    *at = static_cast<int>(place);
    return place < static_cast<unsigned>(best);              // a sum below 0 wraps to 2^31 or more
}

// Grid: (cluster size, heads, batch), a cluster along x.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 2) kv_select_kernel(const EvictParams p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ uint32_t keys[];
    __shared__ __align__(16) int hist[3][kSelectBins];
    __shared__ int groups[3][kSelectGroups];     // sums of 32 bins
    __shared__ int warp_sums[2][kWarps];
    __shared__ int s_counts[2], s_before[2];     // larger and equal keys: this block's, those of the blocks before
    __shared__ int s_digit, s_need, s_count, s_n;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int head = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < 3 * kSelectBins; i += kThreads) (&hist[0][0])[i] = 0;
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
        if (blocks == 1) return;
        // The blocks of a cluster go on together to every barrier, whatever length each of them has read.
    }
    __syncthreads();                             // the keys are there

    uint32_t prefix = 0, counted = ~0u;          // the limit, and its bits that count
    int need = best;                             // rank of the limit among the keys with this prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digit_mask = pass == 2 ? 1023 : 2047;
        const uint32_t mask = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
#pragma unroll 4
        for (int i = threadIdx.x; i < size; i += kThreads) {
            const uint32_t key = key_at(i);
            if ((key & mask) == prefix) atomicAdd(&hist[pass][(key >> shift) & digit_mask], 1);
        }
        __syncthreads();
        if (blocks == 1) {
            // Thread t has the bins from kSelectBins - 1 - t * kPer down; the one in which the running sum from the
            // top reaches `need` has the limit's digit.  (The last pass leaves the upper bins empty.)
            constexpr int kPer = kSelectBins / kThreads;
            const int low = kSelectBins - kPer - static_cast<int>(threadIdx.x) * kPer;
            int c[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const int2 x = *reinterpret_cast<const int2 *>(&hist[pass][low + i]);
                c[i] = x.x;
                c[i + 1] = x.y;
                sum += x.x + x.y;
            }
            const int upto = warp_scan(sum);
            if (lane == 31) warp_sums[0][warp] = upto;
            __syncthreads();
            int above = upto - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[0][lane] : 0);
            if (above < need && above + sum >= need) {
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i) {
                    if (above < need && above + c[i] >= need) {
                        s_digit = low + i;
                        s_need = need - above;
                        s_count = c[i];
                    }
                    above += c[i];
                }
            }
        } else {
#pragma unroll 2
            for (int i = warp; i < kSelectGroups; i += kWarps) {
                const int sum = __reduce_add_sync(0xffffffffu, hist[pass][i * 32 + lane]);
                if (lane == 0) groups[pass][i] = sum;
            }
            cluster.sync();
            if (warp == 0) {
                // Sums over the blocks, from the top: lane l has groups 63 - 2 l and 62 - 2 l, then bin 31 - l of
                // the group in which the running sum reaches `need`.
                int c0 = 0, c1 = 0, c = 0;
#pragma unroll
                for (int q = 0; q < kSelectMaxBlocks; ++q) {
                    const int *const other = cluster.map_shared_rank(groups[pass], q < blocks ? q : rank);
                    const int x0 = other[63 - 2 * lane], x1 = other[62 - 2 * lane];
                    c0 += q < blocks ? x0 : 0;
                    c1 += q < blocks ? x1 : 0;
                }
                const int above = warp_scan(c0 + c1) - c0 - c1;
                const unsigned found = __ballot_sync(0xffffffffu, above < need && above + c0 + c1 >= need);
                const int owner = __ffs(found) - 1;
                const bool second = above + c0 < need;
                const int group = __shfl_sync(0xffffffffu, 63 - 2 * lane - (second ? 1 : 0), owner);
                const int left = need - __shfl_sync(0xffffffffu, above + (second ? c0 : 0), owner);
#pragma unroll
                for (int q = 0; q < kSelectMaxBlocks; ++q) {
                    const int x = cluster.map_shared_rank(hist[pass], q < blocks ? q : rank)[group * 32 + 31 - lane];
                    c += q < blocks ? x : 0;
                }
                const int over = warp_scan(c) - c;
                if (over < left && over + c >= left) {
                    s_digit = group * 32 + 31 - lane;
                    s_need = left - over;
                }
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_digit) << shift;
        need = s_need;
        // All keys that share these bits stay: the others do not matter.  (Only where no other block waits.)
        if (blocks == 1 && need == s_count) {
            counted = ~0u << shift;
            break;
        }
    }

    // Each warp has a contiguous part of the slice: its larger and equal keys are counted, then written after
    // those of the warps and blocks before.
    const int part = ((size + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int from = min(size, warp * part), to = min(size, from + part);
    int larger = 0, equal = 0;
#pragma unroll 4
    for (int i = from + lane; i < to; i += 32) {
        const uint32_t key = key_at(i) & counted;
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
    const int a = lane < kWarps ? warp_sums[0][lane] : 0, e = lane < kWarps ? warp_sums[1][lane] : 0;
    int at_larger = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
    int at_equal = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
    if (blocks > 1) {
        if (warp == 0) {
            const int x = __reduce_add_sync(0xffffffffu, a), y = __reduce_add_sync(0xffffffffu, e);
            if (lane == 0) {
                s_counts[0] = x;
                s_counts[1] = y;
            }
        }
        cluster.sync();
        if (warp == 0) {
            const int *const other = cluster.map_shared_rank(s_counts, min(lane, rank));
            const int x = lane < rank ? other[0] : 0, y = lane < rank ? other[1] : 0;
            const int larger_before = __reduce_add_sync(0xffffffffu, x), equal_before = __reduce_add_sync(0xffffffffu, y);
            if (lane == 0) {
                s_before[0] = larger_before;
                s_before[1] = equal_before;
            }
        }
        cluster.sync();                          // no block leaves while its counts are read
        at_larger += s_before[0];
        at_equal += s_before[1];
    }
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < to ? key_at(i) & counted : 0u;
        const bool is_larger = i < to && key > prefix, is_equal = i < to && key == prefix;
        const unsigned ml = __ballot_sync(0xffffffffu, is_larger), me = __ballot_sync(0xffffffffu, is_equal);
        const int ties = at_equal + __popc(me & below);
        if (is_larger || (is_equal && ties < need)) {
            int at;
            const bool inside = kv_kept_place(at_larger + __popc(ml & below), ties, need, best, &at);
            if (TGEMM_CHECK(inside, kChkKvOutput, p.status) && inside) {
                kept[at] = lo + i;
                to_w[at] = mine[i];
            }
        }
        at_larger += __popc(ml);
        at_equal += __popc(me);
    }
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
