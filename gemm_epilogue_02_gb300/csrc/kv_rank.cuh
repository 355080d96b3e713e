// The `best` largest of a list of 32-bit keys, in order of position, found by a
// block alone or by a cluster of blocks with a slice of the list each.
//
// The key of rank `best` is found 11 bits at a time (11 + 11 + 10) from
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
constexpr int kSelectMaxBlocks = 8;                   // of a cluster
constexpr int kSelectGroups = kSelectBins / 32;
static_assert(kSelectGroups == 64, "two groups a lane");

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

template <int kThreads>
struct RankShared {
    static constexpr int kWarps = kThreads / 32;
    __align__(16) int hist[3][kSelectBins];
    int groups[3][kSelectGroups];                // sums of 32 bins
    int warp_sums[2][kWarps];
    int counts[2], before[2];                    // larger and equal keys: this block's, those of the blocks before
    int digit, need, count;
};

template <int kThreads>
__device__ __forceinline__ void kv_rank_clear(RankShared<kThreads> &sh) {
    for (int i = threadIdx.x; i < 3 * kSelectBins; i += kThreads) (&sh.hist[0][0])[i] = 0;
}

// This block has `size` keys, key_at(0) .. key_at(size - 1); put(at, i) is called for each of its keys i that is among the
// `best`, at = 0 .. best - 1 its place among them.  Called by all threads of all blocks of a cluster (whatever their sizes),
// after a barrier that follows kv_rank_clear().
// kBy: by what the launch decides, by one block (whether it has a cluster or not), or by a cluster of two or more.
enum class RankBy { kLaunch, kBlock, kCluster };

template <RankBy kBy = RankBy::kLaunch, int kThreads, typename KeyAt, typename Put>
__device__ __forceinline__ void kv_rank(RankShared<kThreads> &sh, int size, int best, unsigned int *status, KeyAt key_at, Put put) {
    constexpr int kWarps = kThreads / 32;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = kBy == RankBy::kBlock ? 1 : static_cast<int>(cluster.num_blocks());
    const int rank = kBy == RankBy::kBlock ? 0 : static_cast<int>(cluster.block_rank());
    const bool alone = kBy != RankBy::kCluster && blocks == 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t prefix = 0, counted = ~0u;          // the limit, and its bits that count
    int need = best;                             // rank of the limit among the keys with this prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, digit_mask = pass == 2 ? 1023 : 2047;
        const uint32_t mask = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
#pragma unroll 4
        for (int i = threadIdx.x; i < size; i += kThreads) {
            const uint32_t key = key_at(i);
            if ((key & mask) == prefix) atomicAdd(&sh.hist[pass][(key >> shift) & digit_mask], 1);
        }
        __syncthreads();
        if (alone) {
            // Thread t has the bins from kSelectBins - 1 - t * kPer down; the one in which the running sum from the
            // top reaches `need` has the limit's digit.  (The last pass leaves the upper bins empty.)
            constexpr int kPer = kSelectBins / kThreads;
            const int low = kSelectBins - kPer - static_cast<int>(threadIdx.x) * kPer;
            int c[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                const int2 x = *reinterpret_cast<const int2 *>(&sh.hist[pass][low + i]);
                c[i] = x.x;
                c[i + 1] = x.y;
                sum += x.x + x.y;
            }
            const int upto = warp_scan(sum);
            if (lane == 31) sh.warp_sums[0][warp] = upto;
            __syncthreads();
            int above = upto - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sums[0][lane] : 0);
            if (above < need && above + sum >= need) {
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i) {
                    if (above < need && above + c[i] >= need) {
                        sh.digit = low + i;
                        sh.need = need - above;
                        sh.count = c[i];
                    }
                    above += c[i];
                }
            }
        } else {
#pragma unroll 2
            for (int i = warp; i < kSelectGroups; i += kWarps) {
                const int sum = __reduce_add_sync(0xffffffffu, sh.hist[pass][i * 32 + lane]);
                if (lane == 0) sh.groups[pass][i] = sum;
            }
            cluster.sync();
            if (warp == 0) {
                // Sums over the blocks, from the top: lane l has groups 63 - 2 l and 62 - 2 l, then bin 31 - l of
                // the group in which the running sum reaches `need`.
                int c0 = 0, c1 = 0, c = 0;
#pragma unroll
                for (int q = 0; q < kSelectMaxBlocks; ++q) {
                    const int *const other = cluster.map_shared_rank(sh.groups[pass], q < blocks ? q : rank);
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
                    const int x = cluster.map_shared_rank(sh.hist[pass], q < blocks ? q : rank)[group * 32 + 31 - lane];
                    c += q < blocks ? x : 0;
                }
                const int over = warp_scan(c) - c;
                if (over < left && over + c >= left) {
                    sh.digit = group * 32 + 31 - lane;
                    sh.need = left - over;
                }
            }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sh.digit) << shift;
        need = sh.need;
        // All keys that share these bits stay: the others do not matter.  (Only where no other block waits.)
        if (alone && need == sh.count) {
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
        sh.warp_sums[0][warp] = larger;
        sh.warp_sums[1][warp] = equal;
    }
    __syncthreads();
    const int a = lane < kWarps ? sh.warp_sums[0][lane] : 0, e = lane < kWarps ? sh.warp_sums[1][lane] : 0;
    int at_larger = __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
    int at_equal = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0);
    if (!alone) {
        if (warp == 0) {
            const int x = __reduce_add_sync(0xffffffffu, a), y = __reduce_add_sync(0xffffffffu, e);
            if (lane == 0) {
                sh.counts[0] = x;
                sh.counts[1] = y;
            }
        }
        cluster.sync();
        if (warp == 0) {
            const int *const other = cluster.map_shared_rank(sh.counts, min(lane, rank));
            const int x = lane < rank ? other[0] : 0, y = lane < rank ? other[1] : 0;
            const int larger_before = __reduce_add_sync(0xffffffffu, x), equal_before = __reduce_add_sync(0xffffffffu, y);
            if (lane == 0) {
                sh.before[0] = larger_before;
                sh.before[1] = equal_before;
            }
        }
        cluster.sync();                          // no block leaves while its counts are read
        at_larger += sh.before[0];
        at_equal += sh.before[1];
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
            if (TGEMM_CHECK(inside, kChkKvOutput, status) && inside) put(at, i);
        }
        at_larger += __popc(ml);
        at_equal += __popc(me);
    }
}

}  // namespace tgemm
