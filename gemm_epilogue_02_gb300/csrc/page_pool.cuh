// The pages of the paged cache as a resource: uses[page] counts the sequences
// that hold a page, 0: free.
//
//   page_take_kernel     gives sequences the lowest free pages, in their order: the
//                      pages that new tokens need (grow), or the page for the rows
//                      of a child's last, partly filled page (fork)
//   page_fork_kernel     the children's lists (their parents' full pages, counted
//                      once more) and the rows of those last pages;
//                      page_fork_few_kernel does both
//   page_free_kernel     counts a sequence's pages once less
//   page_plan_kernel     compaction: which pages move where, and the new counts
//   page_move_kernel     moves them, and translates the lists;
//                      page_compact_few_kernel does both
//
// The counts are whole numbers, and which page goes where follows from order
// alone, so nothing depends on how the work is split.  The planning kernels read
// 4 bytes a page and are bound by latency; the copies read and write each row
// once (400 MB moved within a pool of 1.6 GB: 134 us, 6.0 TB/s of both).  Where
// there is little to copy, a launch costs more than it: a cluster of eight blocks
// then plans and copies in one (8 children of two prompts, with freeing and growing:
// 15.5 us as called, with a launch more 18; a pool of 140 pages compacted: 7.9, 9.7).
#pragma once
#include "page_bounds.cuh"
#include "kv_cache.cuh"

namespace tgemm {

// Lists and lengths that a kernel writes.
struct KvLists {
    int *pages;                    // [batch, stride], `width` columns used
    int *lengths;
    long long stride;
    int width, batch;
};

struct PagesParams {
    KvView cache;
    KvTable table;                 // fork: the parents; compact: what there is
    KvLists to;                    // what is written
    int *uses;
    const int *parents;            // fork: [to.batch]
    const int *fresh;              // grow: new tokens, null: one each
    unsigned int *status;
};

constexpr int kTakeThreads = 1024;
constexpr int kTakeDeep = 8;                               // pages that a thread looks at in a round
constexpr int kTakeRound = kTakeThreads * kTakeDeep;

// Inclusive sum over a block of 1024, with its total; `sums` has 33 entries.  Ends with a barrier.
__device__ __forceinline__ int block_scan(int x, int *sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int upto = warp_scan(x);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        const int s = sums[lane];
        const int before = warp_scan(s);
        sums[lane] = before - s;
        if (lane == 31) sums[32] = before;
    }
    __syncthreads();
    const int out = upto + sums[warp];
    *total = sums[32];
    __syncthreads();
    return out;
}

// Pages that n positions take.
__host__ __device__ inline int kv_pages_of(int n, int page_size) { return n / page_size + (n % page_size > 0 ? 1 : 0); }

// A parent's length, cut to what its list holds (*bad); 0 for a bad parent, or where the child's list has no room for it.
__host__ __device__ inline int fork_length(const int *lengths, int batch, int parent, int width, int page_size, int to_width, bool *bad) {
    if (parent == -1) return 0;
    if (parent < 0 || parent >= batch) {
        *bad = true;
        return 0;
    }
    const int n = kv_length(lengths[parent], width, page_size, bad);
    if (kv_pages_of(n, page_size) > to_width) {
        *bad = true;
        return 0;
    }
    return n;
}

// What a child of `parent` takes over: its positions, or none where that cannot be done.
__device__ __forceinline__ int fork_positions(const PagesParams &p, int parent, bool *bad) {
    const int n = fork_length(p.table.lengths, p.table.batch, parent, p.table.width, p.cache.page_size, p.to.width, bad);
    return *bad ? 0 : n;                   // (of a list that is not all its parent's, which entries are is not known)
}

// By one block of kTakeThreads.
template <bool kFork>
__device__ __forceinline__ void take_pages(const PagesParams &p) {
    constexpr int kWarps = kTakeThreads / 32;
    __shared__ int s_free[kTakeRound];                     // free pages found, in order
    __shared__ int s_end[kTakeThreads + 1];                // pages wanted by the sequences of this round, summed up
    __shared__ int s_cnt[kTakeDeep * kWarps];
    __shared__ int s_sums[33];
    __shared__ int s_found;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, size = p.cache.page_size;
    long long pos = 0;                                     // pages looked at
    int at = 0, have = 0;                                  // of s_free
    for (int b0 = 0; b0 < p.to.batch; b0 += kTakeThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int n = 0, more = 0, first = 0, need = 0;          // positions there, new ones; list index of the first new page
        bool bad = false;
        if (b < p.to.batch) {
            if (kFork) {
                n = fork_positions(p, p.parents[b], &bad);
                first = n / size;
                need = n % size > 0 ? 1 : 0;
            } else {
                n = kv_length(p.to.lengths[b], p.to.width, size, &bad);
                more = p.fresh ? p.fresh[b] : 1;
                if (bad || more < 0 || more > static_cast<long long>(p.to.width) * size - n) {
                    bad = true;
                    more = 0;
                }
                first = kv_pages_of(n, size);
                need = kv_pages_of(n + more, size) - first;
            }
        }
        int wanted;
        const int end = block_scan(need, s_sums, &wanted);
        s_end[threadIdx.x + 1] = end;
        if (threadIdx.x == 0) s_end[0] = 0;
        __syncthreads();
        int taken = 0;
        while (taken < wanted) {
            if (have == 0) {
                if (pos >= p.cache.pages) break;
                // The next pages: thread t looks at page pos + i * 1024 + t, so that order is by i, then warp, then lane.
                int u[kTakeDeep];
#pragma unroll
                for (int i = 0; i < kTakeDeep; ++i) {
                    const long long page = pos + i * kTakeThreads + threadIdx.x;
                    u[i] = page < p.cache.pages ? p.uses[page] : 1;
                }
#pragma unroll
                for (int i = 0; i < kTakeDeep; ++i) {
                    const unsigned m = __ballot_sync(0xffffffffu, u[i] == 0);
                    if (lane == 0) s_cnt[i * kWarps + warp] = __popc(m);
                }
                __syncthreads();
                if (warp == 0) {
                    int c[kTakeDeep], sum = 0;
#pragma unroll
                    for (int i = 0; i < kTakeDeep; ++i) {
                        c[i] = s_cnt[lane * kTakeDeep + i];
                        sum += c[i];
                    }
                    int before = warp_scan(sum) - sum;
                    if (lane == 31) s_found = before + sum;
#pragma unroll
                    for (int i = 0; i < kTakeDeep; ++i) {
                        s_cnt[lane * kTakeDeep + i] = before;
                        before += c[i];
                    }
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kTakeDeep; ++i) {
                    const unsigned m = __ballot_sync(0xffffffffu, u[i] == 0);
                    if (u[i] == 0)
                        s_free[s_cnt[i * kWarps + warp] + __popc(m & ((1u << lane) - 1u))] =
                            static_cast<int>(pos + i * kTakeThreads + threadIdx.x);
                }
                have = s_found;
                at = 0;
                pos += kTakeRound;
                __syncthreads();
                if (have == 0) continue;
            }
            const int m = min(wanted - taken, have);
            for (int j = threadIdx.x; j < m; j += kTakeThreads) {
                const int rank = taken + j, page = s_free[at + j];
                int lo = 0, hi = kTakeThreads;             // s_end[lo] <= rank < s_end[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_end[mid] <= rank) lo = mid;
                    else hi = mid;
                }
                // The list index is the owner's `first` plus the page's place among those that it wants.
                int f;
                if (kFork) {
                    bool ignore = false;
                    f = fork_positions(p, p.parents[b0 + lo], &ignore) / size;
                } else {
                    bool ignore = false;
                    f = kv_pages_of(kv_length(p.to.lengths[b0 + lo], p.to.width, size, &ignore), size) + rank - s_end[lo];
                }
                if (f < p.to.width) {                      // (unless another stream changes a length meanwhile)
                    p.to.pages[(b0 + lo) * p.to.stride + f] = page;
                    p.uses[page] = 1;
                }
            }
            taken += m;
            at += m;
            have -= m;
            __syncthreads();
        }
        if (b < p.to.batch) {
            const bool fits = need == 0 || end <= taken;
            if (!fits) {
                // No page left: what a sequence has taken of those that it wants goes back.
                bad = true;
                for (int i = 0; i < taken - (end - need); ++i) p.uses[p.to.pages[b * p.to.stride + first + i]] = 0;
            }
            if (kFork) p.to.lengths[b] = fits ? n : n / size * size;
            else if (fits && more > 0) p.to.lengths[b] = n + more;
            if (bad) record_status(p.status, kStatusCache);
        }
        __syncthreads();
    }
}

template <bool kFork>
__global__ void __launch_bounds__(kTakeThreads, 1) page_take_kernel(const PagesParams p) {
    griddep_wait();
    griddep_launch_dependents();
    take_pages<kFork>(p);
}

// ---------------------------------------------------------------- copies of rows
constexpr int kPageThreads = 256;

// Row r of a page, in the order in which rows lie in memory.
__device__ __forceinline__ void page_row(const KvView &c, int r, bool slots_first, int *slot, int *head) {
    const int by = slots_first ? c.page_size : c.heads, q = r / by, rest = r - q * by;
    *slot = slots_first ? rest : q;
    *head = slots_first ? q : rest;
}

// The list of child c and the rows of its last page, by block `chunk` of `chunks`.
template <int kThreads, int kLanes>
__device__ __forceinline__ void fork_child(const PagesParams &p, int c, int chunk, int chunks) {
    constexpr int kPass = kThreads / kLanes, kUnroll = 4;
    const int size = p.cache.page_size, parent = p.parents[c];
    bool bad = false;
    const int n = fork_positions(p, parent, &bad);
    const int full = n / size, rest = p.to.lengths[c] > full * size ? n - full * size : 0;
    if (n == 0) return;
    const int *const list = p.table.pages + parent * p.table.stride;
    int *const to = p.to.pages + c * p.to.stride;
    for (int i = chunk * kThreads + threadIdx.x; i < full; i += chunks * kThreads) {
        const int page = list[i];
        to[i] = page;
        if (page >= 0 && page < p.cache.pages) atomicAdd(p.uses + page, 1);
        else record_status(p.status, kStatusCache);
    }
    if (rest == 0) return;
    const int src = list[full], dst = to[full];
    if (src < 0 || src >= p.cache.pages || dst < 0 || dst >= p.cache.pages) {
        if (threadIdx.x == 0) record_status(p.status, kStatusCache);
        return;
    }
    const int rows = rest * p.cache.heads, piece = threadIdx.x % kLanes, in_pass = threadIdx.x / kLanes;
    const bool inside = piece * 16 < p.cache.row_bytes;
    const long long from_page = src * p.cache.page_stride, to_page = dst * p.cache.page_stride;
    for (int r0 = chunk * kPass * kUnroll; r0 < rows; r0 += chunks * kPass * kUnroll) {
        uint4 x[kUnroll][2];
        long long o[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * kPass + in_pass;
            o[u] = -1;
            if (r < rows && inside) {
                const int slot = r / p.cache.heads, head = r - slot * p.cache.heads;
                o[u] = slot * p.cache.slot_stride + head * p.cache.head_stride + piece * 16;
                x[u][0] = *reinterpret_cast<const uint4 *>(p.cache.k + from_page + o[u]);
                x[u][1] = *reinterpret_cast<const uint4 *>(p.cache.v + from_page + o[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (o[u] >= 0 && TGEMM_CHECK(to_page + o[u] + 16 <= p.cache.dbg_bytes, kChkKvRow, p.status)) {
                *reinterpret_cast<uint4 *>(p.cache.k + to_page + o[u]) = x[u][0];
                *reinterpret_cast<uint4 *>(p.cache.v + to_page + o[u]) = x[u][1];
            }
    }
    if (p.cache.k_scale)
        for (int r = chunk * kThreads + threadIdx.x; r < rows; r += chunks * kThreads) {
            const int slot = r / p.cache.heads, head = r - slot * p.cache.heads;
            const long long a = kv_scale_offset(p.cache, src, slot, head), z = kv_scale_offset(p.cache, dst, slot, head);
            p.cache.k_scale[z] = p.cache.k_scale[a];
            p.cache.v_scale[z] = p.cache.v_scale[a];
        }
}

// Grid: (chunks, children).
template <int kLanes>
__global__ void __launch_bounds__(kPageThreads) page_fork_kernel(const PagesParams p) {
    griddep_wait();
    griddep_launch_dependents();
    fork_child<kPageThreads, kLanes>(p, blockIdx.y, blockIdx.x, gridDim.x);
}

// Both in one launch, for little to copy: the first block of a cluster finds the pages, then all copy.
constexpr int kForkBlocks = 8;

template <int kLanes>
__global__ void __launch_bounds__(kTakeThreads, 1) page_fork_few_kernel(const PagesParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int rank = static_cast<int>(cluster_ctarank());
    if (rank == 0) take_pages<true>(p);
    cluster_sync();                                        // releases what the first block has written, and acquires it
    for (int c = rank; c < p.to.batch; c += kForkBlocks) fork_child<kTakeThreads, kLanes>(p, c, 0, 1);
}

// One block a sequence: its pages' counts go down, its length to 0.
__global__ void __launch_bounds__(kPageThreads) page_free_kernel(const PagesParams p) {
    __shared__ int s_n;
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x;
    if (threadIdx.x == 0) {
        bool bad = false;
        const int n = kv_length(p.to.lengths[b], p.to.width, p.cache.page_size, &bad);
        s_n = bad ? 0 : n;                                 // which pages such a sequence holds is not known: it stays
        if (bad) record_status(p.status, kStatusCache);
        else p.to.lengths[b] = 0;
    }
    __syncthreads();
    const int count = kv_pages_of(s_n, p.cache.page_size);
    for (int i = threadIdx.x; i < count; i += kPageThreads) {
        const int page = p.to.pages[b * p.to.stride + i];
        if (page < 0 || page >= p.cache.pages) {
            record_status(p.status, kStatusCache);
        } else if (atomicSub(p.uses + page, 1) <= 0) {     // it was free already
            atomicAdd(p.uses + page, 1);
            record_status(p.status, kStatusCache);
        }
    }
}

// ---------------------------------------------------------------- compaction
struct CompactParams {
    KvView cache;
    KvTable table;
    KvLists to;
    KvBounds bounds;               // base null: none
    const int *uses;
    int *to_uses, *in_use;
    int *head;                     // workspace: pages in use, pages that move
    int *below, *above, *map;      // free pages below their number; pages in use above; a page's place among these, -1: none
    bool slots_first;
    unsigned int *status;
};

// By one block of kTakeThreads.  Pages come in rounds: thread t has pages kDeep t ..
// of a round, which are read once (again where there are several rounds).
template <int kDeep>
__device__ __forceinline__ void plan_moves(const CompactParams &p) {
    constexpr int kRound = kTakeThreads * kDeep;
    __shared__ int s_sums[33];
    const int pages = static_cast<int>(p.cache.pages), rounds = (pages + kRound - 1) / kRound;
    int u[kDeep];
    auto read = [&](int round) {
        const int first = round * kRound + static_cast<int>(threadIdx.x) * kDeep;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) u[i] = first + i < pages ? p.uses[first + i] : 0;
        return first;
    };
    int mine = 0, total;
    for (int r = 0; r < rounds; ++r) {
        read(r);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) mine += u[i] > 0;
    }
    block_scan(mine, s_sums, &total);
    int holes = 0, moved = 0;
    for (int r = 0; r < rounds; ++r) {
        const int first = rounds == 1 ? static_cast<int>(threadIdx.x) * kDeep : read(r);
        // Both at once: a round has 8192 of either at most.
        int both = 0, n;
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const bool used = u[i] > 0, in = first + i < pages;
            both += (in && first + i < total && !used ? 1 : 0) | (first + i >= total && used ? 1 << 16 : 0);
        }
        const int before = block_scan(both, s_sums, &n) - both;
        int hole = holes + (before & 0xFFFF), move = moved + (before >> 16);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int page = first + i;
            if (page < total) {
                if (page < pages) {
                    if (u[i] > 0) p.to_uses[page] = u[i];
                    else p.below[hole++] = page;
                }
            } else if (page < pages) {
                p.map[page] = u[i] > 0 ? move : -1;
                if (u[i] > 0) p.above[move++] = page;
            }
        }
        holes += n & 0xFFFF;
        moved += n >> 16;
    }
    moved = min(moved, holes);                             // the same, unless another stream changes a count meanwhile
    __syncthreads();
    for (int i = threadIdx.x; i < moved; i += kTakeThreads) p.to_uses[p.below[i]] = p.uses[p.above[i]];
    __syncthreads();                                       // to_uses may be uses
    for (int i = total + threadIdx.x; i < pages; i += kTakeThreads) p.to_uses[i] = 0;
    if (threadIdx.x == 0) {
        p.head[0] = total;
        p.head[1] = moved;
        *p.in_use = total;
    }
}

template <int kDeep>
__global__ void __launch_bounds__(kTakeThreads, 1) page_plan_kernel(const CompactParams p) {
    griddep_wait();
    griddep_launch_dependents();
    plan_moves<kDeep>(p);
}

// The pages that move and the lists, by block `block` of `blocks`.
template <int kThreads, int kLanes>
__device__ __forceinline__ void move_pages(const CompactParams &p, int block, int blocks) {
    constexpr int kPass = kThreads / kLanes, kUnroll = 4, kRows = kPass * kUnroll;
    const int total = p.head[0], moved = p.head[1];
    const int rows = p.cache.page_size * p.cache.heads, chunks = (rows + kRows - 1) / kRows;
    const int piece = threadIdx.x % kLanes, in_pass = threadIdx.x / kLanes;
    const bool inside = piece * 16 < p.cache.row_bytes;
    for (long long unit = block; unit < static_cast<long long>(moved) * chunks; unit += blocks) {
        const int m = static_cast<int>(unit / chunks), r0 = static_cast<int>(unit - static_cast<long long>(m) * chunks) * kRows;
        const int src = p.above[m], dst = p.below[m];
        const long long from_page = src * p.cache.page_stride, to_page = dst * p.cache.page_stride;
        uint4 x[kUnroll][2];
        long long o[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * kPass + in_pass;
            o[u] = -1;
            if (r < rows && inside) {
                int slot, head;
                page_row(p.cache, r, p.slots_first, &slot, &head);
                o[u] = slot * p.cache.slot_stride + head * p.cache.head_stride + piece * 16;
                x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(p.cache.k + from_page + o[u]));
                x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(p.cache.v + from_page + o[u]));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (o[u] >= 0 && TGEMM_CHECK(to_page + o[u] + 16 <= p.cache.dbg_bytes, kChkKvRow, p.status)) {
                __stcs(reinterpret_cast<uint4 *>(p.cache.k + to_page + o[u]), x[u][0]);
                __stcs(reinterpret_cast<uint4 *>(p.cache.v + to_page + o[u]), x[u][1]);
            }
        if (p.cache.k_scale)
            for (int r = r0 + threadIdx.x; r < min(rows, r0 + kRows); r += kThreads) {
                int slot, head;
                page_row(p.cache, r, p.slots_first, &slot, &head);
                const long long a = kv_scale_offset(p.cache, src, slot, head), z = kv_scale_offset(p.cache, dst, slot, head);
                p.cache.k_scale[z] = p.cache.k_scale[a];
                p.cache.v_scale[z] = p.cache.v_scale[a];
            }
        if (p.bounds.base && r0 == 0) {
            const int words = p.cache.heads * p.cache.dim / 8;         // 16 bytes each
            const uint4 *const a = reinterpret_cast<const uint4 *>(p.bounds.base) + static_cast<long long>(src) * words;
            uint4 *const z = reinterpret_cast<uint4 *>(p.bounds.base) + static_cast<long long>(dst) * words;
            for (int i = threadIdx.x; i < words; i += kThreads) z[i] = a[i];
            for (int i = threadIdx.x; i < p.cache.heads; i += kThreads)
                p.bounds.scale[static_cast<long long>(dst) * p.cache.heads + i] = p.bounds.scale[static_cast<long long>(src) * p.cache.heads + i];
        }
    }
    // The lists.
    for (int b = block; b < p.table.batch; b += blocks) {
        bool bad = false;
        const int count = kv_pages_of(kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad), p.cache.page_size);
        for (int i = threadIdx.x; i < count; i += kThreads) {
            int page = p.table.pages[b * p.table.stride + i];
            if (page < 0 || page >= p.cache.pages) bad = true;
            else if (page >= total) {
                const int k = p.map[page];
                if (k >= 0 && k < moved) page = p.below[k];
                else bad = true;                           // nothing counts it
            }
            p.to.pages[b * p.to.stride + i] = page;
        }
        if (bad) record_status(p.status, kStatusCache);
    }
}

template <int kLanes>
__global__ void __launch_bounds__(kPageThreads) page_move_kernel(const CompactParams p) {
    griddep_wait();
    griddep_launch_dependents();
    move_pages<kPageThreads, kLanes>(p, blockIdx.x, gridDim.x);
}

// Both in one launch, for a small pool.
template <int kLanes>
__global__ void __launch_bounds__(kTakeThreads, 1) page_compact_few_kernel(const CompactParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int rank = static_cast<int>(cluster_ctarank());
    if (rank == 0) {
        if (p.cache.pages <= kTakeThreads) plan_moves<1>(p);
        else plan_moves<kTakeDeep>(p);
    }
    cluster_sync();                                        // releases what the first block has written, and acquires it
    move_pages<kTakeThreads, kLanes>(p, rank, kForkBlocks);
}

}  // namespace tgemm
