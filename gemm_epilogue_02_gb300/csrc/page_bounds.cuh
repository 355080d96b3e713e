// Bounds of the keys on a page, and the choice of pages by them.
//
// page_bounds_kernel keeps, for each page and key head, every channel's least and
// largest key in 8 bits: with s the least power of two (2^-100 at least) such
// that no key exceeds 127 s, lo = floor(min / s), hi = ceil(max / s).  A power of
// two makes every step exact: what the bounds are does not depend on how they
// were computed.
//
// page_choose_kernel bounds the product of a query with any key of a page: q in
// whole numbers of a power of two found in the same way, sum_d max(q_d lo_d, q_d
// hi_d), times both powers; a page's score is the largest over the group's
// heads.  The sum is that of q+ hi + q- lo (q+ = max(q, 0), q- = min(q, 0)), two
// products of 8-bit whole numbers with pages as rows and heads as columns.  A
// sum is below 2^23, so the score is exact in fp32, and the same pages are
// chosen however the work is split.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"
#include "kv_rank.cuh"

namespace tgemm {

// The bounds [pages, heads, 2, dim] (lo, then hi) and their scales [pages, heads].
struct KvBounds {
    signed char *base;
    float *scale;
    long long dbg_rows;            // debug builds: pages * heads
};

// The least power of two s >= 2^-100 with top <= 127 s; top is finite.
__host__ __device__ inline float kv_bounds_scale(float top) {
    uint32_t bits;
#ifdef __CUDA_ARCH__
    bits = __float_as_uint(top);
#else
    __builtin_memcpy(&bits, &top, 4);
#endif
    constexpr float kLeast = 0x1p-100f;
    if (!(top > 127.0f * kLeast)) return kLeast;
    // top = f 2^x, 1 <= f < 2: 2^(x - 6) if f <= 127 / 64, else 2^(x - 5)
    const uint32_t e = (bits >> 23) - ((bits & 0x7FFFFFu) <= 0x7E0000u ? 6u : 5u);
    float s;
#ifdef __CUDA_ARCH__
    s = __uint_as_float(e << 23);
#else
    const uint32_t out = e << 23;
    __builtin_memcpy(&s, &out, 4);
#endif
    return s;
}

// 1 / s for a power of two that kv_bounds_scale() returns.
__host__ __device__ inline float kv_bounds_inverse(float s) {
    return 1.0f / s;
}

// NaN to 0, infinities to the largest finite numbers.
__device__ __forceinline__ float kv_finite(float x) {
    return x != x ? 0.0f : fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
}

// ---------------------------------------------------------------- bounds
struct BoundsParams {
    KvView cache;                  // its keys
    KvTable table;
    KvBounds bounds;
    const int *starts;             // null: one new token each
    unsigned int *status;
};

constexpr int kBoundsThreads = 256, kBoundsCtas = 4;     // per SM

// Pages of sequence b that its newest tokens complete: [*from, return).
__host__ __device__ inline int kv_completed(int n, long long fresh, int page_size, int *from) {
    long long before = n - fresh;
    if (before < 0) before = 0;
    if (before > n) before = n;
    *from = static_cast<int>(before / page_size);
    return n / page_size;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
    if (kBf16) {
        const __nv_bfloat162 m = __hmin2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    const __half2 m = __hmin2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t most_pair(uint32_t a, uint32_t b) {
    if (kBf16) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <bool kBf16>
__device__ __forceinline__ float2 bounds_widen(uint32_t w) {
    if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// A warp has one page and head at a time; kLanes lanes hold a row in 16-byte
// pieces, 32 / kLanes rows at once.  Neighbouring warps have neighbouring heads
// of a page.
template <bool kBf16, bool kE4m3, int kLanes>
__global__ void __launch_bounds__(kBoundsThreads, kBoundsCtas) page_bounds_kernel(const BoundsParams p) {
    constexpr int kWarps = kBoundsThreads / 32, kRows = 32 / kLanes, kPer = kE4m3 ? 16 : 8, kUnroll = 8;
    __shared__ int s_end[kBoundsThreads + 1];      // pages of the sequences of this round, summed up
    __shared__ int s_from[kBoundsThreads];
    __shared__ int s_sum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = lane % kLanes, row = lane / kLanes;
    const bool inside = piece * 16 < p.cache.row_bytes;
    griddep_wait();
    griddep_launch_dependents();
    const long long warps = static_cast<long long>(gridDim.x) * kWarps, me = static_cast<long long>(blockIdx.x) * kWarps + warp;
    long long base = 0;                            // items of the rounds before
    for (int b0 = 0; b0 < p.table.batch; b0 += kBoundsThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        int mine = 0, from = 0;
        if (b < p.table.batch) {
            bool bad = false;
            const int n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
            const long long fresh = p.starts ? static_cast<long long>(p.starts[b + 1]) - p.starts[b] : 1;
            if (fresh < 0 || fresh > n + (p.starts ? 0 : 1)) bad = true;
            const int to = kv_completed(n, fresh, p.cache.page_size, &from);
            mine = to - from;
            if (bad && blockIdx.x == 0) record_status(p.status, kStatusCache);
        }
        const int upto = warp_scan(mine);
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
        const int before = __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
        s_end[threadIdx.x + 1] = before + upto;
        if (threadIdx.x == 0) s_end[0] = 0;
        s_from[threadIdx.x] = from;
        __syncthreads();
        const long long items = static_cast<long long>(s_end[kBoundsThreads]) * p.cache.heads;
        // Warp `me` has the items i with (base + i) % warps == me.
        for (long long i = (me + warps - base % warps) % warps; i < items; i += warps) {
            const int at = static_cast<int>(i / p.cache.heads), head = static_cast<int>(i - static_cast<long long>(at) * p.cache.heads);
            int lo = 0, hi = kBoundsThreads;       // s_end[lo] <= at < s_end[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_end[mid] <= at) lo = mid;
                else hi = mid;
            }
            const int page = p.table.pages[(b0 + lo) * p.table.stride + s_from[lo] + at - s_end[lo]];
            if (page < 0 || page >= p.cache.pages) {
                if (lane == 0) record_status(p.status, kStatusCache);
                continue;
            }
            const unsigned char *const keys = p.cache.k + kv_offset(p.cache, page, 0, head) + (inside ? piece * 16 : 0);
            const float *const scales = kE4m3 ? p.cache.k_scale + kv_scale_offset(p.cache, page, 0, head) : nullptr;
            float least[kPer], most[kPer];
            if constexpr (!kE4m3) {
                constexpr uint32_t kNan = 0x7FFF7FFFu;      // gives way to any number
                uint32_t a[4] = {kNan, kNan, kNan, kNan}, z[4] = {kNan, kNan, kNan, kNan};
                for (int s0 = row; s0 < p.cache.page_size; s0 += kRows * kUnroll) {
                    uint4 x[kUnroll];
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const int slot = s0 + u * kRows;
                        x[u] = make_uint4(kNan, kNan, kNan, kNan);
                        if (inside && slot < p.cache.page_size)
                            x[u] = __ldcs(reinterpret_cast<const uint4 *>(keys + slot * p.cache.slot_stride));
                    }
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[j] = min_pair<kBf16>(a[j], w[j]);
                            z[j] = most_pair<kBf16>(z[j], w[j]);
                        }
                    }
                }
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[j] = min_pair<kBf16>(a[j], __shfl_xor_sync(0xffffffffu, a[j], o));
                        z[j] = most_pair<kBf16>(z[j], __shfl_xor_sync(0xffffffffu, z[j], o));
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = bounds_widen<kBf16>(a[j]), g = bounds_widen<kBf16>(z[j]);
                    least[2 * j] = f.x, least[2 * j + 1] = f.y;
                    most[2 * j] = g.x, most[2 * j + 1] = g.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) least[j] = most[j] = __uint_as_float(0x7FFFFFFFu);
                constexpr int kSome = 4;
                for (int s0 = row; s0 < p.cache.page_size; s0 += kRows * kSome) {
                    uint4 x[kSome];
                    float scale[kSome];
#pragma unroll
                    for (int u = 0; u < kSome; ++u) {
                        const int slot = s0 + u * kRows;
                        x[u] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        scale[u] = 1.0f;
                        if (inside && slot < p.cache.page_size) {
                            x[u] = __ldcs(reinterpret_cast<const uint4 *>(keys + slot * p.cache.slot_stride));
                            scale[u] = scales[slot * p.cache.scale_slot_stride];
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kSome; ++u) {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
                                    static_cast<__nv_fp8x2_storage_t>((w[j] >> (16 * h)) & 0xFFFFu), __NV_E4M3);
                                const float2 f = __half22float2(__half2(r));
                                const float v0 = f.x * scale[u], v1 = f.y * scale[u];
                                const int e = 4 * j + 2 * h;
                                least[e] = fminf(least[e], v0), most[e] = fmaxf(most[e], v0);
                                least[e + 1] = fminf(least[e + 1], v1), most[e + 1] = fmaxf(most[e + 1], v1);
                            }
                    }
                }
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        least[j] = fminf(least[j], __shfl_xor_sync(0xffffffffu, least[j], o));
                        most[j] = fmaxf(most[j], __shfl_xor_sync(0xffffffffu, most[j], o));
                    }
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                least[j] = kv_finite(least[j]);
                most[j] = kv_finite(most[j]);
                top = fmaxf(top, fmaxf(-least[j], most[j]));
            }
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float s = kv_bounds_scale(top), up = kv_bounds_inverse(s);
            const long long to = static_cast<long long>(page) * p.cache.heads + head;
            uint32_t out[2][kPer / 4];
#pragma unroll
            for (int j = 0; j < kPer / 4; ++j) {
                out[0][j] = out[1][j] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = least[4 * j + i], y = most[4 * j + i];
                    // (a product that fp32 rounds to zero still is a number below or above it)
                    const int f = min(static_cast<int>(floorf(x * up)), x < 0.0f ? -1 : 127);
                    const int c = max(static_cast<int>(ceilf(y * up)), y > 0.0f ? 1 : -127);
                    out[0][j] |= (static_cast<uint32_t>(f) & 255u) << (8 * i);
                    out[1][j] |= (static_cast<uint32_t>(c) & 255u) << (8 * i);
                }
            }
            if (row == 0 && inside && TGEMM_CHECK(to < p.bounds.dbg_rows, kChkKvOutput, p.status)) {
                signed char *const dst = p.bounds.base + to * 2 * p.cache.dim + piece * kPer;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if constexpr (kE4m3)
                        *reinterpret_cast<uint4 *>(dst + w * p.cache.dim) = make_uint4(out[w][0], out[w][1], out[w][kPer / 8], out[w][kPer / 4 - 1]);
                    else
                        *reinterpret_cast<uint2 *>(dst + w * p.cache.dim) = make_uint2(out[w][0], out[w][1]);
                }
                if (piece == 0) p.bounds.scale[to] = s;
            }
        }
        base += items;
        __syncthreads();                           // the sums have been read
    }
}

// ---------------------------------------------------------------- choice
struct ChooseParams {
    KvView cache;
    KvTable table;
    KvBounds bounds;
    const unsigned char *q;
    long long q_batch_stride, q_head_stride;       // bytes
    int group;                                     // query heads of a key head
    int *to_pages;                                 // [batch, heads, keep]
    long long to_batch_stride, to_head_stride;
    int *to_lengths;
    int keep, first, recent;
    int cached;                                    // keys that a block has room for
    unsigned int *status;
};

constexpr int kChooseMaxCached = 32 * 1024;        // keys of a block's slice (128 KiB)
constexpr int kChooseGroup = 128;                  // query heads of a key head, at most

// Bytes of shared memory: keys, then the queries' two halves with their scales.
// Rows lie an odd multiple of 64 bytes apart: the 16-byte reads of two of them fall into different banks.
__host__ __device__ inline int choose_pitch(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 192 : 320; }
__host__ __device__ inline int choose_bytes(int cached, int group, int dim) {
    const int heads = (group + 7) / 8 * 8;
    return (cached + 3) / 4 * 16 + heads * (2 * choose_pitch(dim) + 4);
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What there is to choose from: of `count` pages the first `first` and the last `recent` stay, and `best` of those between.
struct ChooseSpan {
    int count, keep, first, middle, best;
};
__host__ __device__ inline ChooseSpan choose_span(int n, int page_size, int keep, int first, int recent) {
    ChooseSpan s;
    s.count = n / page_size + (n % page_size > 0 ? 1 : 0);
    s.keep = s.count < keep ? s.count : keep;
    const bool all = s.count <= keep;
    s.first = all ? s.count : first;
    s.middle = all ? 0 : s.count - first - recent;
    s.best = all ? 0 : keep - first - recent;
    return s;
}

// Grid: (cluster size, heads, batch), a cluster along x that shares a sequence
// and key head.  kChunks: 64-byte pieces of a row of bounds.
template <int kThreads, bool kBf16, int kChunks>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) page_choose_kernel(const ChooseParams p) {
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ RankShared<kThreads> sh;
    __shared__ int s_n;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int head = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads8 = (p.group + 7) / 8 * 8, pitch = choose_pitch(p.cache.dim);
    unsigned char *const positive = reinterpret_cast<unsigned char *>(keys) + (p.cached + 3) / 4 * 16;
    unsigned char *const negative = positive + heads8 * pitch;
    float *const s_scale = reinterpret_cast<float *>(negative + heads8 * pitch);
    kv_rank_clear(sh);
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        bool bad = false;
        s_n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
        if (bad && rank == 0) record_status(p.status, kStatusCache);
    }
    // The queries in whole numbers, one head a warp at a time.
    for (int h = warp; h < heads8; h += kWarps) {
        constexpr int kPer = 2 * kChunks;                        // dims lane * kPer ..
        float x[kPer], top = 0.0f;
        const unsigned char *const row = p.q + b * p.q_batch_stride + (static_cast<long long>(head) * p.group + h) * p.q_head_stride;
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            const int d = lane * kPer + i;
            uint32_t w = 0;
            if (h < p.group && d < p.cache.dim) w = *reinterpret_cast<const uint32_t *>(row + 2 * d);
            const float2 f = bounds_widen<kBf16>(w);
            x[i] = kv_finite(f.x);
            x[i + 1] = kv_finite(f.y);
            top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float s = kv_bounds_scale(top), up = kv_bounds_inverse(s);
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
            const int y0 = static_cast<int>(rintf(x[i] * up)), y1 = static_cast<int>(rintf(x[i + 1] * up));
            const int at = h * pitch + lane * kPer + i;
            *reinterpret_cast<unsigned short *>(positive + at) = static_cast<unsigned short>(max(y0, 0) | (max(y1, 0) << 8));
            *reinterpret_cast<unsigned short *>(negative + at) =
                static_cast<unsigned short>((min(y0, 0) & 255) | ((min(y1, 0) & 255) << 8));
        }
        if (lane == 0) s_scale[h] = s;
    }
    __syncthreads();
    const int n = s_n;
    const ChooseSpan span = choose_span(n, p.cache.page_size, p.keep, p.first, p.recent);
    const int *const list = p.table.pages + b * p.table.stride;
    int *const to = p.to_pages + b * p.to_batch_stride + head * p.to_head_stride;
    if (head == 0 && rank == 0 && threadIdx.x == 0)
        p.to_lengths[b] = n - (span.count - span.keep) * p.cache.page_size;
    // What stays whatever its score, and -1 past the pages kept.
    for (int i = rank * kThreads + threadIdx.x; i < p.keep; i += blocks * kThreads) {
        if (i >= span.keep) to[i] = -1;
        else if (i < span.first) to[i] = list[i];
        else if (i >= span.first + span.best) to[i] = list[span.count - span.keep + i];
    }
    const bool some = span.best > 0;
    if (!some && blocks == 1) return;
    // The blocks of a cluster go on together to every barrier, whatever length each of them has read.
    const int slice = min((span.middle + blocks - 1) / blocks, p.cached);
    const int lo = span.first + min(span.middle, rank * slice), size = some ? min(span.middle, (rank + 1) * slice) - (lo - span.first) : 0;

    // Scores: a warp has 16 pages at a time, lane (g, t4) 16 bytes of each 64 of pages g and g + 8.
    const int g = lane >> 2, t4 = lane & 3;
    const long long row_bytes = 2 * static_cast<long long>(p.cache.dim);
    for (int i0 = warp * 16; i0 < size; i0 += kWarps * 16) {
        int page = -1;
        if (lane < 16 && i0 + lane < size) page = list[lo + i0 + lane];
        const bool valid = page >= 0 && page < p.cache.pages;
        const unsigned ok = __ballot_sync(0xffffffffu, valid), want = __ballot_sync(0xffffffffu, lane < 16 && i0 + lane < size);
        if (ok != want && lane == 0) record_status(p.status, kStatusCache);
        uint4 a[2][2][kChunks];                                  // [lo, hi][page g, g + 8]
        float scale[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int pg = __shfl_sync(0xffffffffu, page, g + 8 * r);
            const bool is = (ok >> (g + 8 * r)) & 1u;
            const long long at = is ? static_cast<long long>(pg) * p.cache.heads + head : 0;
            scale[r] = is ? p.bounds.scale[at] : 0.0f;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int d = c * 64 + t4 * 16;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    a[w][r][c] = make_uint4(0, 0, 0, 0);
                    if (is && d < p.cache.dim)
                        a[w][r][c] = *reinterpret_cast<const uint4 *>(p.bounds.base + at * row_bytes + w * p.cache.dim + d);
                }
            }
        }
        float best[2] = {-INFINITY, -INFINITY};
        for (int h0 = 0; h0 < heads8; h0 += 8) {
            int acc[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int at = (h0 + g) * pitch + c * 64 + t4 * 16;
                const uint4 qn = *reinterpret_cast<const uint4 *>(negative + at), qp = *reinterpret_cast<const uint4 *>(positive + at);
                mma_s8(acc, a[0][0][c].x, a[0][1][c].x, a[0][0][c].y, a[0][1][c].y, qn.x, qn.y);
                mma_s8(acc, a[0][0][c].z, a[0][1][c].z, a[0][0][c].w, a[0][1][c].w, qn.z, qn.w);
                mma_s8(acc, a[1][0][c].x, a[1][1][c].x, a[1][0][c].y, a[1][1][c].y, qp.x, qp.y);
                mma_s8(acc, a[1][0][c].z, a[1][1][c].z, a[1][0][c].w, a[1][1][c].w, qp.z, qp.w);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = h0 + 2 * t4 + i;
                const float s = s_scale[h];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (h < p.group) best[r] = fmaxf(best[r], static_cast<float>(acc[2 * r + i]) * scale[r] * s);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
            const int i = i0 + g + 8 * r;
            if (t4 == 0 && i < size) keys[i] = (ok >> (g + 8 * r)) & 1u ? kv_weight_key(__float_as_uint(best[r])) : 0u;
        }
    }
    __syncthreads();
    kv_rank(
        sh, size, span.best, p.status, [&](int i) { return keys[i]; },
        [&](int at, int i) { to[span.first + at] = list[lo + i]; });
}

}  // namespace tgemm
