// Bounds of the keys on a page, and the choice of pages by them.
//
// page_bounds_kernel keeps, for each page and key head, every channel's least and
// largest key in 8 bits: with s the least power of two (2^-100 at least) such
// that no key exceeds 127 s, lo = floor(min / s), hi = ceil(max / s).  A power of
// two makes every step exact: what the bounds are does not depend on how they
// were computed.
//
// page_choose_kernel: with q the query in whole numbers, to nearest, of a power of
// two found in the same way (8 bits of its largest element), sum_d max(q_d lo_d,
// q_d hi_d) times both powers; a page's score is the largest over the group's
// heads.  It bounds the product of any key of the page with the rounded query, the
// query's own to within its rounding.  The sum is that of q+ hi + q- lo (q+ =
// max(q, 0), q- = min(q, 0)), two products with pages as rows and heads as columns.
// The whole numbers are widened to fp16 for them (m16n8k16 takes 2.1 cycles of an
// SM, m16n8k32 of 8-bit whole numbers 16.3) with 1152 added, which the accumulators
// of 64 dims each begin without: what they hold stays below 2^24, so every sum is
// exact in fp32 in any order, and the same pages are chosen however the work is
// split.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "copy_async.cuh"
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

constexpr int kBoundsThreads = 256;
// Positions of a page, at most, whose rows one group of lanes goes through alone.  200000 positions of 8 heads, 128 wide, in
// pages of 16: 16 bits 69 us (groups together: 72), e4m3 63 (112); pages of 32: 69 (68), 57 (71).  Pages of 64: 68 (67), 54
// (61), but one page that comes alone 10 us (6.4).
constexpr int kBoundsAlone = 32;

// Pages of sequence b that its newest tokens complete: [*from, return).
__host__ __device__ inline int kv_completed(int n, long long fresh, int page_size, int *from) {
    long long before = n - fresh;
    if (before < 0) before = 0;
    if (before > n) before = n;
    *from = static_cast<int>(before / page_size);
    return n / page_size;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {       // a NaN gives way to a number
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
__device__ __forceinline__ float min3(float a, float b, float c) {           // NaN gives way to numbers
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Both of a times s.
__device__ __forceinline__ float2 scale2(float2 a, float s) {
    float2 d;
    asm("{\n\t.reg .b64 a, s, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmul.rn.f32x2 d, a, s;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(s));
    return d;
}

// A warp's minima of its rows' groups of kLanes lanes, `values` of each lane:
// group 2^k's lanes hand half of what they have to the other's, down to each group
// having its share (group r: share r of the kRows shares, in order).  The least
// is taken of all, so bounds from above go in with their signs changed.
template <int kLanes, bool kAlone, int N, typename T, typename Min>
__device__ __forceinline__ void bounds_scatter(T (&x)[N], int row, Min least) {
    if (kAlone) return;
    int n = N;
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) {
        n /= 2;
        const bool upper = (row * kLanes) & o;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            if (i < n) {
                const T give = upper ? x[i] : x[i + n], keep = upper ? x[i + n] : x[i];
                x[i] = least(keep, __shfl_xor_sync(0xffffffffu, give, o));
            }
    }
}

// kLanes lanes hold a row in 16-byte pieces; kUnroll rows of a lane are requested
// together.  An item is a page and head.  kAlone: each group of kLanes lanes has an
// item of its own and goes through its rows one by one, so that what an item costs
// besides its rows is shared by the groups; otherwise the groups share an item's
// rows, which a long page wants that comes alone.  Neighbouring groups and warps
// have neighbouring heads of a page.  With 16 bits the reading bounds it; with e4m3
// a warp requests its rows, waits, and widens and scales them while none are on
// their way (issue slots 62 % busy, DRAM 46 %).
template <bool kBf16, bool kE4m3, int kLanes, int kUnroll, bool kAlone>
__global__ void __launch_bounds__(kBoundsThreads, kE4m3 ? (kUnroll > 4 ? 2 : 3) : 4) page_bounds_kernel(const BoundsParams p) {
    constexpr int kWarps = kBoundsThreads / 32, kGroups = 32 / kLanes, kPer = kE4m3 ? 16 : 8;
    constexpr int kRows = kAlone ? 1 : kGroups, kItems = kAlone ? kGroups : 1;       // rows at once; items of a warp
    __shared__ int s_end[kBoundsThreads + 1];      // pages of the sequences of this round, summed up
    __shared__ int s_from[kBoundsThreads];
    __shared__ int s_sum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int piece = lane % kLanes, row = kAlone ? 0 : lane / kLanes, group = kAlone ? lane / kLanes : 0;
    griddep_wait();
    griddep_launch_dependents();
    const long long warps = static_cast<long long>(gridDim.x) * kWarps, me = static_cast<long long>(blockIdx.x) * kWarps + warp;
    const int skip_pages = static_cast<int>(warps * kItems / p.cache.heads), skip_heads = static_cast<int>(warps * kItems % p.cache.heads);
    long long base = 0;                            // units of kItems items in the rounds before
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
        const long long items = static_cast<long long>(s_end[kBoundsThreads]) * p.cache.heads, units = (items + kItems - 1) / kItems;
        // Warp `me` has the units i with (base + i) % warps == me; the next one's pages are looked up a step ahead.  Item j is
        // head j % heads of page j / heads, counted over the round's sequences.
        long long i = (me + warps - base % warps) % warps;
        long long item = i * kItems + group;
        int at = static_cast<int>(item / p.cache.heads), at_head = static_cast<int>(item - static_cast<long long>(at) * p.cache.heads), of = 0;
        if (item < items)                                      // the first one's sequence
            for (int step = kBoundsThreads / 2; step > 0; step /= 2)
                if (s_end[of + step] <= at) of += step;
        // The page of the lane's item, -1 past the last, and its head; then on to the next.
        auto find = [&](int *head) {
            *head = at_head;
            int page = -1;
            if (item < items) {
                while (s_end[of + 1] <= at) ++of;              // (an item that there is lies below the last sum)
                page = p.table.pages[(b0 + of) * p.table.stride + s_from[of] + at - s_end[of]];
                if (page < 0 || page >= p.cache.pages) {
                    record_status(p.status, kStatusCache);
                    page = -1;
                }
            }
            item += warps * kItems;
            at += skip_pages;
            at_head += skip_heads;
            if (at_head >= p.cache.heads) {
                at_head -= p.cache.heads;
                ++at;
            }
            return page;
        };
        int next_head, next_page = find(&next_head);
        for (; i < units; i += warps) {
            const bool there = next_page >= 0;
            const int page = there ? next_page : 0, head = next_head;
            next_page = find(&next_head);
            const bool inside = there && piece * 16 < p.cache.row_bytes;
            const unsigned char *const keys = p.cache.k + kv_offset(p.cache, page, 0, head) + (inside ? piece * 16 : 0);
            const float *const scales = kE4m3 ? p.cache.k_scale + kv_scale_offset(p.cache, page, 0, head) : nullptr;
            // Each channel's least key, and its largest with the sign changed: after the exchange a lane has kOwn of
            // these 2 * kPer.
            constexpr int kOwn = 2 * kPer / kRows;
            float least[kOwn];
            if constexpr (!kE4m3) {
                constexpr uint32_t kNan = 0x7FFF7FFFu;      // gives way to any number
                uint32_t m[8], z[4];                        // least; largest
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = z[j] = kNan;
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
                            m[j] = min_pair<kBf16>(m[j], w[j]);
                            z[j] = most_pair<kBf16>(z[j], w[j]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) m[4 + j] = z[j] ^ 0x80008000u;
                bounds_scatter<kLanes, kAlone>(m, row, [](uint32_t a, uint32_t b) { return min_pair<kBf16>(a, b); });
#pragma unroll
                for (int j = 0; j < kOwn / 2; ++j) {
                    const float2 f = bounds_widen<kBf16>(m[j]);
                    least[2 * j] = f.x, least[2 * j + 1] = f.y;
                }
            } else {
                float m[2 * kPer];
#pragma unroll
                for (int j = 0; j < 2 * kPer; ++j) m[j] = __uint_as_float(0x7FFFFFFFu);
                for (int s0 = row; s0 < p.cache.page_size; s0 += kRows * kUnroll) {
                    uint4 x[kUnroll];
                    float scale[kUnroll];
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        const int slot = s0 + u * kRows;
                        x[u] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        scale[u] = 1.0f;
                        if (inside && slot < p.cache.page_size) {
                            x[u] = __ldcs(reinterpret_cast<const uint4 *>(keys + slot * p.cache.slot_stride));
                            scale[u] = scales[slot * p.cache.scale_slot_stride];
                        }
                    }
                    // Two rows at a time.
#pragma unroll
                    for (int u = 0; u < kUnroll; u += 2) {
                        if (s0 - row + u * kRows >= p.cache.page_size) break;      // all rows of the warp
                        const uint32_t w[2][4] = {{x[u].x, x[u].y, x[u].z, x[u].w}, {x[u + 1].x, x[u + 1].y, x[u + 1].z, x[u + 1].w}};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float2 v[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(
                                        static_cast<__nv_fp8x2_storage_t>((w[k][j] >> (16 * h)) & 0xFFFFu), __NV_E4M3);
                                    v[k] = scale2(__half22float2(__half2(r)), scale[u + k]);
                                }
                                const int e = 4 * j + 2 * h;
                                m[e] = min3(m[e], v[0].x, v[1].x);
                                m[e + 1] = min3(m[e + 1], v[0].y, v[1].y);
                                m[kPer + e] = max3(m[kPer + e], v[0].x, v[1].x);
                                m[kPer + e + 1] = max3(m[kPer + e + 1], v[0].y, v[1].y);
                            }
                    }
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j) m[kPer + j] = -m[kPer + j];
                bounds_scatter<kLanes, kAlone>(m, row, [](float a, float b) { return fminf(a, b); });
#pragma unroll
                for (int j = 0; j < kOwn; ++j) least[j] = m[j];
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                least[j] = kv_finite(least[j]);
                top = fmaxf(top, -least[j]);
            }
            if constexpr (kAlone) {
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            } else {
                // (numbers >= 0 have the order of their bits)
                top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            }
            const float s = kv_bounds_scale(top), up = kv_bounds_inverse(s);
            const long long to = static_cast<long long>(page) * p.cache.heads + head;
            // Shares 0 .. kRows / 2 - 1 are the lower bounds' channels in order, the others the upper ones'.  With one row
            // at a time a lane has both.
            uint32_t out[kOwn / 4];
#pragma unroll
            for (int j = 0; j < kOwn / 4; ++j) {
                out[j] = 0;
                const bool upper = kRows == 1 ? j >= kOwn / 8 : row >= kRows / 2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = least[4 * j + i];
                    // (a product that fp32 rounds to zero still stands for a number below it)
                    const int f = min(static_cast<int>(floorf(x * up)), x < 0.0f ? -1 : 127);
                    out[j] |= (static_cast<uint32_t>(upper ? -f : f) & 255u) << (8 * i);
                }
            }
            if (inside && TGEMM_CHECK(to < p.bounds.dbg_rows, kChkKvOutput, p.status)) {
                signed char *const dst = p.bounds.base + to * 2 * p.cache.dim + piece * kPer;
                if constexpr (kRows == 1 && kE4m3) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
                    *reinterpret_cast<uint4 *>(dst + p.cache.dim) = make_uint4(out[kOwn / 4 - 4], out[kOwn / 4 - 3], out[kOwn / 4 - 2], out[kOwn / 4 - 1]);
                } else if constexpr (kRows == 1) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
                    *reinterpret_cast<uint2 *>(dst + p.cache.dim) = make_uint2(out[kOwn / 4 - 2], out[kOwn / 4 - 1]);
                } else {
                    constexpr int kShares = kRows / 2;       // of kPer channels
                    signed char *const at = dst + (row / kShares) * p.cache.dim + (row % kShares) * kOwn;
                    if constexpr (kOwn == 4) *reinterpret_cast<uint32_t *>(at) = out[0];
                    else if constexpr (kOwn == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(out[0], out[1]);
                    else *reinterpret_cast<uint4 *>(at) = make_uint4(out[0], out[1], out[kOwn / 4 - 2], out[kOwn / 4 - 1]);
                }
                if (piece == 0 && row == 0) p.bounds.scale[to] = s;
            }
        }
        base += units;
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
    bool gather;                                   // a cluster's first block has room for the keys of all
    unsigned int *status;
};

constexpr int kChooseGroup = 64;                  // query heads of a key head, at most

// Bytes of shared memory: keys, then the queries' two halves (fp16) with their scales.  Rows lie 16 bytes more than a
// multiple of 128 apart: the 16-byte reads of two of them fall into different banks.
__host__ __device__ constexpr int choose_pitch(int dim) { return (dim <= 64 ? 128 : dim <= 128 ? 256 : 512) + 16; }
// A page's bounds in a warp's ring: the 16-byte pieces of row r are exchanged by choose_swizzle(r) (xor), for the same
// reason.
constexpr int choose_row(int chunks) { return chunks * 128; }
__device__ __forceinline__ int choose_swizzle(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }
// The ring, or, after it, what the ranking takes; keys; queries with their scales and the accumulators' beginnings.
template <int kThreads, int kChunks, int kStages>
struct ChooseShape {
    static constexpr int kStage = 16 * choose_row(kChunks) + 128;         // a step's rows, their scales and which there are
    static constexpr int kRing = kThreads / 32 * kStages * kStage;
    static constexpr int kRank = (static_cast<int>(sizeof(RankShared<kThreads>)) + 15) / 16 * 16;
    static constexpr int kFront = kRing > kRank ? kRing : kRank;
    __host__ __device__ static constexpr int bytes(int cached, int group, int dim) {
        return kFront + (cached + 3) / 4 * 16 + (group + 7) / 8 * 8 * (2 * choose_pitch(dim) + 4 + 8 * kChunks);
    }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8-bit whole numbers as fp16, 1152 more than they are: x + 128 put below 1024's bits.  The first and third, then
// the second and fourth.
constexpr float kChooseBias = 1152.0f;
__device__ __forceinline__ void widen_s8(uint32_t x, uint32_t &even, uint32_t &odd) {
    even = (x & 0x00FF00FFu) ^ 0x64806480u;
    odd = ((x >> 8) & 0x00FF00FFu) ^ 0x64806480u;
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
// kFew: at most eight query heads, whose operands stay in registers.
template <int kThreads, bool kBf16, int kChunks, int kStages, bool kFew>
__global__ void __launch_bounds__(kThreads, kThreads * kChunks > 512 ? 1 : 2) page_choose_kernel(const ChooseParams p) {
    using Shape = ChooseShape<kThreads, kChunks, kStages>;
    constexpr int kWarps = kThreads / 32, kRow = choose_row(kChunks), kPitch = kChunks * 128 + 16;     // choose_pitch()
    extern __shared__ __align__(128) unsigned char choose_smem[];
    RankShared<kThreads> &sh = *reinterpret_cast<RankShared<kThreads> *>(choose_smem);
    __shared__ int s_n;
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int head = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads8 = (p.group + 7) / 8 * 8, pitch = kPitch;
    unsigned char *const ring = choose_smem + warp * kStages * Shape::kStage;
    uint32_t *const keys = reinterpret_cast<uint32_t *>(choose_smem + Shape::kFront);
    unsigned char *const positive = reinterpret_cast<unsigned char *>(keys) + (p.cached + 3) / 4 * 16;
    unsigned char *const negative = positive + heads8 * pitch;
    float *const s_scale = reinterpret_cast<float *>(negative + heads8 * pitch);
    float *const s_bias = s_scale + heads8;                      // [2 * kChunks][heads8]: of lo's and hi's sums over 64 dims
    griddep_wait();
    if (p.gather) cluster.barrier_arrive();      // this block has begun: the others may write to its shared memory
    if (threadIdx.x == 0) {
        bool bad = false;
        s_n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
        if (bad && rank == 0) record_status(p.status, kStatusCache);
    }
    // The queries in whole numbers, one head a warp at a time.
    bool far = false;                                            // a power above 2^100
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
            // (of four dims the second and third change places, as widen_s8() has them)
            const float y0 = rintf(x[i] * up), y1 = rintf(x[i + 1] * up);
            const int d = lane * kPer + i, at = h * pitch + 2 * (d & ~3) + (d & 2);
            *reinterpret_cast<__half *>(positive + at) = __float2half_rn(fmaxf(y0, 0.0f));
            *reinterpret_cast<__half *>(positive + at + 4) = __float2half_rn(fmaxf(y1, 0.0f));
            *reinterpret_cast<__half *>(negative + at) = __float2half_rn(fminf(y0, 0.0f));
            *reinterpret_cast<__half *>(negative + at + 4) = __float2half_rn(fminf(y1, 0.0f));
        }
        // Lanes of the same 64 dims: 32 / kChunks of them.
        float below = 0.0f, above = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            below += fminf(rintf(x[i] * up), 0.0f);
            above += fmaxf(rintf(x[i] * up), 0.0f);
        }
#pragma unroll
        for (int o = 16 / kChunks; o > 0; o >>= 1) {
            below += __shfl_xor_sync(0xffffffffu, below, o);
            above += __shfl_xor_sync(0xffffffffu, above, o);
        }
        if (lane % (32 / kChunks) == 0) {
            const int c = lane / (32 / kChunks);
            s_bias[2 * c * heads8 + h] = -kChooseBias * below;
            s_bias[(2 * c + 1) * heads8 + h] = -kChooseBias * above;
        }
        if (lane == 0) s_scale[h] = s;
        far |= s > 0x1p100f;
    }
    far = __syncthreads_or(far);
    const int n = s_n;
    const ChooseSpan span = choose_span(n, p.cache.page_size, p.keep, p.first, p.recent);
    const int *const list = p.table.pages + b * p.table.stride;
    int *const to = p.to_pages + b * p.to_batch_stride + head * p.to_head_stride;
    if (head == 0 && rank == 0 && threadIdx.x == 0)
        p.to_lengths[b] = n - (span.count - span.keep) * p.cache.page_size;
    const bool some = span.best > 0;
    // The blocks of a cluster go on together to every barrier, whatever length each of them has read.
    const int slice = min((span.middle + blocks - 1) / blocks, p.cached);      // (of a gathered list: p.cached for all)
    const int lo = span.first + min(span.middle, rank * slice), size = some ? min(span.middle, (rank + 1) * slice) - (lo - span.first) : 0;
    // The slice's page numbers wait where its keys go: each is read before its key is written.
    for (int i = threadIdx.x; i < size; i += kThreads) keys[i] = static_cast<uint32_t>(list[lo + i]);
    // The queries' powers at most 2^100, by a factor that all scores share: a sum times its query's power stays in fp32's
    // range, and the page's power takes it out of there only with the score itself.
    if (far && warp == 0) {
        float top = 0.0f;
        for (int h = lane; h < p.group; h += 32) top = fmaxf(top, s_scale[h]);
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        for (int h = lane; h < p.group; h += 32) s_scale[h] *= 0x1p100f / top;
    }
    // What stays whatever its score, and -1 past the pages kept.
    for (int i = rank * kThreads + threadIdx.x; i < p.keep; i += blocks * kThreads) {
        if (i >= span.keep) to[i] = -1;
        else if (i < span.first) to[i] = list[i];
        else if (i >= span.first + span.best) to[i] = list[span.count - span.keep + i];
    }
    if (!some && blocks == 1) {
        griddep_launch_dependents();
        return;
    }
    __syncthreads();

    // Scores: a warp has 16 pages at a time, whose bounds are copied to its ring kStages - 1 steps ahead.  A row is
    // both bounds of a page and head, 2 * dim bytes in one piece.
    const int g = lane >> 2, t4 = lane & 3, pieces = p.cache.dim / 8;
    const bool mine = lane % (8 * kChunks) < pieces;
    const int page_bytes = p.cache.heads * 2 * p.cache.dim;
    const signed char *const from = p.bounds.base + static_cast<long long>(head) * 2 * p.cache.dim + (mine ? lane % (8 * kChunks) * 16 : 0);
    const uint32_t to_ring = smem_u32(ring);
    int at_piece[kChunks][2];                                    // where the lane's piece of 64 dims is in row g (and g + 8)
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int w = 0; w < 2; ++w)
            at_piece[c][w] = g * kRow + ((min(w * pieces / 2 + c * 4 + t4, 8 * kChunks - 1) ^ choose_swizzle(g)) << 4);
    int ahead = warp * 16;
    auto request = [&](int stage) {
        const int i0 = ahead;
        ahead += kWarps * 16;
        const bool there = lane < 16 && i0 + lane < size;
        const int page = there ? static_cast<int>(keys[i0 + lane]) : -1;
        const bool valid = page >= 0 && page < p.cache.pages;
        const unsigned ok = __ballot_sync(0xffffffffu, valid);
        if (ok != __ballot_sync(0xffffffffu, there) && lane == 0) record_status(p.status, kStatusCache);
        const uint32_t to = to_ring + stage * Shape::kStage;
        if (valid) cp_async4(to + 16 * kRow + 4 * lane, p.bounds.scale + static_cast<long long>(page) * p.cache.heads + head, true);
        if (lane == 0) *reinterpret_cast<unsigned *>(ring + stage * Shape::kStage + 16 * kRow + 64) = ok;
        // A lane copies one 16-byte piece of every 32 / kPieces rows.
        constexpr int kPieces = 8 * kChunks, kEach = 32 / kPieces;
#pragma unroll
        for (int u = 0; u < 16 / kEach; ++u) {
            const int r = u * kEach + lane / kPieces, pg = __shfl_sync(0xffffffffu, page, r);
            if (((ok >> r) & 1u) && mine)
                cp_async16(to + r * kRow + ((lane % kPieces ^ choose_swizzle(r)) << 4), from + static_cast<long long>(pg) * page_bytes);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) request(k);
    int stage = 0;
    auto queries = [&](int h0, int half, uint4 (&q)[2 * kChunks]) {
#pragma unroll
        for (int k = 0; k < 2 * kChunks; ++k)
            q[k] = *reinterpret_cast<const uint4 *>((k % 2 ? positive : negative) + (h0 + g) * pitch + k / 2 * 128 + t4 * 32 + half * 16);
    };
    uint4 kept_q[2][2 * kChunks];
    if (kFew) {
        queries(0, 0, kept_q[0]);
        queries(0, 1, kept_q[1]);
    }
    for (int i0 = warp * 16; i0 < size; i0 += kWarps * 16) {
        cp_async_wait<kStages - 2>();
        __syncwarp();
        // the stage that the step before has read takes the one kStages - 1 steps on
        request(stage == 0 ? kStages - 1 : stage - 1);
        const unsigned char *const at_hand = ring + stage * Shape::kStage;
        const unsigned ok = *reinterpret_cast<const unsigned *>(at_hand + 16 * kRow + 64);
        const float *const stage_scale = reinterpret_cast<const float *>(at_hand + 16 * kRow);
        const float scale[2] = {stage_scale[g], stage_scale[g + 8]};
        stage = stage + 1 == kStages ? 0 : stage + 1;
        float best[2] = {-INFINITY, -INFINITY};
        for (int h0 = 0; h0 < (kFew ? 8 : heads8); h0 += 8) {
            // One chain of products for each bound of 64 dims, a step of each in turn.
            float acc[2 * kChunks][4];
            uint4 xs[2 * kChunks], ys[2 * kChunks];
#pragma unroll
            for (int k = 0; k < 2 * kChunks; ++k) {
                const float2 bias = *reinterpret_cast<const float2 *>(s_bias + k * heads8 + h0 + 2 * t4);
                acc[k][0] = acc[k][2] = bias.x;
                acc[k][1] = acc[k][3] = bias.y;
                // Past dim the queries are 0 and the bounds whatever the ring holds, as whole numbers.
                const unsigned char *const at = at_hand + at_piece[k / 2][k % 2];
                xs[k] = *reinterpret_cast<const uint4 *>(at);
                ys[k] = *reinterpret_cast<const uint4 *>(at + 8 * kRow);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!kFew) queries(h0, half, kept_q[half]);
                const uint4 (&q)[2 * kChunks] = kept_q[half];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2 * kChunks; ++k) {
                        const uint32_t x = half ? (j ? xs[k].w : xs[k].z) : (j ? xs[k].y : xs[k].x);
                        const uint32_t y = half ? (j ? ys[k].w : ys[k].z) : (j ? ys[k].y : ys[k].x);
                        uint32_t x0, x1, y0, y1;
                        widen_s8(x, x0, x1);
                        widen_s8(y, y0, y1);
                        mma_f16(acc[k], x0, y0, x1, y1, j ? q[k].z : q[k].x, j ? q[k].w : q[k].y);
                    }
            }
#pragma unroll
            for (int c = 1; c < 2 * kChunks; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[0][i] += acc[c][i];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = h0 + 2 * t4 + i;
                const float s = s_scale[h];
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    if (h < p.group) best[r] = fmaxf(best[r], acc[0][2 * r + i] * s * scale[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
            const int i = i0 + g + 8 * r;
            if (t4 == 0 && i < size)
                keys[i] = (ok >> (g + 8 * r)) & 1u ? kv_weight_key(__float_as_uint(best[r])) : 0u;
        }
    }
    griddep_launch_dependents();                 // what follows would take the places of blocks that have not begun
    cp_async_wait<0>();
    if (p.gather) {
        // The first block ranks the keys of all: two barriers of the cluster instead of five.
        uint32_t *const all_keys = cluster.map_shared_rank(keys, 0);
        cluster.barrier_wait();
        __syncthreads();
        if (rank > 0)
            for (int i = threadIdx.x; i < size; i += kThreads)
                if (lo - span.first + i < p.cached) all_keys[lo - span.first + i] = keys[i];
        cluster.sync();
        if (rank > 0) return;
        kv_rank_clear(sh);                       // in the ring's place
        __syncthreads();
        kv_rank<RankBy::kBlock>(
            sh, some ? min(span.middle, p.cached) : 0, span.best, p.status, [&](int i) { return keys[i]; },
            [&](int at, int i) { to[span.first + at] = list[span.first + i]; });
        return;
    }
    __syncthreads();
    kv_rank_clear(sh);                           // in the ring's place
    __syncthreads();
    kv_rank(
        sh, size, span.best, p.status, [&](int i) { return keys[i]; },
        [&](int at, int i) { to[span.first + at] = list[lo + i]; });
}

}  // namespace tgemm
