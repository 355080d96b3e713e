// Writing new tokens' keys and values into the paged cache:
//
//     row(b, lengths[b] - n_b + i) = token starts[b] + i         0 <= i < n_b = starts[b + 1] - starts[b]
//
// (without starts, one token per sequence), as it is (16-bit cache) or in e4m3
// with a scale per row: scale = max |x| / 448 (1 for a row of zeros), element =
// x / scale rounded to nearest even.  448 is e4m3's largest value.
//
// Reading and writing each row once bounds it.  Where a row goes takes a chain
// of dependent loads (starts, lengths, page list), so a block first finds the
// places of a whole chunk of rows, one thread each, and then streams the chunk:
// as many lanes as a row has 16-byte pieces, every piece of the chunk (keys and
// values) requested before the first is used, and the next chunk's places found
// while they are on their way.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fp32x2.cuh"
#include "kv_cache.cuh"

namespace tgemm {

struct AppendParams {
    KvView cache;
    KvTable table;
    KvWeights weights;
    const unsigned char *k, *v;
    long long token_stride, head_stride;      // bytes
    const int *starts;
    long long tokens;
    unsigned int *status;
};

// The sequence of token t: the b with starts[b] <= t < starts[b + 1], or -1.
__host__ __device__ inline int kv_sequence_of(const int *starts, int batch, long long t) {
    if (t < starts[0] || t >= starts[batch]) return -1;
    int lo = 0, hi = batch;                   // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Eight 16-bit elements as floats.
template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kBf16) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// A row's scale from its largest magnitude, and -x[i] / scale in place of its
// elements (with the minus, zeros keep their signs).  A product with the reciprocal would move some elements by a whole
// e4m3 step, and eight divisions cost more than the row's traffic; but with r =
// 1 / b and q = a r rounded, q + (a - q b) r is the rounded quotient, the
// parenthesis being exact (Markstein 1990, "Computation of elementary functions
// on the IBM RISC System/6000 processor").  For 1 / 448 r is the rounded
// reciprocal, as the theorem asks; for the elements it is an approximation with
// one Newton step, which leaves the quotient off its rounding only within
// 2^-23 of a unit in the last place of a midpoint.  While nothing leaves fp32's
// normal range that holds; scales outside 2^+-60 take divisions, and within, an
// element so small that it might is zero in e4m3 either way.
template <int N>
__device__ __forceinline__ float scale_row(float (&x)[N], float top) {
    if (!(top > 448 * 0x1p-60f && top < 448 * 0x1p60f)) {
        const float scale = top > 0.0f ? top / 448.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] / -scale;
        return scale;
    }
    constexpr float kInv = 1.0f / 448.0f;
    const float q = top * kInv, scale = fmaf(fmaf(-q, 448.0f, top), kInv, q);
    float r = __fdividef(1.0f, scale);
    r = fmaf(fmaf(-r, scale, 1.0f), r, r);
    const float2 rr = make_float2(-r, -r), ss = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 a = make_float2(x[i], x[i + 1]), q2 = mul2(a, rr), y = fma2(fma2(q2, ss, a), rr, q2);
        x[i] = y.x;
        x[i + 1] = y.y;
    }
    return scale;
}

// Largest magnitude of eight 16-bit elements, in both halves' larger one.
template <bool kBf16>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    if (kBf16) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t top8(const uint4 &u) {       // both halves count
    constexpr uint32_t kMagnitude = 0x7FFF7FFFu;
    return max_pair<kBf16>(max_pair<kBf16>(u.x & kMagnitude, u.y & kMagnitude),
                           max_pair<kBf16>(u.z & kMagnitude, u.w & kMagnitude));
}

// Eight floats' negatives as e4m3.
__device__ __forceinline__ uint2 pack8_negated(const float *x) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE,
                                                                    __NV_E4M3))
                     << (16 * (i & 1));
    return make_uint2(w[0] ^ 0x80808080u, w[1] ^ 0x80808080u);
}

// Blocks take chunks of kRows rows, a row being the keys and values of one
// (token, head), kUnroll passes of kRowThreads / kLanes rows; a lane has kPieces
// 16-byte pieces of a row, kLanes apart (two where a row's maximum and scale
// cost more than its copy: a lane's share of them halves).
constexpr int kRowThreads = 256, kAppendCtas = 4;     // per SM

template <bool kBf16, bool kE4m3, int kLanes, int kPieces, int kUnroll>
__global__ void __launch_bounds__(kRowThreads, kAppendCtas) kv_append_kernel(const AppendParams p) {
    constexpr int kPass = kRowThreads / kLanes, kRows = kPass * kUnroll;
    __shared__ long long s_src[2][kRows], s_dst[2][kRows], s_scale[2][kRows];
    griddep_wait();
    griddep_launch_dependents();
    const long long rows = p.tokens * p.cache.heads, step = static_cast<long long>(gridDim.x) * kRows;
    const int piece = threadIdx.x % kLanes, in_pass = threadIdx.x / kLanes;
    bool inside[kPieces];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) inside[c] = (piece + c * kLanes) * 8 < p.cache.dim;
    // Thread i < kRows finds the place of row r0 + i.
    auto place = [&](long long r0, int to) {
        if (threadIdx.x >= kRows) return;
        const long long r = r0 + threadIdx.x;
        long long src = 0, dst = -1, scale = 0;
        if (r < rows) {
            const long long t = r / p.cache.heads;
            const int head = static_cast<int>(r - t * p.cache.heads);
            int b = static_cast<int>(t);
            long long back = 1;                 // positions from the sequence's end
            if (p.starts) {
                b = kv_sequence_of(p.starts, p.table.batch, t);
                if (b >= 0) back = p.starts[b + 1] - t;
            }
            if (b >= 0) {
                const long long pos = p.table.lengths[b] - back;
                int page, slot;
                if (pos < 0 || pos >= static_cast<long long>(p.table.width) * p.cache.page_size ||
                    !kv_row(p.table.pages + b * p.table.stride, static_cast<int>(pos), p.cache.page_size,
                            p.cache.pages, &page, &slot)) {
                    record_status(p.status, kStatusCache);
                } else {
                    src = t * p.token_stride + head * p.head_stride;
                    dst = kv_offset(p.cache, page, slot, head);
                    if (!TGEMM_CHECK(dst + p.cache.row_bytes <= p.cache.dbg_bytes, kChkKvRow, p.status)) dst = -1;
                    if (kE4m3) scale = kv_scale_offset(p.cache, page, slot, head);
                    if (p.weights.base) {
                        if (pos < p.weights.width)
                            p.weights.base[b * p.weights.batch_stride + head * p.weights.head_stride + pos] = 0.0f;
                        else
                            record_status(p.status, kStatusCache);
                    }
                }
            }
        }
        s_src[to][threadIdx.x] = src;
        s_dst[to][threadIdx.x] = dst;
        s_scale[to][threadIdx.x] = scale;
    };
    long long r0 = static_cast<long long>(blockIdx.x) * kRows;
    place(r0, 0);
    __syncthreads();
    for (int at = 0; r0 < rows; r0 += step, at ^= 1) {
        uint4 x[kUnroll][2][kPieces];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kPass + in_pass;
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                x[u][0][c] = x[u][1][c] = make_uint4(0, 0, 0, 0);
                if (s_dst[at][i] >= 0 && inside[c]) {
                    x[u][0][c] = __ldcs(reinterpret_cast<const uint4 *>(p.k + s_src[at][i]) + piece + c * kLanes);
                    x[u][1][c] = __ldcs(reinterpret_cast<const uint4 *>(p.v + s_src[at][i]) + piece + c * kLanes);
                }
            }
        }
        if (r0 + step < rows) place(r0 + step, at ^ 1);      // while the rows are on their way
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = u * kPass + in_pass;
            const long long dst = s_dst[at][i];
            uint32_t top = 0;                    // keys' largest magnitude below, values' above
            if (kE4m3) {
                uint32_t a = top8<kBf16>(x[u][0][0]), b = top8<kBf16>(x[u][1][0]);
#pragma unroll
                for (int c = 1; c < kPieces; ++c) {
                    a = max_pair<kBf16>(a, top8<kBf16>(x[u][0][c]));
                    b = max_pair<kBf16>(b, top8<kBf16>(x[u][1][c]));
                }
                top = max_pair<kBf16>(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = max_pair<kBf16>(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                unsigned char *pool = which ? p.cache.v : p.cache.k;
                if constexpr (!kE4m3) {
#pragma unroll
                    for (int c = 0; c < kPieces; ++c)
                        if (dst >= 0 && inside[c]) *(reinterpret_cast<uint4 *>(pool + dst) + piece + c * kLanes) = x[u][which][c];
                } else {
                    float f[8 * kPieces];
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) unpack8<kBf16>(x[u][which][c], f + 8 * c);
                    const uint32_t half = which ? top >> 16 : top & 0xFFFFu;
                    const float scale = scale_row(f, kBf16 ? __uint_as_float(half << 16)
                                                           : __half2float(__ushort_as_half(static_cast<unsigned short>(half))));
#pragma unroll
                    for (int c = 0; c < kPieces; ++c)
                        if (dst >= 0 && inside[c])
                            *(reinterpret_cast<uint2 *>(pool + dst) + piece + c * kLanes) = pack8_negated(f + 8 * c);
                    if (dst >= 0 && piece == 0) (which ? p.cache.v_scale : p.cache.k_scale)[s_scale[at][i]] = scale;
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace tgemm
