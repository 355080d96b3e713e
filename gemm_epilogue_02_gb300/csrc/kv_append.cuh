// Writing new tokens' keys and values into the paged cache:
//
//     row(b, lengths[b] - n_b + i) = token starts[b] + i         0 <= i < n_b = starts[b + 1] - starts[b]
//
// (without starts, one token per sequence), as it is (16-bit cache) or in e4m3
// with a scale per row: scale = max |x| / 448 (1 for a row of zeros), element =
// x / scale rounded to nearest even.  448 is e4m3's largest value.  The
// quotient is a true division: a product with the reciprocal would move some
// elements by a whole e4m3 step.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace tgemm {

constexpr int kAppendThreads = 256;

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
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
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

// One warp per row pair (token, head): its key row, then its value row; a lane
// holds eight elements.
template <bool kBf16, bool kE4m3>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long rows = p.tokens * p.cache.heads;
    const long long warps = static_cast<long long>(gridDim.x) * (kAppendThreads / 32);
    for (long long r = static_cast<long long>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5); r < rows;
         r += warps) {
        const long long t = r / p.cache.heads;
        const int head = static_cast<int>(r - t * p.cache.heads);
        int b, count, index;
        if (p.starts) {
            b = kv_sequence_of(p.starts, p.table.batch, t);
            if (b < 0) continue;
            count = p.starts[b + 1] - p.starts[b];
            index = static_cast<int>(t - p.starts[b]);
        } else {
            b = static_cast<int>(t);
            count = 1;
            index = 0;
        }
        const int length = p.table.lengths[b];
        const long long pos = static_cast<long long>(length) - count + index;
        int page = 0, slot = 0;
        if (pos < 0 || pos >= static_cast<long long>(p.table.width) * p.cache.page_size ||
            !kv_row(p.table.pages + b * p.table.stride, static_cast<int>(pos), p.cache.page_size, p.cache.pages,
                    &page, &slot)) {
            if (lane == 0) record_status(p.status, kStatusCache);
            continue;
        }
        if (p.weights.base && lane == 0) {
            if (pos < p.weights.width)
                p.weights.base[b * p.weights.batch_stride + head * p.weights.head_stride + pos] = 0.0f;
            else
                record_status(p.status, kStatusCache);
        }
        const bool has = lane * 8 < p.cache.dim;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const unsigned char *src = (which ? p.v : p.k) + t * p.token_stride + head * p.head_stride;
            unsigned char *dst = (which ? p.cache.v : p.cache.k) + kv_offset(p.cache, page, slot, head);
            uint4 u = make_uint4(0, 0, 0, 0);
            if (has) u = *reinterpret_cast<const uint4 *>(src + lane * 16);
            if (!kE4m3) {
                if (has) *reinterpret_cast<uint4 *>(dst + lane * 16) = u;
                continue;
            }
            float x[8];
            unpack8<kBf16>(u, x);
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float scale = top > 0.0f ? top / 448.0f : 1.0f;
            uint32_t packed[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                packed[i >> 2] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(x[i] / scale, __NV_SATFINITE, __NV_E4M3))
                                  << (8 * (i & 3));
            if (has) *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(packed[0], packed[1]);
            if (lane == 0)
                (which ? p.cache.v_scale : p.cache.k_scale)[kv_scale_offset(p.cache, page, slot, head)] = scale;
        }
    }
}

}  // namespace tgemm
