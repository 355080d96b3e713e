// Attention of one new token per sequence over the paged cache:
//
//     o[b, h] = sum_j p_j v_j,  p = softmax over lo <= j < n of s_j = cap(scale q[b, h] . k_j),
//
// n = lengths[b], lo = max(0, n - window) (0 without a window), cap(s) =
// c tanh(s / c) when c > 0.  Heads share the keys of head h / group.  n = 0
// gives zeros.  With weights, weights[b, g, j] grows by the sum of p_j over the
// group's heads.
//
// Simple form: one block per sequence and key head, one warp per key, the
// running maximum, sum and output of a warp in registers, joined at the end.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace tgemm {

constexpr int kAttendWarps = 8;
constexpr int kAttendMaxDim = 256;

struct AttendParams {
    KvView cache;
    KvTable table;
    KvWeights weights;
    const unsigned char *q;
    unsigned char *o;
    long long q_batch_stride, q_head_stride, o_batch_stride, o_head_stride;   // bytes
    int group;
    int window;
    float scale, cap;
    unsigned int *status;
};

template <bool kBf16>
__device__ __forceinline__ float load16(const unsigned char *p, int i) {
    if (kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(reinterpret_cast<const __half *>(p)[i]);
}

template <bool kBf16, bool kE4m3>
__device__ __forceinline__ float load_row(const unsigned char *p, int i) {
    if (kE4m3) {
        const __nv_fp8_storage_t b = p[i];
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
    }
    return load16<kBf16>(p, i);
}

template <bool kBf16, bool kE4m3>
__global__ void __launch_bounds__(kAttendWarps * 32) kv_attend_kernel(const AttendParams p) {
    constexpr int kPer = kAttendMaxDim / 32;
    __shared__ float part_o[kAttendWarps][kAttendMaxDim];
    __shared__ float part_m[kAttendWarps], part_l[kAttendWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int head = blockIdx.x, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad = false;
    const int n = kv_length(p.table.lengths[b], p.table.width, p.cache.page_size, &bad);
    if (bad && threadIdx.x == 0) record_status(p.status, kStatusCache);
    const int lo = p.window > 0 && n > p.window ? n - p.window : 0;
    const int *list = p.table.pages + b * p.table.stride;
    float q[kPer];
    auto score = [&](int j, float *ks_out, const unsigned char **vrow, float *vs) {
        int page, slot;
        if (!kv_row(list, j, p.cache.page_size, p.cache.pages, &page, &slot)) return false;
        const unsigned char *krow = p.cache.k + kv_offset(p.cache, page, slot, head);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < p.cache.dim) s += q[i] * load_row<kBf16, kE4m3>(krow, lane + 32 * i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (kE4m3) {
            const long long at = kv_scale_offset(p.cache, page, slot, head);
            s *= p.cache.k_scale[at];
            *vs = p.cache.v_scale[at];
        } else {
            *vs = 1.0f;
        }
        s *= p.scale;
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        *vrow = p.cache.v + kv_offset(p.cache, page, slot, head);
        *ks_out = s;
        return true;
    };
    for (int g = 0; g < p.group; ++g) {
        const int qh = head * p.group + g;
        const unsigned char *qrow = p.q + b * p.q_batch_stride + qh * p.q_head_stride;
#pragma unroll
        for (int i = 0; i < kPer; ++i) q[i] = lane + 32 * i < p.cache.dim ? load16<kBf16>(qrow, lane + 32 * i) : 0.0f;
        float m = -INFINITY, l = 0.0f, o[kPer] = {};
        for (int j = lo + warp; j < n; j += kAttendWarps) {
            float s, vs;
            const unsigned char *vrow;
            if (!score(j, &s, &vrow, &vs)) {
                if (lane == 0) record_status(p.status, kStatusCache);
                continue;
            }
            const float m_new = fmaxf(m, s);
            const float a = expf(m - m_new), w = expf(s - m_new);
            l = l * a + w;
            m = m_new;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < p.cache.dim)
                    o[i] = o[i] * a + w * vs * load_row<kBf16, kE4m3>(vrow, lane + 32 * i);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) part_o[warp][lane + 32 * i] = o[i];
        if (lane == 0) {
            part_m[warp] = m;
            part_l[warp] = l;
        }
        __syncthreads();
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, part_m[w]);
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < kAttendWarps; ++w) sum += part_l[w] * expf(part_m[w] - ref);
        for (int d = threadIdx.x; d < p.cache.dim; d += kAttendWarps * 32) {
            float v = 0.0f;
            for (int w = 0; w < kAttendWarps; ++w) v += part_o[w][d] * expf(part_m[w] - ref);
            v = sum != 0.0f ? v / sum : 0.0f;
            unsigned char *orow = p.o + b * p.o_batch_stride + qh * p.o_head_stride;
            if (kBf16) reinterpret_cast<__nv_bfloat16 *>(orow)[d] = __float2bfloat16_rn(v);
            else reinterpret_cast<__half *>(orow)[d] = __float2half_rn(v);
        }
        if (p.weights.base) {
            float *w = p.weights.base + b * p.weights.batch_stride + head * p.weights.head_stride;
            for (int j = lo + warp; j < n; j += kAttendWarps) {
                float s, vs;
                const unsigned char *vrow;
                if (!score(j, &s, &vrow, &vs) || lane != 0) continue;
                if (j < p.weights.width) w[j] += expf(s - ref) / sum;
                else record_status(p.status, kStatusCache);
            }
        }
        __syncthreads();
    }
}

}  // namespace tgemm
