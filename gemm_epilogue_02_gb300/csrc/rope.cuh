// Norms of queries and keys for each head with the position rotation in the
// same pass, and its gradient:
//
//     y = R (x r w),   r = 1 / sqrt(mean x^2 + eps)
//
// R turns the pairs (i, i + pairs) or (2 i, 2 i + 1) of the first 2 * pairs
// elements by the angle p_i f_i, p_i the token's position on pair i's axis.  With
// g = R^T dy:
//
//     dw = sum over rows of g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Reading and writing each row once bounds it.  Angles: a frequency is given in
// turns as a 64-bit fraction, so that position * frequency, which wraps at whole
// turns by itself, keeps 2^-33 of a turn at any 32-bit position; the upper 32
// bits then go through sincospi in fp32.  (fp32 angles are off by whole
// radians at far positions, fp64 runs at 1/64 of fp32's rate here.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "debug_checks.cuh"
#include "ptx.cuh"

namespace tgemm {

constexpr int kRopePairs = 128;             // at most (dim 256)
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxBlocks = 1024;        // whose partial sums of weight gradients the workspace holds

struct RopeSide {
    const unsigned char *x, *g;             // rows, and (backward) gradients of what the forward pass wrote
    unsigned char *y;                       // what is written: rotated rows, or (backward) gradients of x
    const void *w;                          // null: ones
    float *dw;                              // null: not wanted
    long long x_token, x_head, g_token, g_head, y_token, y_head;     // bytes
    int heads;
};

struct RopeParams {
    RopeSide side[2];                       // queries, keys
    const int *positions;                   // [axes, tokens]
    long long axis_stride, tokens;
    float *partials;                        // [blocks][2][dim]
    float eps;
    int norm, weight_f32, shift, dim, pairs;
    int chunks;                             // parts that a token's rows are cut into
    int blocks;                             // of the pass that left the partial sums
    unsigned int *status;
    long long dbg_y[2];                     // debug builds: bytes of what is written
    unsigned long long turns[kRopePairs];
    unsigned char axis[kRopePairs];
};

// A lane has two units of V elements of a row whose elements turn with one
// another: a[i] with b[i].
template <bool kBf16>
__device__ __forceinline__ float2 rope_unpack(uint32_t w) {
    if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t rope_pack(float lo, float hi) {
    if (kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int V>
struct RopeRaw {
    uint32_t w[2][V / 2];
};

template <int V>
__device__ __forceinline__ void rope_read(RopeRaw<V> &raw, const unsigned char *row, const int (&unit)[2], const bool (&is)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (V == 8) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (is[j]) u = __ldcs(reinterpret_cast<const uint4 *>(row) + unit[j]);
            raw.w[j][0] = u.x, raw.w[j][1] = u.y, raw.w[j][2] = u.z, raw.w[j][3] = u.w;
        } else {
            uint2 u = make_uint2(0, 0);
            if (is[j]) u = __ldcs(reinterpret_cast<const uint2 *>(row) + unit[j]);
            raw.w[j][0] = u.x, raw.w[j][1] = u.y;
        }
    }
}

template <bool kBf16, int V, bool kInterleaved>
__device__ __forceinline__ void rope_split(const RopeRaw<V> &raw, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = rope_unpack<kBf16>(raw.w[j][i]);
            if (kInterleaved) {
                a[j * (V / 2) + i] = f.x;
                b[j * (V / 2) + i] = f.y;
            } else {
                (j ? b : a)[2 * i] = f.x;
                (j ? b : a)[2 * i + 1] = f.y;
            }
        }
}

template <bool kBf16, int V, bool kInterleaved>
__device__ __forceinline__ void rope_write(unsigned char *row, const float (&a)[V], const float (&b)[V], const int (&unit)[2],
                                           const bool (&is)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if (kInterleaved)
                w[i] = rope_pack<kBf16>(a[j * (V / 2) + i], b[j * (V / 2) + i]);
            else
                w[i] = rope_pack<kBf16>((j ? b : a)[2 * i], (j ? b : a)[2 * i + 1]);
        }
        if (!is[j]) continue;
        if constexpr (V == 8)
            *(reinterpret_cast<uint4 *>(row) + unit[j]) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *(reinterpret_cast<uint2 *>(row) + unit[j]) = make_uint2(w[0], w[1]);
    }
}

// Element of the row that a[i] (j = 0) or b[i] (j = 1) is.
template <int V, bool kInterleaved>
__device__ __forceinline__ int rope_element(int i, int j, const int (&unit)[2]) {
    if (kInterleaved) return unit[i / (V / 2)] * V + 2 * (i % (V / 2)) + j;
    return unit[j] * V + i;
}

template <bool kBf16, int V, bool kInterleaved>
__device__ __forceinline__ void rope_weights(const void *w, bool f32, int dim, const int (&unit)[2], float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = rope_element<V, kInterleaved>(i, j, unit);
            float x = 1.0f;
            if (w && e < dim) {
                if (f32) x = static_cast<const float *>(w)[e];
                else if (kBf16) x = __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[e]);
                else x = __half2float(static_cast<const __half *>(w)[e]);
            }
            (j ? b : a)[i] = x;
        }
}

// Where lane `l` of a row's kLanes has its two units.
template <int V, bool kInterleaved>
__device__ __forceinline__ void rope_units(int l, int dim, int pairs, int (&unit)[2], bool (&is)[2]) {
    const int units = dim / V, half = pairs / V;
    if (kInterleaved || l >= half) {
        const int from = kInterleaved ? 0 : half;
        unit[0] = 2 * from + 2 * (l - from);
        unit[1] = unit[0] + 1;
    } else {
        unit[0] = l;
        unit[1] = l + half;
    }
    is[0] = unit[0] < units;
    is[1] = unit[1] < units;
}

template <int N>
__device__ __forceinline__ float rope_sum(float x) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The angles of one token's pairs.
template <int V>
__device__ __forceinline__ void rope_angles(const RopeParams &p, long long token, const unsigned long long (&turns)[V],
                                            const unsigned (&axis)[V], int first, float (&c)[V], float (&s)[V]) {
    long long pos = 0;
    unsigned last = ~0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
        if (first + i < p.pairs) {
            if (axis[i] != last) {
                last = axis[i];
                pos = static_cast<long long>(p.positions[last * p.axis_stride + token]) + p.shift;
            }
            const unsigned long long t = static_cast<unsigned long long>(pos) * turns[i];
            sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, &s[i], &c[i]);
        }
    }
}

// kLanes lanes have a row, a warp 32 / kLanes rows of one token's queries or
// keys at a time; its sines and cosines stay in registers for all of them.
template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kUnroll = 2;
    const int lane = threadIdx.x & 31, l = lane % kLanes, row = lane / kLanes;
    int unit[2];
    bool is[2];
    rope_units<V, kInterleaved>(l, p.dim, p.pairs, unit, is);
    unsigned long long turns[V];
    unsigned axis[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = min(l * V + i, kRopePairs - 1);
        turns[i] = p.turns[at];
        axis[i] = p.axis[at];
    }
    griddep_wait();
    griddep_launch_dependents();
    float wa[2][V], wb[2][V];
#pragma unroll
    for (int q = 0; q < 2; ++q) rope_weights<kBf16, V, kInterleaved>(p.side[q].w, p.weight_f32, p.dim, unit, wa[q], wb[q]);
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const long long items = p.tokens * p.chunks;
    const long long warps = static_cast<long long>(gridDim.x) * (kRopeThreads / 32);
    const int passes_q = (p.side[0].heads + kRows - 1) / kRows, passes = passes_q + (p.side[1].heads + kRows - 1) / kRows;
    for (long long item = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5); item < items; item += warps) {
        const long long token = p.chunks == 1 ? item : item / p.chunks;
        const int chunk = static_cast<int>(item - token * p.chunks);
        const int from = static_cast<int>(static_cast<long long>(chunk) * passes / p.chunks);
        const int to = static_cast<int>(static_cast<long long>(chunk + 1) * passes / p.chunks);
        float c[V], s[V];
        rope_angles<V>(p, token, turns, axis, l * V, c, s);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const RopeSide &side = p.side[q];
            const int lo = q ? max(from - passes_q, 0) : min(from, passes_q), hi = q ? max(to - passes_q, 0) : min(to, passes_q);
            const unsigned char *const x = side.x + token * side.x_token;
            unsigned char *const y = side.y + token * side.y_token;
            for (int pass = lo; pass < hi; pass += kUnroll) {
                RopeRaw<V> raw[kUnroll];
                bool in[kUnroll][2];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int head = (pass + u) * kRows + row;
                    const bool there = pass + u < hi && head < side.heads;
                    in[u][0] = there && is[0];
                    in[u][1] = there && is[1];
                    rope_read<V>(raw[u], x + (there ? head : 0) * side.x_head, unit, in[u]);
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float a[V], b[V], r = 1.0f;
                    rope_split<kBf16, V, kInterleaved>(raw[u], a, b);
                    if (p.norm) {
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < V; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
                        r = rsqrtf(fmaf(rope_sum<kLanes>(sum), inv_dim, p.eps));
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float f = a[i] * r * wa[q][i], g = b[i] * r * wb[q][i];
                        a[i] = f * c[i] - g * s[i];
                        b[i] = g * c[i] + f * s[i];
                    }
                    const long long at = ((pass + u) * kRows + row) * side.y_head;
                    if ((in[u][0] || in[u][1]) &&
                        TGEMM_CHECK(token * side.y_token + at + 2 * p.dim <= p.dbg_y[q], kChkRope, p.status))
                        rope_write<kBf16, V, kInterleaved>(y + at, a, b, unit, in[u]);
                }
            }
        }
    }
}

template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_backward_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kWarps = kRopeThreads / 32;
    __shared__ float s_dw[kWarps][2][2 * kRopePairs];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % kLanes, row = lane / kLanes;
    int unit[2];
    bool is[2];
    rope_units<V, kInterleaved>(l, p.dim, p.pairs, unit, is);
    unsigned long long turns[V];
    unsigned axis[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = min(l * V + i, kRopePairs - 1);
        turns[i] = p.turns[at];
        axis[i] = p.axis[at];
    }
    griddep_wait();
    griddep_launch_dependents();
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const long long items = p.tokens * p.chunks;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps;
    const int passes_q = (p.side[0].heads + kRows - 1) / kRows, passes = passes_q + (p.side[1].heads + kRows - 1) / kRows;
    float da[2][V], db[2][V];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) da[q][i] = db[q][i] = 0.0f;
    for (long long item = static_cast<long long>(blockIdx.x) * kWarps + warp; item < items; item += warps) {
        const long long token = p.chunks == 1 ? item : item / p.chunks;
        const int chunk = static_cast<int>(item - token * p.chunks);
        const int from = static_cast<int>(static_cast<long long>(chunk) * passes / p.chunks);
        const int to = static_cast<int>(static_cast<long long>(chunk + 1) * passes / p.chunks);
        float c[V], s[V];
        rope_angles<V>(p, token, turns, axis, l * V, c, s);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const RopeSide &side = p.side[q];
            const int lo = q ? max(from - passes_q, 0) : min(from, passes_q), hi = q ? max(to - passes_q, 0) : min(to, passes_q);
            if (lo >= hi) continue;
            float wa[V], wb[V];
            rope_weights<kBf16, V, kInterleaved>(side.w, p.weight_f32, p.dim, unit, wa, wb);
            for (int pass = lo; pass < hi; ++pass) {
                const int head = pass * kRows + row;
                const bool there = head < side.heads;
                const bool in[2] = {there && is[0], there && is[1]};
                const long long h = there ? head : 0;
                RopeRaw<V> rx, rg;
                rope_read<V>(rg, side.g + token * side.g_token + h * side.g_head, unit, in);
                if (p.norm) rope_read<V>(rx, side.x + token * side.x_token + h * side.x_head, unit, in);
                float a[V], b[V], x[V], y[V];
                rope_split<kBf16, V, kInterleaved>(rg, a, b);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = a[i] * c[i] + b[i] * s[i];
                    b[i] = b[i] * c[i] - a[i] * s[i];
                    a[i] = f;
                }
                if (p.norm) {
                    rope_split<kBf16, V, kInterleaved>(rx, x, y);
                    float sum = 0.0f, dot = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
                        dot = fmaf(a[i] * wa[i], x[i], fmaf(b[i] * wb[i], y[i], dot));
                    }
                    sum = rope_sum<kLanes>(sum);
                    dot = rope_sum<kLanes>(dot);
                    const float r = rsqrtf(fmaf(sum, inv_dim, p.eps)), back = r * r * dot * inv_dim;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        da[q][i] = fmaf(a[i], x[i] * r, da[q][i]);
                        db[q][i] = fmaf(b[i], y[i] * r, db[q][i]);
                        a[i] = r * fmaf(-x[i], back, a[i] * wa[i]);
                        b[i] = r * fmaf(-y[i], back, b[i] * wb[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        a[i] *= wa[i];
                        b[i] *= wb[i];
                    }
                }
                const long long at = token * side.y_token + h * side.y_head;
                if (there && TGEMM_CHECK(at + 2 * p.dim <= p.dbg_y[q], kChkRope, p.status))
                    rope_write<kBf16, V, kInterleaved>(side.y + at, a, b, unit, in);
            }
        }
    }
    if (!p.partials) return;
    // The block's sums of the weight gradients: rows of a warp, then the warps.
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = j ? db[q][i] : da[q][i];
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                const int e = rope_element<V, kInterleaved>(i, j, unit);
                if (row == 0 && e < p.dim) s_dw[warp][q][e] = x;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += kRopeThreads) {
        const int q = i >= p.dim, e = i - q * p.dim;
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += s_dw[w][q][e];
        p.partials[static_cast<long long>(blockIdx.x) * 2 * p.dim + i] = x;
    }
}

// Adds the blocks' sums up in a fixed order, 32 columns a block.
__global__ void __launch_bounds__(kRopeThreads) rope_weight_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kWarps = kRopeThreads / 32;
    __shared__ float s_sum[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = static_cast<int>(blockIdx.x) * 32 + lane;
    griddep_wait();
    griddep_launch_dependents();
    float x = 0.0f;
    if (col < 2 * p.dim) {
#pragma unroll 8
        for (int b = warp; b < p.blocks; b += kWarps) x += p.partials[static_cast<long long>(b) * 2 * p.dim + col];
    }
    s_sum[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && col < 2 * p.dim) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_sum[w][lane];
        const int q = col >= p.dim;
        float *const dw = p.side[q].dw;
        if (dw) dw[col - q * p.dim] = sum;
    }
}

}  // namespace tgemm
