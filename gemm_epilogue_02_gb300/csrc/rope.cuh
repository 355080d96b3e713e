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
constexpr int kRopeBackThreads = 128, kRopeBackCtas = 3;     // per SM
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
    int norm, weight_f32, shift, dim, pairs, axes;
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

// The weights in shared memory, as each lane of a row takes them: 16 bytes of lane l at [chunk][l].
template <int V, int kLanes>
struct RopeWeights {
    float4 part[2 * V / 4][kLanes];
};

template <bool kBf16, int V, int kLanes, bool kInterleaved, int kThreads = kRopeThreads>
__device__ __forceinline__ void rope_stage_weights(RopeWeights<V, kLanes> &to, const void *w, bool f32, int dim, int pairs) {
    for (int i = threadIdx.x; i < 2 * V * kLanes; i += kThreads) {
        const int l = i / (2 * V), k = i - l * (2 * V);              // lane l's a[0 .. V - 1], then b
        int unit[2];
        bool is[2];
        rope_units<V, kInterleaved>(l, dim, pairs, unit, is);
        const int j = k / V, at = k - j * V;
        const int e = kInterleaved ? (at / (V / 2) ? unit[1] : unit[0]) * V + 2 * (at % (V / 2)) + j : (j ? unit[1] : unit[0]) * V + at;
        float x = 1.0f;
        if (w && e < dim) {
            if (f32) x = static_cast<const float *>(w)[e];
            else if (kBf16) x = __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[e]);
            else x = __half2float(static_cast<const __half *>(w)[e]);
        }
        reinterpret_cast<float *>(&to.part[k / 4][l])[k % 4] = x;
    }
}

// chunk k of lane l: weights 4 k .. 4 k + 3 of its a and b in a row
template <int V, int kLanes>
__device__ __forceinline__ void rope_weights(const RopeWeights<V, kLanes> &from, int l, float (&a)[V], float (&b)[V]) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
        const float4 x = from.part[k][l], y = from.part[V / 4 + k][l];
        a[4 * k] = x.x, a[4 * k + 1] = x.y, a[4 * k + 2] = x.z, a[4 * k + 3] = x.w;
        b[4 * k] = y.x, b[4 * k + 1] = y.y, b[4 * k + 2] = y.z, b[4 * k + 3] = y.w;
    }
}

template <int N>
__device__ __forceinline__ float rope_sum(float x) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The angles of a token's pairs.  The rows of a warp belong to one token, so each
// of their lanes works out kOwn of the row's pairs and takes the others from the
// lanes of the other rows.
template <int V, int kLanes>
struct RopeAngles {
    static constexpr int kRows = 32 / kLanes, kOwn = V / kRows;
    static_assert(kOwn >= 1 && kOwn * kRows == V, "a lane's pairs");
    unsigned long long turns[kOwn];
    int axis[kOwn];
    int first;                              // of the lane's own pairs

    __device__ __forceinline__ void init(const RopeParams &p, int l, int row) {
        first = l * V + row * kOwn;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int at = min(first + j, kRopePairs - 1);
            turns[j] = p.turns[at];         // 0 past the last pair: turned by nothing
            axis[j] = p.axis[at];
        }
    }
    // places: lane a's position on axis a
    __device__ __forceinline__ void turn(int places, int shift, int l, float (&c)[V], float (&s)[V]) const {
        float oc[kOwn], os[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const long long pos = static_cast<long long>(__shfl_sync(0xffffffffu, places, axis[j])) + shift;
            const unsigned long long t = static_cast<unsigned long long>(pos) * turns[j];
            sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, &os[j], &oc[j]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = __shfl_sync(0xffffffffu, oc[i % kOwn], i / kOwn * kLanes + l);
            s[i] = __shfl_sync(0xffffffffu, os[i % kOwn], i / kOwn * kLanes + l);
        }
    }
};

// Work.  A pass is 32 / kLanes rows, of one token's queries or of its keys, for a
// warp; the passes of all tokens in a row are cut into equal runs, one a warp.
struct RopeCursor {
    long long token;
    int pass;
};

// Passes ahead of the one at hand whose rows are on their way.
template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kWarps = kRopeThreads / 32, kAhead = 3;
    __shared__ RopeWeights<V, kLanes> s_w[2];
    const int lane = threadIdx.x & 31, l = lane % kLanes, row = lane / kLanes;
    int unit[2];
    bool is[2];
    rope_units<V, kInterleaved>(l, p.dim, p.pairs, unit, is);
    RopeAngles<V, kLanes> angles;
    angles.init(p, l, row);
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const int passes_q = (p.side[0].heads + kRows - 1) / kRows, passes = passes_q + (p.side[1].heads + kRows - 1) / kRows;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps, warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long all = p.tokens * passes, begin = warp * all / warps;
    int left = static_cast<int>((warp + 1) * all / warps - begin);
    RopeCursor use, load;
    use.token = begin / passes;
    use.pass = static_cast<int>(begin - use.token * passes);
    load = use;
    griddep_wait();
    griddep_launch_dependents();
    auto next = [&](RopeCursor &u) {
        if (++u.pass == passes) {
            u.pass = 0;
            ++u.token;
        }
    };
    int loads = left;
    RopeRaw<V> ring[kAhead];
    auto request = [&](RopeRaw<V> &raw) {
        const bool q = load.pass >= passes_q;
        const RopeSide &side = p.side[q ? 1 : 0];
        const int head = (load.pass - (q ? passes_q : 0)) * kRows + row;
        const bool there = loads > 0 && head < side.heads;
        const bool in[2] = {there && is[0], there && is[1]};
        rope_read<V>(raw, side.x + load.token * side.x_token + (there ? head : 0) * side.x_head, unit, in);
        if (--loads > 0) next(load);
    };
    auto places_of = [&](long long token) {
        return lane < p.axes && token < p.tokens ? p.positions[lane * p.axis_stride + token] : 0;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) request(ring[i]);
    int places = places_of(use.token);
    rope_stage_weights<kBf16, V, kLanes, kInterleaved>(s_w[0], p.side[0].w, p.weight_f32, p.dim, p.pairs);
    rope_stage_weights<kBf16, V, kLanes, kInterleaved>(s_w[1], p.side[1].w, p.weight_f32, p.dim, p.pairs);
    __syncthreads();
    float c[V], s[V];
    bool fresh = true;                      // the token's angles are to be worked out
    // A slot of the ring is refilled as soon as it is unpacked: moving rows that are on their way would wait for them.
    auto step = [&](RopeRaw<V> &raw) {
        if (fresh) {
            angles.turn(places, p.shift, l, c, s);
            places = places_of(use.token + 1);
        }
        float a[V], b[V], wa[V], wb[V];
        rope_split<kBf16, V, kInterleaved>(raw, a, b);
        request(raw);
        const bool q = use.pass >= passes_q;
        const RopeSide &side = p.side[q ? 1 : 0];
        const int head = (use.pass - (q ? passes_q : 0)) * kRows + row;
        rope_weights(s_w[q ? 1 : 0], l, wa, wb);
        float r = 1.0f;
        if (p.norm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
            r = rsqrtf(fmaf(rope_sum<kLanes>(sum), inv_dim, p.eps));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float f = a[i] * r * wa[i], g = b[i] * r * wb[i];
            a[i] = f * c[i] - g * s[i];
            b[i] = g * c[i] + f * s[i];
        }
        const bool there = head < side.heads;
        const bool in[2] = {there && is[0], there && is[1]};
        const long long at = use.token * side.y_token + (there ? head : 0) * side.y_head;
        if (there && TGEMM_CHECK(at + 2 * p.dim <= p.dbg_y[q ? 1 : 0], kChkRope, p.status))
            rope_write<kBf16, V, kInterleaved>(side.y + at, a, b, unit, in);
        const long long token = use.token;
        next(use);
        fresh = use.token != token;
    };
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (left-- > 0) step(ring[i]);
    }
}

template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeBackThreads, kRopeBackCtas) rope_backward_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kWarps = kRopeBackThreads / 32, kAhead = 2;
    __shared__ RopeWeights<V, kLanes> s_w[2];
    __shared__ float s_dw[kWarps][2][2 * kRopePairs];
    const int lane = threadIdx.x & 31, l = lane % kLanes, row = lane / kLanes;
    int unit[2];
    bool is[2];
    rope_units<V, kInterleaved>(l, p.dim, p.pairs, unit, is);
    RopeAngles<V, kLanes> angles;
    angles.init(p, l, row);
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const int passes_q = (p.side[0].heads + kRows - 1) / kRows, passes = passes_q + (p.side[1].heads + kRows - 1) / kRows;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps, warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long all = p.tokens * passes, begin = warp * all / warps;
    int left = static_cast<int>((warp + 1) * all / warps - begin);
    RopeCursor use, load;
    use.token = passes > 0 ? begin / passes : 0;
    use.pass = passes > 0 ? static_cast<int>(begin - use.token * passes) : 0;
    load = use;
    griddep_wait();
    griddep_launch_dependents();
    auto next = [&](RopeCursor &u) {
        if (++u.pass == passes) {
            u.pass = 0;
            ++u.token;
        }
    };
    int loads = left;
    RopeRaw<V> ring_x[kAhead], ring_g[kAhead];
    auto request = [&](RopeRaw<V> &next_x, RopeRaw<V> &next_g) {
        const bool q = load.pass >= passes_q;
        const RopeSide &side = p.side[q ? 1 : 0];
        const int head = (load.pass - (q ? passes_q : 0)) * kRows + row;
        const bool there = loads > 0 && head < side.heads;
        const bool in[2] = {there && is[0], there && is[1]};
        const bool x_in[2] = {in[0] && p.norm, in[1] && p.norm};
        rope_read<V>(next_g, side.g + load.token * side.g_token + (there ? head : 0) * side.g_head, unit, in);
        rope_read<V>(next_x, side.x + load.token * side.x_token + (there ? head : 0) * side.x_head, unit, x_in);
        if (--loads > 0) next(load);
    };
    auto places_of = [&](long long token) {
        return lane < p.axes && token < p.tokens ? p.positions[lane * p.axis_stride + token] : 0;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) request(ring_x[i], ring_g[i]);
    int places = places_of(use.token);
    rope_stage_weights<kBf16, V, kLanes, kInterleaved, kRopeBackThreads>(s_w[0], p.side[0].w, p.weight_f32, p.dim, p.pairs);
    rope_stage_weights<kBf16, V, kLanes, kInterleaved, kRopeBackThreads>(s_w[1], p.side[1].w, p.weight_f32, p.dim, p.pairs);
    __syncthreads();
    float da[2][V], db[2][V];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) da[q][i] = db[q][i] = 0.0f;
    float c[V], s[V];
    bool fresh = true;                      // the token's angles are to be worked out
    auto step = [&](RopeRaw<V> &raw_x, RopeRaw<V> &raw_g, float (&da)[V], float (&db)[V], const RopeWeights<V, kLanes> &weights,
                    const RopeSide &side, int pass, long long dbg) {
        float a[V], b[V], x[V], y[V];
        rope_split<kBf16, V, kInterleaved>(raw_g, a, b);
        rope_split<kBf16, V, kInterleaved>(raw_x, x, y);
        request(raw_x, raw_g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float f = a[i] * c[i] + b[i] * s[i];
            b[i] = b[i] * c[i] - a[i] * s[i];
            a[i] = f;
        }
        if (p.norm) {
            float sum = 0.0f, dot = 0.0f;
            {
                float wa[V], wb[V];
                rope_weights(weights, l, wa, wb);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
                    dot = fmaf(a[i] * wa[i], x[i], fmaf(b[i] * wb[i], y[i], dot));
                }
            }
            sum = rope_sum<kLanes>(sum);
            dot = rope_sum<kLanes>(dot);
            const float r = rsqrtf(fmaf(sum, inv_dim, p.eps)), back = r * r * dot * inv_dim;
            float wa[V], wb[V];
            rope_weights(weights, l, wa, wb);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                da[i] = fmaf(a[i], x[i] * r, da[i]);
                db[i] = fmaf(b[i], y[i] * r, db[i]);
                a[i] = r * fmaf(-x[i], back, a[i] * wa[i]);
                b[i] = r * fmaf(-y[i], back, b[i] * wb[i]);
            }
        }
        const int head = pass * kRows + row;
        const bool there = head < side.heads;
        const bool in[2] = {there && is[0], there && is[1]};
        const long long at = use.token * side.y_token + (there ? head : 0) * side.y_head;
        if (there && TGEMM_CHECK(at + 2 * p.dim <= dbg, kChkRope, p.status))
            rope_write<kBf16, V, kInterleaved>(side.y + at, a, b, unit, in);
    };
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (left-- <= 0) break;
            if (fresh) {
                angles.turn(places, p.shift, l, c, s);
                places = places_of(use.token + 1);
            }
            if (use.pass < passes_q) step(ring_x[i], ring_g[i], da[0], db[0], s_w[0], p.side[0], use.pass, p.dbg_y[0]);
            else step(ring_x[i], ring_g[i], da[1], db[1], s_w[1], p.side[1], use.pass - passes_q, p.dbg_y[1]);
            const long long token = use.token;
            next(use);
            fresh = use.token != token;
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
                if (row == 0 && e < p.dim) s_dw[threadIdx.x >> 5][q][e] = x;
            }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.dim; i += kRopeBackThreads) {
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
