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
// Elements past the pairs are passed through.
//
// Reading and writing each row once bounds it.  Angles: a frequency is given in
// turns as a 64-bit fraction, so that position * frequency, which wraps at whole
// turns by itself, keeps 2^-31 of a turn at any 32-bit position; the upper 32
// bits then go through sincospi in fp32.  (fp32 angles are off by whole
// radians at far positions, fp64 runs at 1/64 of fp32's rate here.)
//
// What keeps the memory busy: a warp's lanes hold elements that turn with one
// another, so a row needs no exchange but that of its sum of squares, and the rows
// of the next passes are on their way while one is worked on.  24571 tokens of 32
// query and 8 key heads, 128 wide (504 MB): 85 us, 5.9 TB/s; with two passes ahead
// instead of three 87, with rows that move through registers 99, a token a warp and
// its angles worked out by every lane 112.  The gradient of 16384 tokens (503 MB)
// 91 us: one block of 12 warps an SM, two passes ahead (four blocks of 4 warps and
// one pass 96; without a pass ahead 236, its registers leaving 8 warps).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "debug_checks.cuh"
#include "fp32x2.cuh"
#include "ptx.cuh"

namespace tgemm {

constexpr int kRopePairs = 128;             // at most (dim 256)
constexpr int kRopeThreads = 256;
constexpr int kRopeBackThreads = 384, kRopeBackCtas = 1;     // per SM
constexpr int kRopeMaxBlocks = 1024;        // whose sums of weight gradients the workspace holds
constexpr int kRopeFan = 32;                // blocks' sums that are added up at once, at most
static_assert(kRopeMaxBlocks <= kRopeFan * kRopeFan, "two levels add up every block's sums");

struct RopeSide {
    const unsigned char *x, *g;             // rows, and (backward) gradients of what the forward pass wrote
    unsigned char *y;                       // what is written: rotated rows, or (backward) gradients of x
    const void *w;                          // null: ones
    float *dw;                              // null: not wanted
    long long x_token, x_head, g_token, g_head, y_token, y_head;     // bytes
    int heads;
};

struct RopeArray {
    unsigned char *base;
    long long token, head;
};

struct RopeParams {
    RopeSide side[2];                       // queries, keys
    const int *positions;                   // [axes, tokens]
    long long axis_stride, tokens;
    // The workspace (null: no weight gradients are wanted): arrivals, zero between calls; sums of the blocks and of groups
    // of them, [kRopeMaxBlocks + kRopeFan][2][dim].
    unsigned *arrivals;                     // [kRopeFan + 1]
    float *partials;
    float eps;
    int norm, weight_f32, shift, dim, pairs, axes;
    int fan;                                // blocks of a group
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

// Chunk k of lane l: weights 4 k .. 4 k + 3 of its a, then of its b.
template <int V, int kLanes>
__device__ __forceinline__ void rope_weights(const RopeWeights<V, kLanes> &from, int l, float2 (&a)[V / 2], float2 (&b)[V / 2]) {
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
        const float4 x = from.part[k][l], y = from.part[V / 4 + k][l];
        a[2 * k] = make_float2(x.x, x.y), a[2 * k + 1] = make_float2(x.z, x.w);
        b[2 * k] = make_float2(y.x, y.y), b[2 * k + 1] = make_float2(y.z, y.w);
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
    __device__ __forceinline__ void turn(int places, int shift, int l, float2 (&c)[V / 2], float2 (&s)[V / 2]) const {
        float oc[kOwn], os[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const long long pos = static_cast<long long>(__shfl_sync(0xffffffffu, places, axis[j])) + shift;
            const unsigned long long t = static_cast<unsigned long long>(pos) * turns[j];
            sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, &os[j], &oc[j]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = __shfl_sync(0xffffffffu, oc[i % kOwn], i / kOwn * kLanes + l);
            const float y = __shfl_sync(0xffffffffu, os[i % kOwn], i / kOwn * kLanes + l);
            (i % 2 ? c[i / 2].y : c[i / 2].x) = x;
            (i % 2 ? s[i / 2].y : s[i / 2].x) = y;
        }
    }
};

// The rows turned (kBack: turned back): slot i of a lane's pairs by the angle whose
// cosine and sine are c and s.  The first `turning` slots are pairs of the
// rotation.  What is past them is kept as it is: a product with a sine of 0 would
// carry an infinity or a NaN to the other element, and lose the sign of a zero.
template <int V, bool kInterleaved, bool kBack>
__device__ __forceinline__ void rope_turn(float2 (&a)[V / 2], float2 (&b)[V / 2], const float2 (&c)[V / 2], const float2 (&s)[V / 2],
                                          int turning) {
    if (turning <= 0) return;
    auto turn = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 minus = make_float2(-s[i].x, -s[i].y), ta = kBack ? s[i] : minus, tb = kBack ? minus : s[i];
            const float2 f = fma2(a[i], c[i], mul2(b[i], ta)), g = fma2(b[i], c[i], mul2(a[i], tb));
            if (whole() || 2 * i < turning) a[i].x = f.x, b[i].x = g.x;
            if (whole() || 2 * i + 1 < turning) a[i].y = f.y, b[i].y = g.y;
        }
    };
    // Pairs that lie apart fill a lane; of those side by side one lane may have both kinds.
    if (!kInterleaved || turning >= V) turn([] { return true; });
    else turn([] { return false; });
}

// Work.  A pass is 32 / kLanes rows, of one token's queries or of its keys, for a
// warp; the passes of all tokens in a row are cut into equal runs, one a warp.
// N arrays of rows are followed together (addresses of the lane's row).
template <int kRows, int N>
struct RopeCursor {
    long long token;
    int side, left, head;                   // passes of the side that are left, this one among them; the lane's row
    unsigned char *at[N];

    // array(side, i): base and strides of array i
    template <typename Array>
    __device__ __forceinline__ void enter(const RopeParams &p, int row, int pass, Array array) {
        left = (p.side[side].heads + kRows - 1) / kRows - pass;
        head = pass * kRows + row;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const RopeArray a = array(p.side[side], i);
            at[i] = a.base + token * a.token + static_cast<long long>(head) * a.head;
        }
    }
    template <typename Array>
    __device__ __forceinline__ void begin(const RopeParams &p, long long pass, int passes_q, int passes, int row, Array array) {
        token = passes > 0 ? pass / passes : 0;
        int in = passes > 0 ? static_cast<int>(pass - token * passes) : 0;
        side = in >= passes_q ? 1 : 0;
        enter(p, row, in - (side ? passes_q : 0), array);
    }
    // The next pass there is; true when it is another token's.
    template <typename Array>
    __device__ __forceinline__ bool next(const RopeParams &p, int row, Array array) {
        if (--left > 0) {
            head += kRows;
#pragma unroll
            for (int i = 0; i < N; ++i) at[i] += kRows * array(p.side[side], i).head;
            return false;
        }
        const int heads = p.side[1 - side].heads;
        const bool other = side == 1 || heads == 0;
        if (other) ++token;
        if (heads > 0) side = 1 - side;
        enter(p, row, 0, array);
        return other;
    }
};

template <bool kBf16, int V, bool kInterleaved>
__device__ __forceinline__ void rope_split2(const RopeRaw<V> &raw, float2 (&a)[V / 2], float2 (&b)[V / 2]) {
    float x[V], y[V];
    rope_split<kBf16, V, kInterleaved>(raw, x, y);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        a[i] = make_float2(x[2 * i], x[2 * i + 1]);
        b[i] = make_float2(y[2 * i], y[2 * i + 1]);
    }
}
template <bool kBf16, int V, bool kInterleaved>
__device__ __forceinline__ void rope_write2(unsigned char *row, const float2 (&a)[V / 2], const float2 (&b)[V / 2], const int (&unit)[2],
                                            const bool (&is)[2]) {
    float x[V], y[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = a[i].x, x[2 * i + 1] = a[i].y;
        y[2 * i] = b[i].x, y[2 * i + 1] = b[i].y;
    }
    rope_write<kBf16, V, kInterleaved>(row, x, y, unit, is);
}

template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kWarps = kRopeThreads / 32, kAhead = 3;     // passes whose rows are on their way
    __shared__ RopeWeights<V, kLanes> s_w[2];
    const int lane = threadIdx.x & 31, l = lane % kLanes, row = lane / kLanes;
    int unit[2];
    bool is[2];
    rope_units<V, kInterleaved>(l, p.dim, p.pairs, unit, is);
    RopeAngles<V, kLanes> angles;
    angles.init(p, l, row);
    const int turning = p.pairs - l * V;    // of the lane's pairs: V or more, all
    const float inv_dim = 1.0f / static_cast<float>(p.dim);
    const int passes_q = (p.side[0].heads + kRows - 1) / kRows, passes = passes_q + (p.side[1].heads + kRows - 1) / kRows;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps, warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const long long all = p.tokens * passes, begin = warp * all / warps;
    int left = static_cast<int>((warp + 1) * all / warps - begin), loads = left;
    auto inputs = [](const RopeSide &s, int) { return RopeArray{const_cast<unsigned char *>(s.x), s.x_token, s.x_head}; };
    auto outputs = [](const RopeSide &s, int) { return RopeArray{s.y, s.y_token, s.y_head}; };
    RopeCursor<kRows, 1> load, use;
    load.begin(p, begin, passes_q, passes, row, inputs);
    use.begin(p, begin, passes_q, passes, row, outputs);
    griddep_wait();
    griddep_launch_dependents();
    RopeRaw<V> ring[kAhead];
    auto request = [&](RopeRaw<V> &raw) {
        const bool there = loads > 0 && load.head < p.side[load.side].heads;
        const bool in[2] = {there && is[0], there && is[1]};
        rope_read<V>(raw, load.at[0], unit, in);
        if (--loads > 0) load.next(p, row, inputs);
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
    float2 c[V / 2], s[V / 2];
    bool fresh = true;                      // the token's angles are to be worked out
    // A slot of the ring is refilled as soon as it is unpacked: moving rows that are on their way would wait for them.
    auto step = [&](RopeRaw<V> &raw) {
        if (fresh) {
            angles.turn(places, p.shift, l, c, s);
            places = places_of(use.token + 1);
        }
        float2 a[V / 2], b[V / 2], wa[V / 2], wb[V / 2];
        rope_split2<kBf16, V, kInterleaved>(raw, a, b);
        request(raw);
        rope_weights(s_w[use.side], l, wa, wb);
        float r = 1.0f;
        if (p.norm) {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) sum = fma2(a[i], a[i], fma2(b[i], b[i], sum));
            r = rsqrtf(fmaf(rope_sum<kLanes>(sum.x + sum.y), inv_dim, p.eps));
        }
        const float2 rr = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            a[i] = mul2(mul2(a[i], rr), wa[i]);
            b[i] = mul2(mul2(b[i], rr), wb[i]);
        }
        rope_turn<V, kInterleaved, false>(a, b, c, s, turning);
        const bool there = use.head < p.side[use.side].heads;
        const bool in[2] = {there && is[0], there && is[1]};
        if (there && TGEMM_CHECK(use.at[0] - p.side[use.side].y + 2 * p.dim <= p.dbg_y[use.side], kChkRope, p.status))
            rope_write2<kBf16, V, kInterleaved>(use.at[0], a, b, unit, in);
        fresh = left > 0 && use.next(p, row, outputs);
    };
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (left-- > 0) step(ring[i]);
    }
}

// Counts up to `last` and from there back to 0; returns the count before.  The
// block's writes before it (through a barrier) are visible to the blocks that
// count after it, and theirs before to this one.
__device__ __forceinline__ unsigned rope_count(unsigned *counter, unsigned last) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(counter), "r"(last) : "memory");
    return old;
}

template <bool kBf16, int V, int kLanes, bool kInterleaved>
__global__ void __launch_bounds__(kRopeBackThreads, kRopeBackCtas) rope_backward_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kRows = 32 / kLanes, kWarps = kRopeBackThreads / 32, kAhead = 2;
    __shared__ RopeWeights<V, kLanes> s_w[2];
    __shared__ float4 s_sum[2][kWarps][2 * (V / 4)][32];
    __shared__ bool s_last;
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
    int left = static_cast<int>((warp + 1) * all / warps - begin), loads = left;
    auto inputs = [](const RopeSide &s, int i) {
        return i ? RopeArray{const_cast<unsigned char *>(s.x), s.x_token, s.x_head}
                 : RopeArray{const_cast<unsigned char *>(s.g), s.g_token, s.g_head};
    };
    auto outputs = [](const RopeSide &s, int) { return RopeArray{s.y, s.y_token, s.y_head}; };
    RopeCursor<kRows, 2> load;
    RopeCursor<kRows, 1> use;
    load.begin(p, begin, passes_q, passes, row, inputs);
    use.begin(p, begin, passes_q, passes, row, outputs);
    griddep_wait();
    griddep_launch_dependents();
    RopeRaw<V> ring_x[kAhead], ring_g[kAhead];
    auto request = [&](RopeRaw<V> &next_x, RopeRaw<V> &next_g) {
        const bool there = loads > 0 && load.head < p.side[load.side].heads;
        const bool in[2] = {there && is[0], there && is[1]}, x_in[2] = {in[0] && p.norm, in[1] && p.norm};
        rope_read<V>(next_g, load.at[0], unit, in);
        rope_read<V>(next_x, load.at[1], unit, x_in);
        if (--loads > 0) load.next(p, row, inputs);
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
    // The weight gradients' sums of the side at hand; those of the other are in shared memory.
    float2 da[V / 2], db[V / 2];
    float4 *const mine = &s_sum[0][threadIdx.x >> 5][0][lane];
    auto fetch = [&](int side) {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) {
            const float4 x = mine[(side * kWarps * 2 * (V / 4) + k) * 32], y = mine[(side * kWarps * 2 * (V / 4) + V / 4 + k) * 32];
            da[2 * k] = make_float2(x.x, x.y), da[2 * k + 1] = make_float2(x.z, x.w);
            db[2 * k] = make_float2(y.x, y.y), db[2 * k + 1] = make_float2(y.z, y.w);
        }
    };
    auto store = [&](int side) {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) {
            mine[(side * kWarps * 2 * (V / 4) + k) * 32] = make_float4(da[2 * k].x, da[2 * k].y, da[2 * k + 1].x, da[2 * k + 1].y);
            mine[(side * kWarps * 2 * (V / 4) + V / 4 + k) * 32] = make_float4(db[2 * k].x, db[2 * k].y, db[2 * k + 1].x, db[2 * k + 1].y);
        }
    };
#pragma unroll
    for (int i = 0; i < V / 2; ++i) da[i] = db[i] = make_float2(0.0f, 0.0f);
    store(0);
    store(1);
    int side_at_hand = 0;
    float2 c[V / 2], s[V / 2];
    bool fresh = true;                      // the token's angles are to be worked out
    auto step = [&](RopeRaw<V> &raw_x, RopeRaw<V> &raw_g) {
        const RopeSide &side = p.side[use.side];
        const RopeWeights<V, kLanes> &weights = s_w[use.side];
        float2 a[V / 2], b[V / 2], x[V / 2], y[V / 2];
        rope_split2<kBf16, V, kInterleaved>(raw_g, a, b);
        rope_split2<kBf16, V, kInterleaved>(raw_x, x, y);
        request(raw_x, raw_g);
        // (from the thread's number each time: with one register more the kernel spills)
        rope_turn<V, kInterleaved, true>(a, b, c, s, p.pairs - static_cast<int>(threadIdx.x) % kLanes * V);
        const bool there = use.head < side.heads;
        if (p.norm) {
            float2 sums = make_float2(0.0f, 0.0f), dots = make_float2(0.0f, 0.0f);
            {
                float2 wa[V / 2], wb[V / 2];
                rope_weights(weights, l, wa, wb);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    sums = fma2(x[i], x[i], fma2(y[i], y[i], sums));
                    dots = fma2(mul2(a[i], wa[i]), x[i], fma2(mul2(b[i], wb[i]), y[i], dots));
                }
            }
            const float sum = rope_sum<kLanes>(sums.x + sums.y), dot = rope_sum<kLanes>(dots.x + dots.y);
            // A row past the last head has no part in the weights' gradients, whatever eps is.
            const float r = there ? rsqrtf(fmaf(sum, inv_dim, p.eps)) : 0.0f, back = -r * (dot * inv_dim);
            const float2 rr = make_float2(r, r), bb = make_float2(back, back);
            float2 wa[V / 2], wb[V / 2];
            rope_weights(weights, l, wa, wb);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                // (x r and r dot stay in fp32's range where r^2 does not)
                x[i] = mul2(x[i], rr);
                y[i] = mul2(y[i], rr);
                da[i] = fma2(a[i], x[i], da[i]);
                db[i] = fma2(b[i], y[i], db[i]);
                a[i] = mul2(rr, fma2(x[i], bb, mul2(a[i], wa[i])));
                b[i] = mul2(rr, fma2(y[i], bb, mul2(b[i], wb[i])));
            }
        }
        const bool in[2] = {there && is[0], there && is[1]};
        if (there && TGEMM_CHECK(use.at[0] - side.y + 2 * p.dim <= p.dbg_y[use.side], kChkRope, p.status))
            rope_write2<kBf16, V, kInterleaved>(use.at[0], a, b, unit, in);
    };
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (left-- <= 0) break;
            if (fresh) {
                angles.turn(places, p.shift, l, c, s);
                places = places_of(use.token + 1);
            }
            if (use.side != side_at_hand) {
                store(side_at_hand);
                side_at_hand = use.side;
                fetch(side_at_hand);
            }
            step(ring_x[i], ring_g[i]);
            fresh = left > 0 && use.next(p, row, outputs);
        }
    }
    if (!p.partials) return;
    // The block's sums of the weight gradients, over the warps and the rows of each.
    store(side_at_hand);
    __syncthreads();
    const int width = 2 * p.dim;
    float *const own = p.partials + static_cast<long long>(blockIdx.x) * width;
    for (int i = threadIdx.x; i < 2 * kLanes * 2 * V; i += kRopeBackThreads) {
        const int q = i / (kLanes * 2 * V), at = i - q * (kLanes * 2 * V), lane_of = at / (2 * V), k = at - lane_of * (2 * V);
        int u[2];
        bool in[2];
        rope_units<V, kInterleaved>(lane_of, p.dim, p.pairs, u, in);
        const int e = rope_element<V, kInterleaved>(k % V, k / V, u);
        if (e >= p.dim) continue;
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
#pragma unroll
            for (int r = 0; r < kRows; ++r) x += reinterpret_cast<const float *>(&s_sum[q][w][k / 4][r * kLanes + lane_of])[k % 4];
        own[q * p.dim + e] = x;
    }
    // The last block of a group to arrive adds the group's sums up, the last group those of all: in a fixed order, whoever
    // is last.
    const int blocks = static_cast<int>(gridDim.x), group = static_cast<int>(blockIdx.x) / p.fan, first = group * p.fan;
    const int members = min(p.fan, blocks - first), groups = (blocks + p.fan - 1) / p.fan;
    auto arrive = [&](unsigned *counter, int count) {
        __syncthreads();
        if (threadIdx.x == 0) s_last = rope_count(counter, static_cast<unsigned>(count - 1)) == static_cast<unsigned>(count - 1);
        __syncthreads();
        return s_last;
    };
    auto total = [&](const float *rows, int count, int column) {
        float x = 0.0f;
#pragma unroll 8
        for (int r = 0; r < count; ++r) x += __ldcg(rows + static_cast<long long>(r) * width + column);
        return x;
    };
    if (!arrive(p.arrivals + group, members)) return;
    const float *rows = p.partials + static_cast<long long>(first) * width;
    float *const all_groups = p.partials + static_cast<long long>(kRopeMaxBlocks) * width;
    if (groups > 1) {
        for (int i = threadIdx.x; i < width; i += kRopeBackThreads) all_groups[static_cast<long long>(group) * width + i] = total(rows, members, i);
        if (!arrive(p.arrivals + kRopeFan, groups)) return;
        rows = all_groups;
    }
    for (int i = threadIdx.x; i < width; i += kRopeBackThreads) {
        const int q = i >= p.dim, e = i - q * p.dim;
        if (p.side[q].dw) p.side[q].dw[e] = total(rows, groups > 1 ? groups : members, i);
    }
}

}  // namespace tgemm
