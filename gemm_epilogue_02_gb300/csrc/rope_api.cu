// C-ABI of the head norms with the position rotation, and their gradient
// (declarations and contract in include/tgemm.h): argument validation and the
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstring>

#include "../../include/tgemm.h"
#include "kv_host.h"
#include "rope.cuh"
#include "runtime.h"

namespace tgemm {
namespace {

// A strided array of rows of heads: [tokens, heads, dim].
struct Rows {
    const unsigned char *base = nullptr;
    int64_t token = 0, head = 0, heads = 0;      // strides in bytes
    int64_t inner = 0, bytes = 0;                // of one token's heads; of all
};

tgemm_status check_rows(const tgemm_rows &r, int64_t tokens, int64_t heads, int64_t dim, bool written, Rows *out) {
    if (tokens == 0 || heads == 0) {             // whatever the strides are
        out->heads = heads;
        return TGEMM_OK;
    }
    const int64_t size[2] = {tokens, heads}, stride[2] = {r.token_stride, r.head_stride};
    const int64_t inner_size[1] = {heads}, inner_stride[1] = {r.head_stride};
    if (!extent(size, stride, 2, dim, 2, written, &out->bytes) || !extent(inner_size, inner_stride, 1, dim, 2, written, &out->inner))
        return TGEMM_ERR_INVALID_ARG;
    if (written && rows_meet(size, stride, dim)) return TGEMM_ERR_ALIAS;
    if (out->bytes > 0) {
        if (!r.data) return TGEMM_ERR_INVALID_ARG;
        if (!aligned16(r.data) || (tokens > 1 && r.token_stride % 8 != 0) || (heads > 1 && r.head_stride % 8 != 0))
            return TGEMM_ERR_ALIGNMENT;
    }
    out->base = static_cast<const unsigned char *>(r.data);
    out->token = r.token_stride * 2;
    out->head = r.head_stride * 2;
    out->heads = heads;
    return TGEMM_OK;
}

// Whether what is written through `a` may touch what is read or written through `b`.  Rows of one token side by side in
// one array (a projection's output) lie apart; the same rows may be replaced in place.
bool clash(const Rows &a, const Rows &b, bool in_place) {
    if (!overlaps({a.base, a.bytes}, {b.base, b.bytes})) return false;
    if (in_place && a.base == b.base && a.token == b.token && a.head == b.head && a.heads == b.heads) return false;
    if (a.token != b.token || a.token <= 0 || a.inner > a.token || b.inner > b.token) return true;
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
    const int64_t m = ((d % a.token) + a.token) % a.token;         // b's first byte after a's, modulo a token
    return m < a.inner || m + b.inner > a.token;
}

int lanes_of(int64_t dim, int v) {
    const int64_t units = (dim / v + 1) / 2;
    if (v == 8) return units <= 4 ? 4 : units <= 8 ? 8 : 16;
    return units <= 8 ? 8 : units <= 16 ? 16 : 32;
}

// What both calls check; fills the parameters that they share.
tgemm_status check_common(const tgemm_qk_norm_rope_args *a, RopeParams *p, int *v, bool *interleaved) {
    const tgemm_rotary *r = a->rotary;
    if (a->tokens < 0 || a->tokens > INT32_MAX || a->q_heads < 0 || a->k_heads < 0 || a->q_heads > 65535 || a->k_heads > 65535 ||
        a->dim < 8 || a->dim > 2 * kRopePairs || a->dim % 8 != 0 || !valid_dtype(a->dtype) || (a->norm != 0 && a->norm != 1) ||
        (a->weight_f32 != 0 && a->weight_f32 != 1) || a->shift < INT32_MIN || a->shift > INT32_MAX || a->axes < 0 || a->axes > 32)
        return TGEMM_ERR_INVALID_ARG;
    if (a->norm ? !(a->eps >= 0.0) || a->eps > FLT_MAX : (a->q_weight || a->k_weight)) return TGEMM_ERR_INVALID_ARG;
    if (!a->norm && !r) return TGEMM_ERR_INVALID_ARG;
    *v = 8;
    *interleaved = false;
    if (r) {
        if (r->pairs < 0 || 2 * r->pairs > a->dim || (r->interleaved != 0 && r->interleaved != 1) || (r->pairs > 0 && !r->turns) ||
            (!r->interleaved && r->pairs % 4 != 0) || (r->pairs > 0 && a->axes < 1))
            return TGEMM_ERR_INVALID_ARG;
        *interleaved = r->interleaved != 0;
        if (!r->interleaved && r->pairs % 8 != 0) *v = 4;
        p->pairs = static_cast<int>(r->pairs);
        for (int i = 0; i < p->pairs; ++i) {
            p->turns[i] = r->turns[i];
            const int32_t axis = r->axes ? r->axes[i] : 0;
            if (axis < 0 || axis >= a->axes) return TGEMM_ERR_INVALID_ARG;
            p->axis[i] = static_cast<unsigned char>(axis);
        }
        if (a->axis_stride < 0 || a->axis_stride > (int64_t(1) << 40)) return TGEMM_ERR_INVALID_ARG;      // 0: the axes share positions
        if (p->pairs > 0 && a->tokens > 0 && !a->positions) return TGEMM_ERR_INVALID_ARG;
    }
    const int weight = a->weight_f32 ? 4 : 2;
    if (!aligned4(a->positions) || reinterpret_cast<uintptr_t>(a->q_weight) % weight || reinterpret_cast<uintptr_t>(a->k_weight) % weight)
        return TGEMM_ERR_ALIGNMENT;
    p->positions = a->positions;
    p->axes = r && r->pairs > 0 ? static_cast<int>(a->axes) : 0;
    p->axis_stride = a->axis_stride;
    p->tokens = a->tokens;
    p->dim = static_cast<int>(a->dim);
    p->shift = static_cast<int>(a->shift);
    p->norm = static_cast<int>(a->norm);
    p->weight_f32 = static_cast<int>(a->weight_f32);
    // (an eps that fp32 rounds to 0 still keeps rows of zeros what they are)
    p->eps = a->eps > 0.0 ? std::max(static_cast<float>(a->eps), FLT_TRUE_MIN) : 0.0f;
    return TGEMM_OK;
}

// The small arrays that a call reads, to e[0 .. 2].
void small_inputs(const tgemm_qk_norm_rope_args *a, Extent *e) {
    const int64_t w = a->dim * (a->weight_f32 ? 4 : 2);
    e[0] = {a->q_weight, a->q_weight ? w : 0};
    e[1] = {a->k_weight, a->k_weight ? w : 0};
    e[2] = {a->positions, a->positions && a->rotary && a->rotary->pairs > 0 ? ((a->axes - 1) * a->axis_stride + a->tokens) * 4 : 0};
}

void set_side(RopeSide &s, const Rows &x, const Rows &y, const Rows *g, const void *w) {
    s.x = x.base;
    s.x_token = x.token;
    s.x_head = x.head;
    s.y = const_cast<unsigned char *>(y.base);
    s.y_token = y.token;
    s.y_head = y.head;
    if (g) {
        s.g = g->base;
        s.g_token = g->token;
        s.g_head = g->head;
    }
    s.w = w;
    s.heads = static_cast<int>(x.heads);
}

// A warp a pass, or as many blocks as fit the GPU at once.
unsigned rope_blocks(const RopeParams &p, int lanes, int threads, int64_t most) {
    const int rows = 32 / lanes;
    const int64_t passes = (p.side[0].heads + rows - 1) / rows + (p.side[1].heads + rows - 1) / rows;
    const int64_t blocks = (p.tokens * passes + threads / 32 - 1) / (threads / 32);
    return static_cast<unsigned>(std::max<int64_t>(1, std::min(blocks, most)));
}

template <bool kBf16, int V, int kLanes, bool kInterleaved>
cudaError_t launch_rope(const RuntimeInfo &rt, RopeParams &p, bool backward, cudaStream_t s) {
    if (!backward)
        return launch(rope_kernel<kBf16, V, kLanes, kInterleaved>, dim3(rope_blocks(p, kLanes, kRopeThreads, static_cast<int64_t>(rt.num_sms) * 2)),
                      kRopeThreads, 0, s, p);
    const unsigned blocks =
        rope_blocks(p, kLanes, kRopeBackThreads, std::min<int64_t>(kRopeMaxBlocks, static_cast<int64_t>(rt.num_sms) * kRopeBackCtas));
    p.fan = 1;
    while (p.fan * p.fan < static_cast<int>(blocks)) ++p.fan;
    return launch(rope_backward_kernel<kBf16, V, kLanes, kInterleaved>, dim3(blocks), kRopeBackThreads, 0, s, p);
}

template <bool kBf16>
cudaError_t launch_rope_shape(const RuntimeInfo &rt, RopeParams &p, int v, bool interleaved, bool backward, cudaStream_t s) {
    const int lanes = lanes_of(p.dim, v);
    if (v == 4)
        return lanes == 8    ? launch_rope<kBf16, 4, 8, false>(rt, p, backward, s)
               : lanes == 16 ? launch_rope<kBf16, 4, 16, false>(rt, p, backward, s)
                             : launch_rope<kBf16, 4, 32, false>(rt, p, backward, s);
    if (interleaved)
        return lanes == 4   ? launch_rope<kBf16, 8, 4, true>(rt, p, backward, s)
               : lanes == 8 ? launch_rope<kBf16, 8, 8, true>(rt, p, backward, s)
                            : launch_rope<kBf16, 8, 16, true>(rt, p, backward, s);
    return lanes == 4   ? launch_rope<kBf16, 8, 4, false>(rt, p, backward, s)
           : lanes == 8 ? launch_rope<kBf16, 8, 8, false>(rt, p, backward, s)
                        : launch_rope<kBf16, 8, 16, false>(rt, p, backward, s);
}

cudaError_t launch_rope_dtype(const RuntimeInfo &rt, RopeParams &p, int64_t dtype, int v, bool interleaved, bool backward, cudaStream_t s) {
    return dtype == TGEMM_BF16 ? launch_rope_shape<true>(rt, p, v, interleaved, backward, s)
                               : launch_rope_shape<false>(rt, p, v, interleaved, backward, s);
}

constexpr int64_t kArrivals = 256;               // bytes
static_assert((kRopeFan + 1) * 4 <= kArrivals, "a counter for each group and one for all");
int64_t workspace_bytes(int64_t dim) { return kArrivals + static_cast<int64_t>(kRopeMaxBlocks + kRopeFan) * 2 * dim * 4; }

}  // namespace

#ifdef TGEMM_DEBUG
int rope_debug_last_check() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_debug_check, sizeof(v)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_debug_check, &zero, sizeof(zero)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return static_cast<int>(v);
}
#endif

}  // namespace tgemm

using namespace tgemm;

extern "C" tgemm_status tgemm_qk_norm_rope(const tgemm_qk_norm_rope_args *a, tgemm_stream_t stream) {
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    if (!a) return TGEMM_ERR_INVALID_ARG;
    int v = 8;
    bool interleaved = false;
    tgemm_status st = check_common(a, &p, &v, &interleaved);
    if (st != TGEMM_OK) return st;
    Rows in[2], out[2];
    const tgemm_rows *const from[2] = {&a->q, &a->k}, *const to[2] = {&a->q_out, &a->k_out};
    const int64_t heads[2] = {a->q_heads, a->k_heads};
    for (int i = 0; i < 2; ++i) {
        st = check_rows(*from[i], a->tokens, heads[i], a->dim, false, &in[i]);
        if (st == TGEMM_OK) st = check_rows(*to[i], a->tokens, heads[i], a->dim, true, &out[i]);
        if (st != TGEMM_OK) return st;
    }
    if (a->tokens == 0 || a->q_heads + a->k_heads == 0) return TGEMM_OK;
    Extent small[3];
    small_inputs(a, small);
    for (int i = 0; i < 2; ++i) {
        if (clash(out[i], in[i], true) || clash(out[i], in[1 - i], false)) return TGEMM_ERR_ALIAS;
        for (const Extent &e : small)
            if (overlaps({out[i].base, out[i].bytes}, e)) return TGEMM_ERR_ALIAS;
    }
    if (clash(out[0], out[1], false)) return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {in[0].bytes ? in[0].base : nullptr, in[1].bytes ? in[1].base : nullptr, out[0].bytes ? out[0].base : nullptr,
                                out[1].bytes ? out[1].base : nullptr, a->q_weight, a->k_weight, p.pairs > 0 ? a->positions : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        set_side(p.side[i], in[i], out[i], nullptr, i ? a->k_weight : a->q_weight);
        p.dbg_y[i] = out[i].bytes;
    }
    p.status = rt.status;
    return done(launch_rope_dtype(rt, p, a->dtype, v, interleaved, false, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" tgemm_status tgemm_qk_norm_rope_backward_workspace(int64_t dim, int64_t *bytes) {
    if (!bytes || dim < 8 || dim > 2 * kRopePairs || dim % 8 != 0) return TGEMM_ERR_INVALID_ARG;
    *bytes = workspace_bytes(dim);
    return TGEMM_OK;
}

extern "C" tgemm_status tgemm_qk_norm_rope_backward(const tgemm_qk_norm_rope_backward_args *b, tgemm_stream_t stream) {
    RopeParams p;
    std::memset(&p, 0, sizeof(p));
    if (!b) return TGEMM_ERR_INVALID_ARG;
    const tgemm_qk_norm_rope_args *const a = &b->forward;
    int v = 8;
    bool interleaved = false;
    tgemm_status st = check_common(a, &p, &v, &interleaved);
    if (st != TGEMM_OK) return st;
    const bool weights = b->q_weight_grad || b->k_weight_grad;
    if (weights && (!a->norm || !b->workspace || b->workspace_bytes < workspace_bytes(a->dim))) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(b->q_weight_grad) || !aligned4(b->k_weight_grad) || (weights && !aligned16(b->workspace))) return TGEMM_ERR_ALIGNMENT;
    Rows in[2], out[2], grad[2];
    const tgemm_rows *const from[2] = {&a->q, &a->k}, *const to[2] = {&a->q_out, &a->k_out}, *const by[2] = {&b->q_grad, &b->k_grad};
    const int64_t heads[2] = {a->q_heads, a->k_heads};
    for (int i = 0; i < 2; ++i) {
        if (a->norm) st = check_rows(*from[i], a->tokens, heads[i], a->dim, false, &in[i]);     // a rotation alone does not need them
        else in[i].heads = heads[i];
        if (st == TGEMM_OK) st = check_rows(*to[i], a->tokens, heads[i], a->dim, true, &out[i]);
        if (st == TGEMM_OK) st = check_rows(*by[i], a->tokens, heads[i], a->dim, false, &grad[i]);
        if (st != TGEMM_OK) return st;
    }
    if ((a->tokens == 0 || a->q_heads + a->k_heads == 0) && !weights) return TGEMM_OK;
    Extent small[6];
    small_inputs(a, small);
    small[3] = {b->q_weight_grad, b->q_weight_grad ? a->dim * 4 : 0};
    small[4] = {b->k_weight_grad, b->k_weight_grad ? a->dim * 4 : 0};
    small[5] = {b->workspace, weights ? workspace_bytes(a->dim) : 0};
    for (int i = 0; i < 2; ++i) {
        if (clash(out[i], in[i], true) || clash(out[i], grad[i], true) || clash(out[i], in[1 - i], false) || clash(out[i], grad[1 - i], false))
            return TGEMM_ERR_ALIAS;
        for (const Extent &e : small)
            if (overlaps({out[i].base, out[i].bytes}, e)) return TGEMM_ERR_ALIAS;
    }
    if (clash(out[0], out[1], false)) return TGEMM_ERR_ALIAS;
    for (int i = 3; i < 6; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(small[i], small[j])) return TGEMM_ERR_ALIAS;
        for (int j = 0; j < 2; ++j)
            if (overlaps(small[i], {in[j].base, in[j].bytes}) || overlaps(small[i], {grad[j].base, grad[j].bytes})) return TGEMM_ERR_ALIAS;
    }
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    for (int i = 0; i < 2; ++i)
        if (!all_device(rt.device, {in[i].bytes ? in[i].base : nullptr, out[i].bytes ? out[i].base : nullptr,
                                    grad[i].bytes ? grad[i].base : nullptr}))
            return TGEMM_ERR_INVALID_ARG;
    if (!all_device(rt.device, {a->q_weight, a->k_weight, p.pairs > 0 ? a->positions : nullptr, b->q_weight_grad, b->k_weight_grad,
                                weights ? b->workspace : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        set_side(p.side[i], in[i], out[i], &grad[i], i ? a->k_weight : a->q_weight);
        p.dbg_y[i] = out[i].bytes;
    }
    p.side[0].dw = b->q_weight_grad;
    p.side[1].dw = b->k_weight_grad;
    if (weights) {
        p.arrivals = static_cast<unsigned *>(b->workspace);
        p.partials = reinterpret_cast<float *>(static_cast<unsigned char *>(b->workspace) + kArrivals);
    }
    p.status = rt.status;
    return done(launch_rope_dtype(rt, p, a->dtype, v, interleaved, true, reinterpret_cast<cudaStream_t>(stream)));
}
