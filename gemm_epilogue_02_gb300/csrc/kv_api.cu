// C-ABI of the paged key-value cache (declarations and contract in
// include/tgemm.h): argument validation and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/tgemm.h"
#include "kv_append.cuh"
#include "kv_attend.cuh"
#include "kv_evict.cuh"
#include "runtime.h"

namespace tgemm {
namespace {

constexpr int64_t kMost = int64_t(1) << 61;       // bytes: no valid allocation is that large

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Extent {
    const void *base = nullptr;
    int64_t bytes = 0;
};

bool overlaps(const Extent &a, const Extent &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    return a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
           y < x + static_cast<uintptr_t>(a.bytes);
}

// Bytes from the first element to the end of the last of a strided array: sum
// of (size - 1) * stride, plus a run of `width`, in elements of `esize` bytes.
// False for a negative size or stride, one too large, or, with `apart`, a
// stride below `width` (elements of different rows would share memory).
bool extent(const int64_t *size, const int64_t *stride, int dims, int64_t width, int64_t esize, bool apart,
            int64_t *bytes) {
    int64_t sum = width;
    for (int i = 0; i < dims; ++i) {
        int64_t part = 0;
        if (size[i] < 0 || stride[i] < 0 || (apart && size[i] > 1 && stride[i] < width)) return false;
        if (size[i] == 0) {
            *bytes = 0;
            return true;
        }
        if (__builtin_mul_overflow(size[i] - 1, stride[i], &part) || __builtin_add_overflow(sum, part, &sum) ||
            sum > kMost)
            return false;
    }
    *bytes = sum * esize;
    return true;
}

// Checks a cache's description and fills the kernels' view of it.
tgemm_status check_cache(const tgemm_kv_cache *c, KvView *view, Extent *k, Extent *v) {
    if (!c) return TGEMM_ERR_INVALID_ARG;
    const int esize = c->e4m3 ? 1 : 2, chunk = 16 / esize;
    if ((c->e4m3 != 0 && c->e4m3 != 1) || c->pages < 0 || c->pages > INT32_MAX || c->page_size < 1 ||
        c->page_size > (1 << 20) || c->heads < 1 || c->heads > 65535 || c->dim < chunk || c->dim > 256 ||
        c->dim % chunk != 0)
        return TGEMM_ERR_INVALID_ARG;
    const int64_t size[3] = {c->pages, c->page_size, c->heads};
    const int64_t stride[3] = {c->page_stride, c->slot_stride, c->head_stride};
    const int64_t sstride[3] = {c->scale_page_stride, c->scale_slot_stride, c->scale_head_stride};
    int64_t bytes = 0, sbytes = 0;
    if (!extent(size, stride, 3, c->dim, esize, true, &bytes)) return TGEMM_ERR_INVALID_ARG;
    if (c->e4m3 && !extent(size, sstride, 3, 1, 4, true, &sbytes)) return TGEMM_ERR_INVALID_ARG;
    if (c->pages > 0) {
        if (!c->k || !c->v || (c->e4m3 && (!c->k_scale || !c->v_scale))) return TGEMM_ERR_INVALID_ARG;
        if (!aligned16(c->k) || !aligned16(c->v)) return TGEMM_ERR_ALIGNMENT;
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1 && stride[i] % chunk != 0) return TGEMM_ERR_ALIGNMENT;
        if (c->e4m3 && (!aligned4(c->k_scale) || !aligned4(c->v_scale))) return TGEMM_ERR_ALIGNMENT;
    }
    view->k = static_cast<unsigned char *>(c->k);
    view->v = static_cast<unsigned char *>(c->v);
    view->k_scale = c->k_scale;
    view->v_scale = c->v_scale;
    view->pages = c->pages;
    view->page_stride = c->page_stride * esize;
    view->slot_stride = c->slot_stride * esize;
    view->head_stride = c->head_stride * esize;
    view->scale_page_stride = c->scale_page_stride;
    view->scale_slot_stride = c->scale_slot_stride;
    view->scale_head_stride = c->scale_head_stride;
    view->page_size = c->page_size;
    view->heads = c->heads;
    view->dim = c->dim;
    view->row_bytes = c->dim * esize;
    *k = {c->k, bytes};
    *v = {c->v, bytes};
    return TGEMM_OK;
}

// Checks the page lists and lengths of `batch` sequences.
tgemm_status check_table(const int32_t *pages, int64_t width, int64_t stride, const int32_t *lengths, bool with_lengths,
                         int64_t batch, int page_size, KvTable *t) {
    if (batch < 0 || batch > 65535 || width < 0 || width > (1 << 30) / page_size || stride < 0 ||
        (batch > 1 && stride < width) || stride > (int64_t(1) << 40))
        return TGEMM_ERR_INVALID_ARG;
    if (batch > 0 && ((width > 0 && !pages) || (with_lengths && !lengths))) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(pages) || !aligned4(lengths)) return TGEMM_ERR_ALIGNMENT;
    t->pages = pages;
    t->lengths = lengths;
    t->stride = stride;
    t->width = static_cast<int>(width);
    t->batch = static_cast<int>(batch);
    return TGEMM_OK;
}

tgemm_status check_weights(const float *base, int64_t width, int64_t batch_stride, int64_t head_stride, int64_t batch,
                           int64_t heads, KvWeights *w) {
    w->base = const_cast<float *>(base);
    w->width = 0;
    w->batch_stride = w->head_stride = 0;
    if (!base) return TGEMM_OK;
    const int64_t size[2] = {batch, heads}, stride[2] = {batch_stride, head_stride};
    int64_t bytes = 0;
    if (width < 0 || width > INT32_MAX || !extent(size, stride, 2, width, 4, true, &bytes))
        return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(base)) return TGEMM_ERR_ALIGNMENT;
    w->width = static_cast<int>(width);
    w->batch_stride = batch_stride;
    w->head_stride = head_stride;
    return TGEMM_OK;
}

bool all_device(int device, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !runtime_is_device_memory(p, device)) return false;
    return true;
}

// A programmatic dependent of the stream's previous kernel: every kernel here
// waits for it (griddepcontrol.wait) before it touches global memory.
template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P &p) {
    cudaLaunchConfig_t lc;
    std::memset(&lc, 0, sizeof(lc));
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    lc.attrs = la;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

tgemm_status done(cudaError_t e) {
    if (e == cudaSuccess) return TGEMM_OK;
    cudaGetLastError();
    return TGEMM_ERR_CUDA;
}

// ---------------------------------------------------------------- attention
int padded_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Blocks of 8 query heads up to 8 heads on a key head, of 16 above (one read of
// the keys instead of two); 256-wide rows leave registers for 8 only.
int head_tiles(int64_t group, int64_t dim) { return group > 8 && dim <= 128 ? 2 : 1; }

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// The workspace's parts; returns its bytes (-1: too many).
int64_t attend_layout(int64_t batch, int64_t q_heads, int64_t group, int64_t dim, int64_t positions, bool weights,
                      unsigned char *base, AttendSpace *out) {
    const int64_t slots = 2 * kAttendMaxCtas, heads = 8 * head_tiles(group, dim);
    int64_t at = 0, scores = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += align256(bytes);
        return here;
    };
    const int64_t parts = take(slots * 4), groups = take(slots * 4);
    const int64_t o = take(slots * heads * padded_dim(dim) * 4), ml = take(slots * heads * 8);
    int64_t stats = 0, s = 0;
    if (weights) {
        if (__builtin_mul_overflow(batch * q_heads * 4, positions, &scores) || scores > kMost) return -1;
        stats = take(batch * q_heads * 8);
        s = take(scores);
    }
    if (out) {
        out->parts = reinterpret_cast<unsigned *>(base + parts);
        out->groups = reinterpret_cast<unsigned *>(base + groups);
        out->out = reinterpret_cast<float *>(base + o);
        out->ml = reinterpret_cast<float2 *>(base + ml);
        out->stats = weights ? reinterpret_cast<float2 *>(base + stats) : nullptr;
        out->scores = weights ? reinterpret_cast<float *>(base + s) : nullptr;
    }
    return at;
}

template <bool kBf16, bool kE4m3, int DP, int NT>
cudaError_t launch_attend(const RuntimeInfo &rt, const AttendParams &p, cudaStream_t s) {
    using Shape = AttendShape<kE4m3, DP, NT>;
    auto kernel = kv_attend_kernel<kBf16, kE4m3, DP, NT>;
    static std::atomic<uint64_t> ready{0};      // bit per device
    const uint64_t bit = uint64_t(1) << rt.device;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    // One CTA per place on the GPU, fewer when there cannot be as many tiles.
    const int64_t tiles = (p.positions + Shape::kTile - 1) / Shape::kTile;
    const int64_t most = static_cast<int64_t>(p.table.batch) * p.cache.heads * p.blocks * std::max<int64_t>(1, tiles);
    const int64_t places = std::min<int64_t>(kAttendMaxCtas, static_cast<int64_t>(rt.num_sms) * Shape::kCtas);
    return launch(kernel, dim3(static_cast<unsigned>(std::min(most, places))), kAttendThreads, Shape::kBytes, s, p);
}

template <bool kBf16, bool kE4m3>
cudaError_t launch_attend_dim(const RuntimeInfo &rt, const AttendParams &p, int tiles, cudaStream_t s) {
    switch (padded_dim(p.cache.dim)) {
        case 64:
            return tiles == 2 ? launch_attend<kBf16, kE4m3, 64, 2>(rt, p, s) : launch_attend<kBf16, kE4m3, 64, 1>(rt, p, s);
        case 128:
            return tiles == 2 ? launch_attend<kBf16, kE4m3, 128, 2>(rt, p, s)
                              : launch_attend<kBf16, kE4m3, 128, 1>(rt, p, s);
        default:
            return launch_attend<kBf16, kE4m3, 256, 1>(rt, p, s);
    }
}

}  // namespace

#ifdef TGEMM_DEBUG
int kv_debug_last_check() {
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

extern "C" tgemm_status tgemm_kv_append(const tgemm_kv_cache *cache, const void *K, const void *V, int64_t tokens,
                                        int64_t token_stride, int64_t head_stride, const int32_t *starts,
                                        const int32_t *pages, int64_t pages_width, int64_t pages_stride,
                                        const int32_t *lengths, int64_t batch, float *weights, int64_t weights_width,
                                        int64_t weights_batch_stride, int64_t weights_head_stride, tgemm_dtype dtype,
                                        tgemm_stream_t stream) {
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv;
    tgemm_status st = check_cache(cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    if ((dtype != TGEMM_F16 && dtype != TGEMM_BF16) || tokens < 0 || tokens > INT32_MAX || (!starts && tokens != batch))
        return TGEMM_ERR_INVALID_ARG;
    st = check_table(pages, pages_width, pages_stride, lengths, true, batch, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_weights(weights, weights_width, weights_batch_stride, weights_head_stride, batch, cache->heads,
                       &p.weights);
    if (st != TGEMM_OK) return st;
    const int64_t size[2] = {tokens, cache->heads}, stride[2] = {token_stride, head_stride};
    int64_t bytes = 0;
    if (!extent(size, stride, 2, cache->dim, 2, false, &bytes)) return TGEMM_ERR_INVALID_ARG;
    if (tokens == 0 || batch == 0) return TGEMM_OK;
    if (!K || !V) return TGEMM_ERR_INVALID_ARG;
    if (!aligned16(K) || !aligned16(V) || !aligned4(starts) || (tokens > 1 && token_stride % 8 != 0) ||
        (cache->heads > 1 && head_stride % 8 != 0))
        return TGEMM_ERR_ALIGNMENT;
    const Extent nk = {K, bytes}, nv = {V, bytes};
    if (overlaps(nk, ck) || overlaps(nk, cv) || overlaps(nv, ck) || overlaps(nv, cv) || cache->k == cache->v)
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {K, V, starts, pages, lengths, weights, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.k = static_cast<const unsigned char *>(K);
    p.v = static_cast<const unsigned char *>(V);
    p.token_stride = token_stride * 2;
    p.head_stride = head_stride * 2;
    p.starts = starts;
    p.tokens = tokens;
    p.status = rt.status;
    const int64_t rows = tokens * cache->heads, per = kAppendThreads / 32;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, rt.num_sms * 8)));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!cache->e4m3) return done(launch(kv_append_kernel<false, false>, grid, kAppendThreads, 0, s, p));
    if (dtype == TGEMM_BF16) return done(launch(kv_append_kernel<true, true>, grid, kAppendThreads, 0, s, p));
    return done(launch(kv_append_kernel<false, true>, grid, kAppendThreads, 0, s, p));
}

extern "C" tgemm_status tgemm_attention_decode_workspace(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t dim,
                                                         int64_t positions, int with_weights, int64_t *bytes) {
    if (!bytes || batch < 0 || batch > 65535 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || dim < 8 ||
        dim > 256 || q_heads > 65535 || positions < 0 || (with_weights != 0 && with_weights != 1))
        return TGEMM_ERR_INVALID_ARG;
    const int64_t need = attend_layout(batch, q_heads, q_heads / kv_heads, dim, positions, with_weights != 0, nullptr, nullptr);
    if (need < 0) return TGEMM_ERR_INVALID_ARG;
    *bytes = need;
    return TGEMM_OK;
}

extern "C" tgemm_status tgemm_attention_decode(const tgemm_kv_cache *cache, const void *Q, void *O, int64_t batch,
                                               int64_t q_heads, int64_t q_batch_stride, int64_t q_head_stride,
                                               int64_t o_batch_stride, int64_t o_head_stride, const int32_t *pages,
                                               int64_t pages_width, int64_t pages_stride, const int32_t *lengths,
                                               float scale, float cap, int64_t window, float *weights,
                                               int64_t weights_width, int64_t weights_batch_stride,
                                               int64_t weights_head_stride, void *workspace, int64_t workspace_bytes,
                                               tgemm_dtype dtype, tgemm_stream_t stream) {
    AttendParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv;
    tgemm_status st = check_cache(cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    if ((dtype != TGEMM_F16 && dtype != TGEMM_BF16) || q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 ||
        !std::isfinite(scale) || !std::isfinite(cap) || cap < 0.0f || window < 0)
        return TGEMM_ERR_INVALID_ARG;
    st = check_table(pages, pages_width, pages_stride, lengths, true, batch, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_weights(weights, weights_width, weights_batch_stride, weights_head_stride, batch, cache->heads,
                       &p.weights);
    if (st != TGEMM_OK) return st;
    const int64_t size[2] = {batch, q_heads};
    const int64_t qs[2] = {q_batch_stride, q_head_stride}, os[2] = {o_batch_stride, o_head_stride};
    int64_t qbytes = 0, obytes = 0;
    if (!extent(size, qs, 2, cache->dim, 2, false, &qbytes) || !extent(size, os, 2, cache->dim, 2, true, &obytes))
        return TGEMM_ERR_INVALID_ARG;
    int64_t need = 0;
    st = tgemm_attention_decode_workspace(batch, q_heads, cache->heads, cache->dim, pages_width * cache->page_size,
                                          weights ? 1 : 0, &need);
    if (st != TGEMM_OK) return st;
    if (batch == 0) return TGEMM_OK;
    if (!Q || !O || !workspace || workspace_bytes < need) return TGEMM_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(O) || !aligned16(workspace) || (batch > 1 && (q_batch_stride | o_batch_stride) % 8) ||
        (q_heads > 1 && (q_head_stride | o_head_stride) % 8))
        return TGEMM_ERR_ALIGNMENT;
    const Extent eo = {O, obytes}, ew = {workspace, need};
    if (overlaps(eo, {Q, qbytes}) || overlaps(eo, ck) || overlaps(eo, cv) || overlaps(ew, eo) ||
        overlaps(ew, {Q, qbytes}) || overlaps(ew, ck) || overlaps(ew, cv))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {Q, O, pages, lengths, weights, workspace, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.q = static_cast<const unsigned char *>(Q);
    p.o = static_cast<unsigned char *>(O);
    p.q_batch_stride = q_batch_stride * 2;
    p.q_head_stride = q_head_stride * 2;
    p.o_batch_stride = o_batch_stride * 2;
    p.o_head_stride = o_head_stride * 2;
    p.group = static_cast<int>(q_heads / cache->heads);
    p.window = static_cast<int>(std::min<int64_t>(window, INT32_MAX));
    constexpr double kLog2e = 1.4426950408889634;
    p.capped = cap > 0.0f;
    p.first = static_cast<float>(p.capped ? scale * 2.0 * kLog2e / cap : scale * kLog2e);
    p.last = static_cast<float>(cap * kLog2e);
    p.positions = pages_width * cache->page_size;
    const int tiles = head_tiles(p.group, cache->dim);
    p.blocks = (p.group + 8 * tiles - 1) / (8 * tiles);
    attend_layout(batch, q_heads, p.group, cache->dim, p.positions, weights != nullptr,
                  static_cast<unsigned char *>(workspace), &p.space);
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == TGEMM_BF16)
        e = cache->e4m3 ? launch_attend_dim<true, true>(rt, p, tiles, s) : launch_attend_dim<true, false>(rt, p, tiles, s);
    else
        e = cache->e4m3 ? launch_attend_dim<false, true>(rt, p, tiles, s) : launch_attend_dim<false, false>(rt, p, tiles, s);
    if (e == cudaSuccess && weights) {
        const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((p.positions + kSpreadThreads - 1) / kSpreadThreads, 64));
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(cache->heads), static_cast<unsigned>(batch));
        e = launch(kv_spread_kernel, grid, kSpreadThreads, 0, s, p);
    }
    return done(e);
}

extern "C" tgemm_status tgemm_kv_evict(const tgemm_kv_cache *from, const int32_t *pages, int64_t pages_width,
                                       int64_t pages_stride, const int32_t *lengths, int64_t batch,
                                       const float *weights, int64_t weights_width, int64_t weights_batch_stride,
                                       int64_t weights_head_stride, const tgemm_kv_cache *to, const int32_t *to_pages,
                                       int64_t to_pages_width, int64_t to_pages_stride, int64_t keep, int64_t recent,
                                       int32_t *kept, int32_t *to_lengths, float *to_weights, int64_t to_weights_width,
                                       int64_t to_weights_batch_stride, int64_t to_weights_head_stride,
                                       tgemm_stream_t stream) {
    EvictParams p;
    std::memset(&p, 0, sizeof(p));
    Extent fk, fv, tk, tv;
    tgemm_status st = check_cache(from, &p.from, &fk, &fv);
    if (st != TGEMM_OK) return st;
    st = check_cache(to, &p.to, &tk, &tv);
    if (st != TGEMM_OK) return st;
    if (from->heads != to->heads || from->dim != to->dim || from->e4m3 != to->e4m3 || keep < 1 || keep > INT32_MAX ||
        recent < 0)
        return TGEMM_ERR_INVALID_ARG;
    st = check_table(pages, pages_width, pages_stride, lengths, true, batch, from->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_table(to_pages, to_pages_width, to_pages_stride, nullptr, false, batch, to->page_size, &p.to_table);
    if (st != TGEMM_OK) return st;
    st = check_weights(weights, weights_width, weights_batch_stride, weights_head_stride, batch, from->heads,
                       &p.weights);
    if (st != TGEMM_OK) return st;
    st = check_weights(to_weights, to_weights_width, to_weights_batch_stride, to_weights_head_stride, batch,
                       from->heads, &p.to_weights);
    if (st != TGEMM_OK) return st;
    if (batch == 0) return TGEMM_OK;
    if (!weights || !kept || !to_lengths || !to_weights || to_weights_width < keep) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(kept) || !aligned4(to_lengths)) return TGEMM_ERR_ALIGNMENT;
    const int64_t heads = from->heads;
    int64_t wb = 0, twb = 0;
    const int64_t size[2] = {batch, heads};
    const int64_t ws[2] = {weights_batch_stride, weights_head_stride};
    const int64_t ts[2] = {to_weights_batch_stride, to_weights_head_stride};
    extent(size, ws, 2, weights_width, 4, true, &wb);
    extent(size, ts, 2, to_weights_width, 4, true, &twb);
    const Extent ew = {weights, wb}, et = {to_weights, twb}, ek = {kept, batch * heads * keep * 4},
                 el = {lengths, batch * 4}, en = {to_lengths, batch * 4};
    if (overlaps(et, ew) || overlaps(ek, ew) || overlaps(ek, et) || overlaps(en, el) || overlaps(en, ek) ||
        overlaps(en, et) || overlaps(en, ew))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device,
                    {pages, lengths, weights, to_pages, kept, to_lengths, to_weights, from->k, from->v, to->k, to->v,
                     from->e4m3 ? from->k_scale : nullptr, from->e4m3 ? from->v_scale : nullptr,
                     to->e4m3 ? to->k_scale : nullptr, to->e4m3 ? to->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.kept = kept;
    p.to_lengths = to_lengths;
    p.keep = static_cast<int>(keep);
    p.recent = static_cast<int>(std::min<int64_t>(recent, INT32_MAX));
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = done(launch(kv_select_kernel, dim3(static_cast<unsigned>(heads), static_cast<unsigned>(batch)),
                     kSelectThreads, 0, s, p));
    if (st != TGEMM_OK) return st;
    const int64_t items = heads * batch, most = std::min<int64_t>(keep, pages_width * from->page_size);
    const int64_t per = kGatherThreads / 32;
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((most + per - 1) / per, 16));
    if (items > 65535) return TGEMM_ERR_INVALID_ARG;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(items));
    return done(launch(from->e4m3 ? kv_gather_kernel<true> : kv_gather_kernel<false>, grid, kGatherThreads, 0, s, p));
}
