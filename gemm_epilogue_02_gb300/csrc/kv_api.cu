// C-ABI of the paged key-value cache (declarations and contract in
// include/tgemm.h): argument validation and the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
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
    view->dbg_bytes = bytes;
    *k = {c->k, bytes};
    *v = {c->v, bytes};
    return TGEMM_OK;
}

// Checks the page lists and lengths of a batch.
tgemm_status check_sequences(const tgemm_kv_sequences &q, bool with_lengths, int page_size, KvTable *t) {
    if (q.batch < 0 || q.batch > 65535 || q.pages_width < 0 || q.pages_width > (1 << 30) / page_size ||
        q.pages_stride < 0 || (q.batch > 1 && q.pages_stride < q.pages_width) || q.pages_stride > (int64_t(1) << 40))
        return TGEMM_ERR_INVALID_ARG;
    if (q.batch > 0 && ((q.pages_width > 0 && !q.pages) || (with_lengths && !q.lengths))) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(q.pages) || !aligned4(q.lengths)) return TGEMM_ERR_ALIGNMENT;
    t->pages = q.pages;
    t->lengths = q.lengths;
    t->stride = q.pages_stride;
    t->width = static_cast<int>(q.pages_width);
    t->batch = static_cast<int>(q.batch);
    return TGEMM_OK;
}

tgemm_status check_weights(const tgemm_kv_weights &a, int64_t batch, int64_t heads, KvWeights *w, Extent *e) {
    std::memset(w, 0, sizeof(*w));
    *e = Extent();
    if (!a.data) return TGEMM_OK;
    const int64_t size[2] = {batch, heads}, stride[2] = {a.batch_stride, a.head_stride};
    int64_t bytes = 0;
    if (a.width < 0 || a.width > INT32_MAX || !extent(size, stride, 2, a.width, 4, true, &bytes))
        return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(a.data)) return TGEMM_ERR_ALIGNMENT;
    w->base = a.data;
    w->width = static_cast<int>(a.width);
    w->batch_stride = a.batch_stride;
    w->head_stride = a.head_stride;
    *e = {a.data, bytes};
    return TGEMM_OK;
}

bool valid_dtype(int64_t d) { return d == TGEMM_F16 || d == TGEMM_BF16; }

bool all_device(int device, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !runtime_is_device_memory(p, device)) return false;
    return true;
}

// A programmatic dependent of the stream's previous kernel: every kernel here
// waits for it (griddepcontrol.wait) before it touches global memory, also what
// an earlier kernel than the previous has written: only this wait makes earlier
// writes visible.  cluster: blocks along x that form a cluster (1: none).
template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P &p, int cluster = 1) {
    cudaLaunchConfig_t lc;
    std::memset(&lc, 0, sizeof(lc));
    cudaLaunchAttribute la[2];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
    lc.gridDim = grid;
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    lc.attrs = la;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&lc, kernel, p);
}

tgemm_status done(cudaError_t e) {
    if (e == cudaSuccess) return TGEMM_OK;
    cudaGetLastError();
    return TGEMM_ERR_CUDA;
}

// ---------------------------------------------------------------- rows
// Lanes that hold a row of `bytes` in 16-byte pieces: the power of two at or above, 8 to 32.
int row_lanes(int bytes) { return bytes <= 128 ? 8 : bytes <= 256 ? 16 : 32; }

// Few rows: one pass a block, so that they reach all SMs; from two blocks an SM
// on, chunks of 64 to 128 rows (256 tokens of 8 heads: one pass 4.6 us on the
// GPU; 52042 tokens to e4m3: one pass 80 us, chunks 59 us).
template <bool kBf16, bool kE4m3, int kLanes>
cudaError_t launch_append_lanes(const RuntimeInfo &rt, const AppendParams &p, cudaStream_t s) {
    constexpr int kPass = kRowThreads / kLanes, kPieces = kE4m3 ? 2 : 1, kUnroll = kE4m3 ? 2 : 4;
    const int64_t passes = (p.tokens * p.cache.heads + kPass - 1) / kPass;
    if (passes <= 2 * rt.num_sms)
        return launch(kv_append_kernel<kBf16, kE4m3, kLanes, kPieces, 1>, dim3(static_cast<unsigned>(passes)), kRowThreads, 0, s, p);
    const int64_t chunks = std::min<int64_t>((passes + kUnroll - 1) / kUnroll, static_cast<int64_t>(rt.num_sms) * kAppendCtas);
    return launch(kv_append_kernel<kBf16, kE4m3, kLanes, kPieces, kUnroll>, dim3(static_cast<unsigned>(chunks)), kRowThreads, 0, s, p);
}

template <bool kBf16, bool kE4m3>
cudaError_t launch_append(const RuntimeInfo &rt, const AppendParams &p, cudaStream_t s) {
    switch (row_lanes(p.cache.dim * 2)) {
        case 8: return launch_append_lanes<kBf16, kE4m3, kE4m3 ? 4 : 8>(rt, p, s);
        case 16: return launch_append_lanes<kBf16, kE4m3, kE4m3 ? 8 : 16>(rt, p, s);
        default: return launch_append_lanes<kBf16, kE4m3, kE4m3 ? 16 : 32>(rt, p, s);
    }
}

template <int kThreads>
cudaError_t launch_select_threads(const RuntimeInfo &rt, EvictParams &p, int64_t positions, int cluster, cudaStream_t s) {
    auto kernel = kv_select_kernel<kThreads>;
    const int64_t slice = (positions + cluster - 1) / cluster;
    p.cached = slice <= kSelectMaxCached ? static_cast<int>(slice) : 0;
    static std::atomic<uint64_t> ready{0};      // bit per device
    const uint64_t bit = uint64_t(1) << rt.device;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const RelaxedCapture relaxed;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectMaxCached * 4);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(cluster), static_cast<unsigned>(p.from.heads), static_cast<unsigned>(p.table.batch));
    return launch(kernel, grid, kThreads, static_cast<size_t>(p.cached) * 4, s, p, cluster);
}

// positions: what a sequence can have at most.  Up to 4096 one block of 256
// threads takes them; beyond, blocks of 1024 take 8192 each, up to eight blocks.
cudaError_t launch_select(const RuntimeInfo &rt, EvictParams &p, int64_t positions, cudaStream_t s) {
    if (positions <= 4096) return launch_select_threads<256>(rt, p, positions, 1, s);
    int cluster = 1;
    while (cluster < 8 && cluster * 8192 < positions) cluster *= 2;
    return launch_select_threads<1024>(rt, p, positions, cluster, s);
}

template <bool kE4m3, int kLanes>
cudaError_t launch_gather_lanes(const EvictParams &p, int64_t most, int heads, int batch, cudaStream_t s) {
    constexpr int kUnroll = 4, kRows = kGatherThreads / kLanes * kUnroll;
    const int64_t chunks = std::min<int64_t>(65535, std::max<int64_t>(1, (most + kRows - 1) / kRows));
    const dim3 grid(static_cast<unsigned>(heads * batch), static_cast<unsigned>(chunks));
    return launch(kv_gather_kernel<kE4m3, kLanes, kUnroll>, grid, kGatherThreads, 0, s, p);
}

template <bool kE4m3>
cudaError_t launch_gather(const EvictParams &p, int64_t most, int heads, int batch, cudaStream_t s) {
    switch (row_lanes(p.from.row_bytes)) {
        case 8: return launch_gather_lanes<kE4m3, 8>(p, most, heads, batch, s);
        case 16: return launch_gather_lanes<kE4m3, 16>(p, most, heads, batch, s);
        default:                                   // e4m3 rows have 256 bytes at most
            if constexpr (kE4m3) return cudaErrorInvalidValue;
            else return launch_gather_lanes<kE4m3, 32>(p, most, heads, batch, s);
    }
}

// ---------------------------------------------------------------- attention
int padded_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Eights of query heads that a block takes, by the tiles of 64 positions that
// there can be for each of two blocks an SM (the host knows what the page lists
// can hold, not the lengths: lists with much room to spare are taken for long
// contexts).  Every block copies the rows for itself, so where the copies bound
// it the fewest blocks are best: three eights at once from 16 tiles on (24 heads,
// 32 contexts of 9000, 8 key heads, 16 bits: 232 us, two and one 309, one at a
// time 339; 16 heads: two 182, one at a time 229; e4m3 16 heads: two 139, one
// 176).  But a block of one eight has more warps, shorter steps and less to join,
// and below 6 tiles that counts more (24 heads, 7 contexts of 8192, 96 wide: one
// 21.2 us, two 23.3, three 27.2; 16 heads, 16 contexts of 300 with 4 key heads:
// one 11.8, two 13.6; with 2 tiles, 16000 e4m3 positions alone, 17.1 and 21.9;
// with 7, 16 contexts of 2000, 8 key heads: 12 heads 38.3 and 32.8, 24 heads 50.2
// and 49.3, three 44.7).  256-wide rows leave registers for one eight, and
// widening e4m3 rows leaves no gain for three.
int head_tiles(int64_t group, int64_t dim, bool e4m3, int64_t batch, int64_t heads, int64_t positions, int num_sms) {
    const int64_t tiles = batch * heads * (positions / 64), places = 2 * num_sms;
    if (group <= 8 || dim > 128 || tiles < 6 * places) return 1;
    if (e4m3 || group <= 16 || tiles < 16 * places) return 2;
    const int64_t eights = (group + 7) / 8;
    return (eights + 2) / 3 < (eights + 1) / 2 ? 3 : 2;
}

int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// The workspace's parts; returns its bytes (-1: too many).
int64_t attend_layout(int64_t batch, int64_t q_heads, int64_t group, int64_t dim, int64_t positions, bool weights,
                      unsigned char *base, AttendSpace *out) {
    const int64_t slots = 2 * kAttendMaxCtas, heads = group <= 8 || dim > 128 ? 8 : group <= 16 ? 16 : 24;   // of a block, at most
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
        const int64_t scored = batch * (q_heads / group) * ((group + 1) / 2 * 2);
        if (__builtin_mul_overflow(scored * 4, positions, &scores) || scores > kMost) return -1;
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
        const RelaxedCapture relaxed;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    // One CTA per place on the GPU, fewer when there cannot be as many tiles.  A run is shared by the heads where
    // that leaves at most a ninth of the places empty.
    const int64_t heads = static_cast<int64_t>(p.cache.heads) * p.blocks;
    const int64_t places = std::min<int64_t>(kAttendMaxCtas, static_cast<int64_t>(rt.num_sms) * Shape::kCtas);
    AttendParams q = p;
    q.lanes = places >= 8 * heads ? static_cast<int>(heads) : 1;
    const int64_t tiles = std::max<int64_t>(1, (p.positions + Shape::kTile - 1) / Shape::kTile);
    const int64_t most = p.table.batch * (q.lanes > 1 ? 1 : heads) * tiles;
    const int64_t grid = std::min(most, places / q.lanes) * q.lanes;
    return launch(kernel, dim3(static_cast<unsigned>(grid)), Shape::kThreads, Shape::kBytes, s, q);
}

template <bool kBf16, bool kE4m3>
cudaError_t launch_attend_dim(const RuntimeInfo &rt, const AttendParams &p, int tiles, cudaStream_t s) {
    switch (padded_dim(p.cache.dim)) {
        case 64:
            if constexpr (!kE4m3)
                if (tiles == 3) return launch_attend<kBf16, kE4m3, 64, 3>(rt, p, s);
            return tiles == 2 ? launch_attend<kBf16, kE4m3, 64, 2>(rt, p, s)
                                : launch_attend<kBf16, kE4m3, 64, 1>(rt, p, s);
        case 128:
            if constexpr (!kE4m3)
                if (tiles == 3) return launch_attend<kBf16, kE4m3, 128, 3>(rt, p, s);
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

extern "C" tgemm_status tgemm_kv_append(const tgemm_kv_append_args *a, tgemm_stream_t stream) {
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv, ew;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    const tgemm_kv_cache *cache = a->cache;
    tgemm_status st = check_cache(cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    const int64_t tokens = a->tokens, batch = a->seq.batch;
    if (!valid_dtype(a->dtype) || tokens < 0 || tokens > INT32_MAX || (!a->starts && tokens != batch))
        return TGEMM_ERR_INVALID_ARG;
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_weights(a->weights, batch, cache->heads, &p.weights, &ew);
    if (st != TGEMM_OK) return st;
    const int64_t size[2] = {tokens, cache->heads}, stride[2] = {a->token_stride, a->head_stride};
    int64_t bytes = 0;
    if (!extent(size, stride, 2, cache->dim, 2, false, &bytes)) return TGEMM_ERR_INVALID_ARG;
    if (tokens == 0 || batch == 0) return TGEMM_OK;
    if (!a->K || !a->V) return TGEMM_ERR_INVALID_ARG;
    if (!aligned16(a->K) || !aligned16(a->V) || !aligned4(a->starts) || (tokens > 1 && a->token_stride % 8 != 0) ||
        (cache->heads > 1 && a->head_stride % 8 != 0))
        return TGEMM_ERR_ALIGNMENT;
    const Extent nk = {a->K, bytes}, nv = {a->V, bytes};
    if (overlaps(nk, ck) || overlaps(nk, cv) || overlaps(nv, ck) || overlaps(nv, cv) ||
        (cache->pages > 0 && cache->k == cache->v))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->K, a->V, a->starts, a->seq.pages, a->seq.lengths, a->weights.data, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.k = static_cast<const unsigned char *>(a->K);
    p.v = static_cast<const unsigned char *>(a->V);
    p.token_stride = a->token_stride * 2;
    p.head_stride = a->head_stride * 2;
    p.starts = a->starts;
    p.tokens = tokens;
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!cache->e4m3) return done(launch_append<false, false>(rt, p, s));
    return done(a->dtype == TGEMM_BF16 ? launch_append<true, true>(rt, p, s) : launch_append<false, true>(rt, p, s));
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

extern "C" tgemm_status tgemm_attention_decode(const tgemm_attention_decode_args *a, tgemm_stream_t stream) {
    AttendParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv, ex;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    const tgemm_kv_cache *cache = a->cache;
    tgemm_status st = check_cache(cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    const int64_t batch = a->seq.batch, q_heads = a->q_heads;
    if (!valid_dtype(a->dtype) || q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 ||
        !std::isfinite(a->scale) || !std::isfinite(a->cap) || a->cap < 0.0 || a->window < 0)
        return TGEMM_ERR_INVALID_ARG;
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_weights(a->weights, batch, cache->heads, &p.weights, &ex);
    if (st != TGEMM_OK) return st;
    const int64_t size[2] = {batch, q_heads};
    const int64_t qs[2] = {a->q_batch_stride, a->q_head_stride}, os[2] = {a->o_batch_stride, a->o_head_stride};
    int64_t qbytes = 0, obytes = 0;
    if (!extent(size, qs, 2, cache->dim, 2, false, &qbytes) || !extent(size, os, 2, cache->dim, 2, true, &obytes))
        return TGEMM_ERR_INVALID_ARG;
    p.group = static_cast<int>(q_heads / cache->heads);
    p.scored = (p.group + 1) / 2 * 2;
    p.positions = a->seq.pages_width * cache->page_size;
    const int64_t need = attend_layout(batch, q_heads, p.group, cache->dim, p.positions, a->weights.data != nullptr,
                                       static_cast<unsigned char *>(a->workspace), &p.space);
    if (need < 0 || batch * q_heads > (int64_t(1) << 42) / std::max<int64_t>(1, p.positions)) return TGEMM_ERR_INVALID_ARG;
    if (batch == 0) return TGEMM_OK;
    if (!a->Q || !a->O || !a->workspace || a->workspace_bytes < need) return TGEMM_ERR_INVALID_ARG;
    if (!aligned16(a->Q) || !aligned16(a->O) || !aligned16(a->workspace) ||
        (batch > 1 && (a->q_batch_stride | a->o_batch_stride) % 8) ||
        (q_heads > 1 && (a->q_head_stride | a->o_head_stride) % 8))
        return TGEMM_ERR_ALIGNMENT;
    const Extent eo = {a->O, obytes}, eq = {a->Q, qbytes}, ew = {a->workspace, need};
    if (overlaps(eo, eq) || overlaps(eo, ck) || overlaps(eo, cv) || overlaps(eo, ex) || overlaps(ew, eo) ||
        overlaps(ew, eq) || overlaps(ew, ck) || overlaps(ew, cv) || overlaps(ew, ex))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->Q, a->O, a->seq.pages, a->seq.lengths, a->weights.data, a->workspace, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    if (cache->pages == 0) {      // the copies of nothing (rows left out) still name an address
        p.cache.k = p.cache.v = static_cast<unsigned char *>(a->workspace);
        p.cache.k_scale = p.cache.v_scale = static_cast<float *>(a->workspace);
    }
    p.q = static_cast<const unsigned char *>(a->Q);
    p.o = static_cast<unsigned char *>(a->O);
    p.q_batch_stride = a->q_batch_stride * 2;
    p.q_head_stride = a->q_head_stride * 2;
    p.o_batch_stride = a->o_batch_stride * 2;
    p.o_head_stride = a->o_head_stride * 2;
    p.window = static_cast<int>(std::min<int64_t>(a->window, INT32_MAX));
    constexpr double kLog2e = 1.4426950408889634;
    // A cap above 2^64 changes no score below 2^52 by fp32's half step.  A product of 0 has to keep a score of 0, so
    // the factor is cut to fp32's range, and before a tanh to 2^60, which leaves e4m3's scales room: what that changes
    // is a score below a cap that is no more than 2^-60 of the scale.
    p.capped = a->cap > 0.0 && a->cap <= 0x1p64;
    const double first = p.capped ? a->scale / a->cap : a->scale * kLog2e;
    const double most_first = p.capped ? 0x1p60 : FLT_MAX;
    p.first = static_cast<float>(std::clamp<double>(first, -most_first, most_first));
    p.last = p.capped ? static_cast<float>(a->cap * kLog2e) : 0.0f;
    p.page_shift = -1;
    for (int i = 0; i <= 20; ++i)
        if (cache->page_size == 1 << i) p.page_shift = i;
    p.dbg_o_bytes = obytes;
    p.dbg_scores = batch * cache->heads * p.positions * p.scored;
    const int64_t most = a->window > 0 ? std::min<int64_t>(p.positions, a->window) : p.positions;
    const int tiles = head_tiles(p.group, cache->dim, cache->e4m3 != 0, batch, cache->heads, most, rt.num_sms);
    p.blocks = (p.group + 8 * tiles - 1) / (8 * tiles);
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (a->dtype == TGEMM_BF16)
        e = cache->e4m3 ? launch_attend_dim<true, true>(rt, p, tiles, s) : launch_attend_dim<true, false>(rt, p, tiles, s);
    else
        e = cache->e4m3 ? launch_attend_dim<false, true>(rt, p, tiles, s) : launch_attend_dim<false, false>(rt, p, tiles, s);
    if (e == cudaSuccess && p.weights.base) {
        constexpr int64_t kPer = kSpreadThreads * kSpreadEach;
        const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((p.positions + kPer - 1) / kPer, 1024));
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(cache->heads), static_cast<unsigned>(batch));
        e = launch(kv_spread_kernel, grid, kSpreadThreads, 0, s, p);
    }
    return done(e);
}

extern "C" tgemm_status tgemm_kv_evict(const tgemm_kv_evict_args *a, tgemm_stream_t stream) {
    EvictParams p;
    std::memset(&p, 0, sizeof(p));
    Extent fk, fv, tk, tv, ew, et;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    const tgemm_kv_cache *from = a->from, *to = a->to;
    tgemm_status st = check_cache(from, &p.from, &fk, &fv);
    if (st != TGEMM_OK) return st;
    st = check_cache(to, &p.to, &tk, &tv);
    if (st != TGEMM_OK) return st;
    const int64_t batch = a->seq.batch, heads = from->heads, keep = a->keep;
    if (to->heads != heads || from->dim != to->dim || from->e4m3 != to->e4m3 || a->to_seq.batch != batch || keep < 1 ||
        keep > (1 << 30) || a->recent < 0 || batch > 65535 || heads * batch > INT32_MAX)
        return TGEMM_ERR_INVALID_ARG;
    st = check_sequences(a->seq, true, from->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    st = check_sequences(a->to_seq, false, to->page_size, &p.to_table);
    if (st != TGEMM_OK) return st;
    st = check_weights(a->weights, batch, heads, &p.weights, &ew);
    if (st != TGEMM_OK) return st;
    st = check_weights(a->to_weights, batch, heads, &p.to_weights, &et);
    if (st != TGEMM_OK) return st;
    if (batch == 0) return TGEMM_OK;
    if (!a->weights.data || !a->kept || !a->to_lengths || !a->to_weights.data || a->to_weights.width < keep)
        return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(a->kept) || !aligned4(a->to_lengths)) return TGEMM_ERR_ALIGNMENT;
    const Extent ek = {a->kept, batch * heads * keep * 4}, el = {a->seq.lengths, batch * 4}, en = {a->to_lengths, batch * 4};
    if (overlaps(et, ew) || overlaps(ek, ew) || overlaps(ek, et) || overlaps(en, el) || overlaps(ek, el) ||
        overlaps(et, el) || overlaps(en, ek) || overlaps(en, et) || overlaps(en, ew))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device,
                    {a->seq.pages, a->seq.lengths, a->weights.data, a->to_seq.pages, a->kept, a->to_lengths,
                     a->to_weights.data, from->k, from->v, to->k, to->v, from->e4m3 ? from->k_scale : nullptr,
                     from->e4m3 ? from->v_scale : nullptr, to->e4m3 ? to->k_scale : nullptr,
                     to->e4m3 ? to->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.kept = a->kept;
    p.to_lengths = a->to_lengths;
    p.keep = static_cast<int>(keep);
    p.recent = static_cast<int>(std::min<int64_t>(a->recent, INT32_MAX));
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t positions = std::min<int64_t>(a->seq.pages_width * from->page_size, a->weights.width);
    st = done(launch_select(rt, p, positions, s));
    if (st != TGEMM_OK) return st;
    const int64_t most = std::min<int64_t>(keep, positions);
    return done(from->e4m3 ? launch_gather<true>(p, most, from->heads, static_cast<int>(batch), s)
                           : launch_gather<false>(p, most, from->heads, static_cast<int>(batch), s));
}
