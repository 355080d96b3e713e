// C-ABI of the bounds of pages, the choice by them, and the pages as a resource
// (declarations and contract in include/tgemm.h): argument validation and the
// launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "../../include/tgemm.h"
#include "page_bounds.cuh"
#include "kv_host.h"
#include "page_pool.cuh"
#include "runtime.h"

namespace tgemm {
namespace {

constexpr int kChooseMaxPages = 1 << 17;      // of a page list: eight blocks' keys then fit their shared memory
constexpr int kChooseGather = 1 << 12;        // pages of a list whose keys a cluster's first block ranks alone (8193: 21.5 us so, 18 together)
constexpr int kChooseMaxBytes = 224 * 1024;   // of a block's dynamic shared memory

tgemm_status check_bounds(const tgemm_kv_page_bounds *b, const tgemm_kv_cache *c, KvBounds *view, Extent *e, Extent *es) {
    if (!b || c->dim % 16 != 0) return TGEMM_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(c->pages) * c->heads;
    if (rows > kMost / 1024) return TGEMM_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!b->bounds || !b->scale) return TGEMM_ERR_INVALID_ARG;
        if (!aligned16(b->bounds) || !aligned4(b->scale)) return TGEMM_ERR_ALIGNMENT;
    }
    view->base = b->bounds;
    view->scale = b->scale;
    view->dbg_rows = rows;
    *e = {b->bounds, rows * 2 * c->dim};
    *es = {b->scale, rows * 4};
    return TGEMM_OK;
}

// Rows of a page, and pages, that the kernels count in 32 bits with room to step past them.
bool countable_pool(const tgemm_kv_cache *c) {
    return c->pages <= (1 << 30) && static_cast<int64_t>(c->page_size) * c->heads <= (1 << 30);
}

// Page counts that the kernels add up in 32 bits stay there.
bool countable(int64_t batch, int64_t width) { return std::min<int64_t>(batch, 1024) * width <= INT32_MAX; }

// Lists that a call writes.
tgemm_status check_lists(int32_t *pages, int32_t *lengths, int64_t width, int64_t stride, int64_t batch, int page_size, KvLists *l,
                         Extent *e) {
    const tgemm_kv_sequences q = {pages, lengths, width, stride, batch};
    KvTable t;
    const tgemm_status st = check_sequences(q, true, page_size, &t);
    if (st != TGEMM_OK) return st;
    if (!countable(batch, width)) return TGEMM_ERR_INVALID_ARG;
    l->pages = pages;
    l->lengths = lengths;
    l->stride = stride;
    l->width = t.width;
    l->batch = t.batch;
    *e = {pages, batch > 0 ? ((batch - 1) * stride + width) * 4 : 0};
    return TGEMM_OK;
}

bool overlaps_any(const Extent &x, std::initializer_list<Extent> others) {
    for (const Extent &o : others)
        if (overlaps(x, o)) return true;
    return false;
}

bool cache_overlaps(const tgemm_kv_cache *c, const Extent &k, const Extent &v, const Extent &x) {
    if (overlaps(x, k) || overlaps(x, v)) return true;
    if (!c->e4m3 || c->pages == 0) return false;
    const int64_t size[3] = {c->pages, c->page_size, c->heads};
    const int64_t stride[3] = {c->scale_page_stride, c->scale_slot_stride, c->scale_head_stride};
    int64_t bytes = 0;
    if (!extent(size, stride, 3, 1, 4, true, &bytes)) return true;
    return overlaps(x, {c->k_scale, bytes}) || overlaps(x, {c->v_scale, bytes});
}

int row_lanes(int bytes) { return bytes <= 128 ? 8 : bytes <= 256 ? 16 : 32; }

// ---------------------------------------------------------------- bounds and choice
template <bool kBf16, bool kE4m3, int kLanes>
cudaError_t launch_bounds_lanes(const RuntimeInfo &rt, const BoundsParams &p, cudaStream_t s) {
    constexpr int kGroups = 32 / kLanes;
    const int64_t most = (p.starts ? static_cast<int64_t>(p.table.batch) * p.table.width : p.table.batch) * p.cache.heads;
    auto grid = [&](int items, int ctas) {       // for as many pages as there can be
        const int64_t units = (most + items - 1) / items, blocks = (units + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
        return dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(blocks, static_cast<int64_t>(rt.num_sms) * ctas))));
    };
    if (p.cache.page_size <= kBoundsAlone && kGroups > 1)
        return launch(page_bounds_kernel<kBf16, kE4m3, kLanes, 8, kGroups != 1>, grid(kGroups, kE4m3 ? 2 : 4), kBoundsThreads, 0, s, p);
    return launch(page_bounds_kernel<kBf16, kE4m3, kLanes, 8, false>, grid(1, kE4m3 ? 2 : 4), kBoundsThreads, 0, s, p);
}

template <bool kBf16, bool kE4m3>
cudaError_t launch_bounds(const RuntimeInfo &rt, const BoundsParams &p, cudaStream_t s) {
    switch (row_lanes(p.cache.row_bytes)) {
        case 8: return launch_bounds_lanes<kBf16, kE4m3, 8>(rt, p, s);
        case 16: return launch_bounds_lanes<kBf16, kE4m3, 16>(rt, p, s);
        default:                                   // e4m3 rows have 256 bytes at most
            if constexpr (kE4m3) return cudaErrorInvalidValue;
            else return launch_bounds_lanes<kBf16, kE4m3, 32>(rt, p, s);
    }
}

template <int kThreads, bool kBf16, int kChunks, int kStages, bool kFew>
cudaError_t launch_choose_stages(const RuntimeInfo &rt, ChooseParams &p, int cluster, cudaStream_t s) {
    using Shape = ChooseShape<kThreads, kChunks, kStages>;
    auto kernel = page_choose_kernel<kThreads, kBf16, kChunks, kStages, kFew>;
    static std::atomic<uint64_t> ready{0};      // bit per device
    const uint64_t bit = uint64_t(1) << rt.device;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const RelaxedCapture relaxed;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChooseMaxBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(cluster), static_cast<unsigned>(p.cache.heads), static_cast<unsigned>(p.table.batch));
    return launch(kernel, grid, kThreads, static_cast<size_t>(Shape::bytes(p.cached, p.group, p.cache.dim)), s, p, cluster);
}

template <int kThreads, bool kBf16, int kChunks>
cudaError_t launch_choose_shape(const RuntimeInfo &rt, ChooseParams &p, cudaStream_t s) {
    // A cluster's barriers cost about 3 us, and a block of 16 warps scores about 250 pages a microsecond where few run: with lists
    // of up to 512 pages a block alone is best, beyond them as many of a cluster as leave each an SM (1251 pages, 8 heads: one
    // 16.1 us, two 14.1, four 11.6, eight 10.8 before the first block ranked alone, 8.2 since; 251 pages: one 6.0, two 9.2; 128
    // lists of 2048: one 24, two 37).
    int cluster = 1;
    const int64_t lists = static_cast<int64_t>(p.table.batch) * p.cache.heads;
    if (p.table.width > 512)
        while (cluster < 8 && 2 * cluster * lists <= rt.num_sms) cluster *= 2;
    while (cluster < 8 && cluster * (kChooseMaxPages / 8) < p.table.width) cluster *= 2;
    p.cached = (p.table.width + cluster - 1) / cluster;
    p.gather = cluster > 1 && p.table.width <= kChooseGather;
    if (p.gather) p.cached = p.table.width;
    // Where no SM has a second block, one of twice the warps (128 lists of 2048 pages: 23.2 -> 19.7 us; with 256 lists of up
    // to 2049 it would be 32.9, two blocks an SM take 30.6).
    if (lists * cluster <= rt.num_sms && p.table.width > 256 && p.group <= 8 &&
        ChooseShape<2 * kThreads, kChunks, 3>::bytes(p.cached, p.group, p.cache.dim) <= kChooseMaxBytes)
        return launch_choose_stages<2 * kThreads, kBf16, kChunks, 3, true>(rt, p, cluster, s);
    // Three stages let an SM have two blocks; the longest lists of large groups 256 wide leave room for two.
    if constexpr (kChunks > 2) {
        if (ChooseShape<kThreads, kChunks, 3>::bytes(p.cached, p.group, p.cache.dim) > kChooseMaxBytes)
            return launch_choose_stages<kThreads, kBf16, kChunks, 2, false>(rt, p, cluster, s);
        static_assert(ChooseShape<kThreads, kChunks, 2>::bytes(kChooseMaxPages / 8, kChooseGroup, 64 * kChunks) <= kChooseMaxBytes, "fits");
    } else {
        static_assert(ChooseShape<kThreads, kChunks, 3>::bytes(kChooseMaxPages / 8, kChooseGroup, 64 * kChunks) <= kChooseMaxBytes, "fits");
    }
    return p.group <= 8 ? launch_choose_stages<kThreads, kBf16, kChunks, 3, true>(rt, p, cluster, s)
                        : launch_choose_stages<kThreads, kBf16, kChunks, 3, false>(rt, p, cluster, s);
}

template <bool kBf16>
cudaError_t launch_choose(const RuntimeInfo &rt, ChooseParams &p, cudaStream_t s) {
    if (p.cache.dim <= 64) return launch_choose_shape<256, kBf16, 1>(rt, p, s);
    if (p.cache.dim <= 128) return launch_choose_shape<256, kBf16, 2>(rt, p, s);
    return launch_choose_shape<128, kBf16, 4>(rt, p, s);
}

}  // namespace

#ifdef TGEMM_DEBUG
int page_debug_last_check() {
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

extern "C" tgemm_status tgemm_kv_bounds(const tgemm_kv_bounds_args *a, tgemm_stream_t stream) {
    BoundsParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv, eb, es;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_cache(a->cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    const tgemm_kv_cache *cache = a->cache;
    st = check_bounds(a->bounds, cache, &p.bounds, &eb, &es);
    if (st != TGEMM_OK) return st;
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    if (!valid_dtype(a->dtype) || !countable(a->seq.batch, a->seq.pages_width)) return TGEMM_ERR_INVALID_ARG;
    if (a->seq.batch == 0 || a->seq.pages_width == 0) return TGEMM_OK;
    if (!aligned4(a->starts)) return TGEMM_ERR_ALIGNMENT;
    if (cache_overlaps(cache, ck, cv, eb) || cache_overlaps(cache, ck, cv, es) || overlaps(eb, es)) return TGEMM_ERR_ALIAS;
    const Extent ep = {a->seq.pages, ((a->seq.batch - 1) * a->seq.pages_stride + a->seq.pages_width) * 4};
    const Extent el = {a->seq.lengths, a->seq.batch * 4}, et = {a->starts, a->starts ? (a->seq.batch + 1) * 4 : 0};
    for (const Extent &x : {eb, es})
        if (overlaps_any(x, {ep, el, et})) return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->seq.pages, a->seq.lengths, a->starts, cache->k, cache->e4m3 ? cache->k_scale : nullptr,
                                a->bounds->bounds, a->bounds->scale}))
        return TGEMM_ERR_INVALID_ARG;
    p.starts = a->starts;
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cache->e4m3) return done(launch_bounds<false, true>(rt, p, s));
    return done(a->dtype == TGEMM_BF16 ? launch_bounds<true, false>(rt, p, s) : launch_bounds<false, false>(rt, p, s));
}

extern "C" tgemm_status tgemm_kv_select(const tgemm_kv_select_args *a, tgemm_stream_t stream) {
    ChooseParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv, eb, es;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_cache(a->cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    const tgemm_kv_cache *cache = a->cache;
    st = check_bounds(a->bounds, cache, &p.bounds, &eb, &es);
    if (st != TGEMM_OK) return st;
    const int64_t batch = a->seq.batch, q_heads = a->q_heads, keep = a->keep;
    if (!valid_dtype(a->dtype) || q_heads < 1 || q_heads > 65535 || q_heads % cache->heads != 0 ||
        q_heads / cache->heads > kChooseGroup || keep < 1 || keep > (1 << 30) || a->first < 0 || a->recent < 1 ||
        a->first > keep || a->recent > keep - a->first)
        return TGEMM_ERR_INVALID_ARG;
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    if (a->seq.pages_width > kChooseMaxPages) return TGEMM_ERR_INVALID_ARG;
    const int64_t qsize[2] = {batch, q_heads}, qstride[2] = {a->q_batch_stride, a->q_head_stride};
    const int64_t tsize[2] = {batch, cache->heads}, tstride[2] = {a->to_batch_stride, a->to_head_stride};
    int64_t qbytes = 0, tbytes = 0;
    if (!extent(qsize, qstride, 2, cache->dim, 2, false, &qbytes) || !extent(tsize, tstride, 2, keep, 4, true, &tbytes))
        return TGEMM_ERR_INVALID_ARG;
    if (batch == 0) return TGEMM_OK;
    if (!a->Q || !a->to_pages || !a->to_lengths) return TGEMM_ERR_INVALID_ARG;
    if (!aligned16(a->Q) || !aligned4(a->to_pages) || !aligned4(a->to_lengths) || (batch > 1 && a->q_batch_stride % 8 != 0) ||
        (q_heads > 1 && a->q_head_stride % 8 != 0))
        return TGEMM_ERR_ALIGNMENT;
    const Extent et = {a->to_pages, tbytes}, en = {a->to_lengths, batch * 4}, el = {a->seq.lengths, batch * 4}, eq = {a->Q, qbytes};
    const Extent ep = {a->seq.pages, ((batch - 1) * a->seq.pages_stride + a->seq.pages_width) * 4};
    for (const Extent &x : {et, en})
        if (cache_overlaps(cache, ck, cv, x) || overlaps(x, eb) || overlaps(x, es) || overlaps(x, el) || overlaps(x, ep) || overlaps(x, eq))
            return TGEMM_ERR_ALIAS;
    if (overlaps(et, en) || rows_meet(tsize, tstride, keep)) return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->Q, a->seq.pages, a->seq.lengths, a->bounds->bounds, a->bounds->scale, a->to_pages, a->to_lengths}))
        return TGEMM_ERR_INVALID_ARG;
    p.q = static_cast<const unsigned char *>(a->Q);
    p.q_batch_stride = a->q_batch_stride * 2;
    p.q_head_stride = a->q_head_stride * 2;
    p.group = static_cast<int>(q_heads / cache->heads);
    p.to_pages = a->to_pages;
    p.to_batch_stride = a->to_batch_stride;
    p.to_head_stride = a->to_head_stride;
    p.to_lengths = a->to_lengths;
    p.keep = static_cast<int>(keep);
    p.first = static_cast<int>(a->first);
    p.recent = static_cast<int>(a->recent);
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return done(a->dtype == TGEMM_BF16 ? launch_choose<true>(rt, p, s) : launch_choose<false>(rt, p, s));
}

// ---------------------------------------------------------------- pages
namespace {

// What fork, grow and free share: the cache, the counts and the lists that change.
tgemm_status check_pages(const tgemm_kv_cache *cache, int32_t *uses, int32_t *pages, int32_t *lengths, int64_t width, int64_t stride,
                         int64_t batch, PagesParams *p, Extent *lists) {
    Extent ck, cv;
    tgemm_status st = check_cache(cache, &p->cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    if (!countable_pool(cache)) return TGEMM_ERR_INVALID_ARG;
    if (!cache->e4m3) p->cache.k_scale = p->cache.v_scale = nullptr;      // the kernels go by them
    st = check_lists(pages, lengths, width, stride, batch, cache->page_size, &p->to, lists);
    if (st != TGEMM_OK) return st;
    if (cache->pages > 0 && !uses) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(uses)) return TGEMM_ERR_ALIGNMENT;
    const Extent eu = {uses, static_cast<int64_t>(cache->pages) * 4}, en = {lengths, batch * 4};
    for (const Extent &x : {eu, en, *lists})
        if (cache_overlaps(cache, ck, cv, x)) return TGEMM_ERR_ALIAS;
    if (overlaps(eu, en) || overlaps(eu, *lists) || overlaps(en, *lists)) return TGEMM_ERR_ALIAS;
    p->uses = uses;
    return TGEMM_OK;
}

// Where there is little to do, a cluster does all in one launch, which saves 2 us of the host's time; beyond, two launches
// fill the GPU.  Both sides below as called among others, and on the GPU alone.
//
// Fork: one child for each of the cluster's blocks, lists of up to 1024 pages, 1 MB of the children's last pages.  With
// freeing, pages of 32 KB: 8 children, lists of 32 pages 10.6 us (two launches 12.4; on the GPU 8.0, 7.7), of 512 10.5
// (12.4; 8.9, 9.4), of 2048 13.2 (13.1; 12.8, 12.1); 32 children 12.6 (12.3; 11.9, 8.1), 128 of 2 KB 29 (8 on the GPU).
constexpr int64_t kForkFew = 1 << 20, kForkChildren = kForkBlocks, kForkList = 1024;
// Compaction: pools of up to 160 pages and 4 MB (half of them move at most), 8 sequences.  Pages of 16 KB: a pool of 29 6.6 us
// (two launches 8.4; on the GPU 5.0, 4.9), of 138 7.4 (8.5; 7.3, 4.9), of 413 15 (8.4; 15, 5.6); 16 sequences on 106 pages
// 7.3 to 8.6 (8.5), 64 10.7 (8.4).
constexpr int64_t kCompactFew = 4 << 20, kCompactPages = 160, kCompactLists = 8;

template <int kLanes>
cudaError_t launch_fork_lanes(const RuntimeInfo &rt, const PagesParams &p, cudaStream_t s) {
    const int64_t page_bytes = static_cast<int64_t>(p.cache.page_size) * p.cache.heads * p.cache.row_bytes * 2;
    if (p.to.batch <= kForkChildren && p.table.width <= kForkList && p.to.batch * page_bytes <= kForkFew)
        return launch(page_fork_few_kernel<kLanes>, dim3(kForkBlocks), kTakeThreads, 0, s, p, kForkBlocks);
    const cudaError_t e = launch(page_take_kernel<true>, dim3(1), kTakeThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    constexpr int kRows = kPageThreads / kLanes * 4;
    const int64_t rows = static_cast<int64_t>(p.cache.page_size) * p.cache.heads;
    const int64_t want = std::max<int64_t>((rows + kRows - 1) / kRows, (p.table.width + kPageThreads - 1) / kPageThreads);
    const int64_t most = std::max<int64_t>(1, static_cast<int64_t>(rt.num_sms) * 16 / p.to.batch);
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min(want, most))), static_cast<unsigned>(p.to.batch));
    return launch(page_fork_kernel<kLanes>, grid, kPageThreads, 0, s, p);
}

template <int kLanes>
cudaError_t launch_move_lanes(const RuntimeInfo &rt, const CompactParams &p, cudaStream_t s) {
    const int64_t page_bytes = static_cast<int64_t>(p.cache.page_size) * p.cache.heads * p.cache.row_bytes * 2;
    if (p.cache.pages <= kCompactPages && p.cache.pages * page_bytes <= kCompactFew && p.table.batch <= kCompactLists)
        return launch(page_compact_few_kernel<kLanes>, dim3(kForkBlocks), kTakeThreads, 0, s, p, kForkBlocks);
    const cudaError_t e = p.cache.pages <= kTakeThreads ? launch(page_plan_kernel<1>, dim3(1), kTakeThreads, 0, s, p)
                                                        : launch(page_plan_kernel<kTakeDeep>, dim3(1), kTakeThreads, 0, s, p);
    if (e != cudaSuccess) return e;
    constexpr int kRows = kPageThreads / kLanes * 4;
    const int64_t rows = static_cast<int64_t>(p.cache.page_size) * p.cache.heads;
    const int64_t want = std::max<int64_t>((rows + kRows - 1) / kRows * ((p.cache.pages + 1) / 2), p.table.batch);
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, static_cast<int64_t>(rt.num_sms) * 6))));
    return launch(page_move_kernel<kLanes>, grid, kPageThreads, 0, s, p);
}

int64_t compact_bytes(int64_t pages) { return 256 + 3 * ((pages * 4 + 255) / 256 * 256); }

}  // namespace

extern "C" tgemm_status tgemm_kv_grow(const tgemm_kv_grow_args *a, tgemm_stream_t stream) {
    PagesParams p;
    std::memset(&p, 0, sizeof(p));
    Extent lists;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_pages(a->cache, a->uses, a->pages, a->lengths, a->pages_width, a->pages_stride, a->batch, &p, &lists);
    if (st != TGEMM_OK) return st;
    if (a->batch == 0) return TGEMM_OK;
    if (!aligned4(a->tokens)) return TGEMM_ERR_ALIGNMENT;
    const Extent et = {a->tokens, a->tokens ? a->batch * 4 : 0}, eu = {a->uses, static_cast<int64_t>(a->cache->pages) * 4};
    if (overlaps_any(et, {eu, lists, {a->lengths, a->batch * 4}})) return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->uses, a->pages, a->lengths, a->tokens})) return TGEMM_ERR_INVALID_ARG;
    p.fresh = a->tokens;
    p.status = rt.status;
    return done(launch(page_take_kernel<false>, dim3(1), kTakeThreads, 0, reinterpret_cast<cudaStream_t>(stream), p));
}

extern "C" tgemm_status tgemm_kv_fork(const tgemm_kv_fork_args *a, tgemm_stream_t stream) {
    PagesParams p;
    std::memset(&p, 0, sizeof(p));
    Extent lists;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_pages(a->cache, a->uses, a->to_pages, a->to_lengths, a->to_width, a->to_stride, a->children, &p, &lists);
    if (st != TGEMM_OK) return st;
    const tgemm_kv_cache *cache = a->cache;
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    if (!countable(a->seq.batch, a->seq.pages_width)) return TGEMM_ERR_INVALID_ARG;
    if (a->children == 0) return TGEMM_OK;
    if (!a->parents) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(a->parents)) return TGEMM_ERR_ALIGNMENT;
    if (cache->pages > 0 && cache->k == cache->v) return TGEMM_ERR_ALIAS;
    // What is read besides the parents' rows is apart from what is written; the children's lists and lengths may be rows of
    // the parents' arrays.
    const Extent ck = {cache->k, p.cache.dbg_bytes}, cv = {cache->v, p.cache.dbg_bytes}, eu = {a->uses, static_cast<int64_t>(cache->pages) * 4};
    const Extent en = {a->to_lengths, a->children * 4}, er = {a->parents, a->children * 4}, el = {a->seq.lengths, a->seq.batch * 4};
    const Extent ep = {a->seq.pages, a->seq.batch > 0 ? ((a->seq.batch - 1) * a->seq.pages_stride + a->seq.pages_width) * 4 : 0};
    if (overlaps_any(er, {eu, en, lists}) || overlaps_any(eu, {ep, el}) || overlaps(lists, el) || overlaps(en, ep)) return TGEMM_ERR_ALIAS;
    for (const Extent &x : {er, ep, el})
        if (cache_overlaps(cache, ck, cv, x)) return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->uses, a->to_pages, a->to_lengths, a->parents, a->seq.pages, a->seq.lengths, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    p.parents = a->parents;
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (row_lanes(p.cache.row_bytes)) {
        case 8: return done(launch_fork_lanes<8>(rt, p, s));
        case 16: return done(launch_fork_lanes<16>(rt, p, s));
        default: return done(launch_fork_lanes<32>(rt, p, s));
    }
}

extern "C" tgemm_status tgemm_kv_free(const tgemm_kv_free_args *a, tgemm_stream_t stream) {
    PagesParams p;
    std::memset(&p, 0, sizeof(p));
    Extent lists;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_pages(a->cache, a->uses, const_cast<int32_t *>(a->pages), a->lengths, a->pages_width, a->pages_stride,
                                  a->batch, &p, &lists);
    if (st != TGEMM_OK) return st;
    if (a->batch == 0) return TGEMM_OK;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->uses, a->pages, a->lengths})) return TGEMM_ERR_INVALID_ARG;
    p.status = rt.status;
    return done(launch(page_free_kernel, dim3(static_cast<unsigned>(a->batch)), kPageThreads, 0, reinterpret_cast<cudaStream_t>(stream), p));
}

extern "C" tgemm_status tgemm_kv_compact_workspace(int64_t pages, int64_t *bytes) {
    if (!bytes || pages < 0 || pages > INT32_MAX) return TGEMM_ERR_INVALID_ARG;
    *bytes = compact_bytes(pages);
    return TGEMM_OK;
}

extern "C" tgemm_status tgemm_kv_compact(const tgemm_kv_compact_args *a, tgemm_stream_t stream) {
    CompactParams p;
    std::memset(&p, 0, sizeof(p));
    Extent ck, cv, eb, es;
    if (!a) return TGEMM_ERR_INVALID_ARG;
    tgemm_status st = check_cache(a->cache, &p.cache, &ck, &cv);
    if (st != TGEMM_OK) return st;
    const tgemm_kv_cache *cache = a->cache;
    if (!countable_pool(cache)) return TGEMM_ERR_INVALID_ARG;
    if (!cache->e4m3) p.cache.k_scale = p.cache.v_scale = nullptr;        // the kernels go by them
    if (a->bounds) {
        st = check_bounds(a->bounds, cache, &p.bounds, &eb, &es);
        if (st != TGEMM_OK) return st;
    }
    st = check_sequences(a->seq, true, cache->page_size, &p.table);
    if (st != TGEMM_OK) return st;
    const int64_t batch = a->seq.batch, pages = cache->pages;
    if (!countable(batch, a->seq.pages_width) || a->to_width < a->seq.pages_width || a->to_width > INT32_MAX || a->to_stride < 0 ||
        a->to_stride > (int64_t(1) << 40) || (batch > 1 && a->to_stride < a->to_width))
        return TGEMM_ERR_INVALID_ARG;
    const int64_t need = compact_bytes(pages);
    if ((batch > 0 && a->seq.pages_width > 0 && !a->to_pages) || (pages > 0 && (!a->uses || !a->to_uses)) || !a->in_use || !a->workspace ||
        a->workspace_bytes < need)
        return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(a->uses) || !aligned4(a->to_uses) || !aligned4(a->in_use) || !aligned4(a->to_pages) || !aligned16(a->workspace))
        return TGEMM_ERR_ALIGNMENT;
    const Extent eu = {a->uses, pages * 4}, etu = {a->to_uses, pages * 4}, ei = {a->in_use, 4}, ew = {a->workspace, need};
    const Extent ep = {a->seq.pages, batch > 0 ? ((batch - 1) * a->seq.pages_stride + a->seq.pages_width) * 4 : 0};
    const Extent etp = {a->to_pages, batch > 0 ? ((batch - 1) * a->to_stride + a->to_width) * 4 : 0};
    const Extent el = {a->seq.lengths, batch * 4};
    const Extent all[] = {eu, etu, ei, ew, ep, etp, el};
    for (const Extent &x : all)
        if (cache_overlaps(cache, ck, cv, x) || (a->bounds && (overlaps(x, eb) || overlaps(x, es)))) return TGEMM_ERR_ALIAS;
    if (a->bounds && (cache_overlaps(cache, ck, cv, eb) || cache_overlaps(cache, ck, cv, es) || overlaps(eb, es))) return TGEMM_ERR_ALIAS;
    // The counts and the lists may be replaced in place; otherwise what is written is apart from all else.
    const bool same_uses = a->uses == a->to_uses, same_lists = a->to_pages == a->seq.pages && a->to_stride == a->seq.pages_stride;
    if ((cache->pages > 0 && cache->k == cache->v) || (!same_uses && overlaps(eu, etu)) || (!same_lists && overlaps(ep, etp)))
        return TGEMM_ERR_ALIAS;
    if (overlaps(etu, ei) || overlaps(etu, ew) || overlaps(etu, ep) || overlaps(etu, etp) || overlaps(etu, el) || overlaps(ei, eu) ||
        overlaps(ei, ew) || overlaps(ei, ep) || overlaps(ei, etp) || overlaps(ei, el) || overlaps(ew, eu) || overlaps(ew, ep) ||
        overlaps(ew, etp) || overlaps(ew, el) || overlaps(etp, eu) || overlaps(etp, el))
        return TGEMM_ERR_ALIAS;
    RuntimeInfo rt;
    st = runtime_current(&rt);
    if (st != TGEMM_OK) return st;
    if (!all_device(rt.device, {a->uses, a->to_uses, a->in_use, a->workspace, a->seq.pages, a->to_pages, a->seq.lengths, cache->k, cache->v,
                                cache->e4m3 ? cache->k_scale : nullptr, cache->e4m3 ? cache->v_scale : nullptr,
                                a->bounds ? a->bounds->bounds : nullptr, a->bounds ? a->bounds->scale : nullptr}))
        return TGEMM_ERR_INVALID_ARG;
    unsigned char *const ws = static_cast<unsigned char *>(a->workspace);
    const int64_t each = (pages * 4 + 255) / 256 * 256;
    p.head = reinterpret_cast<int *>(ws);
    p.below = reinterpret_cast<int *>(ws + 256);
    p.above = reinterpret_cast<int *>(ws + 256 + each);
    p.map = reinterpret_cast<int *>(ws + 256 + 2 * each);
    p.uses = a->uses;
    p.to_uses = a->to_uses;
    p.in_use = a->in_use;
    p.to.pages = a->to_pages;
    p.to.stride = a->to_stride;
    p.to.width = static_cast<int>(a->to_width);
    p.to.batch = static_cast<int>(batch);
    p.slots_first = cache->slot_stride < cache->head_stride;
    p.status = rt.status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (row_lanes(p.cache.row_bytes)) {
        case 8: return done(launch_move_lanes<8>(rt, p, s));
        case 16: return done(launch_move_lanes<16>(rt, p, s));
        default: return done(launch_move_lanes<32>(rt, p, s));
    }
}
