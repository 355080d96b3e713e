// What the entry points of the paged key-value cache share on the host: the
// checks of a call's description and the launch of a kernel.
#pragma once
#include <cuda_runtime.h>

#include <cstring>
#include <initializer_list>

#include "../../include/tgemm.h"
#include "kv_cache.cuh"
#include "runtime.h"

namespace tgemm {

constexpr int64_t kMost = int64_t(1) << 61;       // bytes: no valid allocation is that large

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Extent {
    const void *base = nullptr;
    int64_t bytes = 0;
};

inline bool overlaps(const Extent &a, const Extent &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
    return a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
           y < x + static_cast<uintptr_t>(a.bytes);
}

// Bytes from the first element to the end of the last of a strided array: sum
// of (size - 1) * stride, plus a run of `width`, in elements of `esize` bytes.
// False for a negative size or stride, one too large, or, with `apart`, a
// stride below `width` (elements of different rows would share memory).
inline bool extent(const int64_t *size, const int64_t *stride, int dims, int64_t width, int64_t esize, bool apart,
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

// Whether rows of `width` elements in two dimensions share memory, with strides that extent() has found apart for each
// dimension alone.
inline bool rows_meet(const int64_t (&size)[2], const int64_t (&stride)[2], int64_t width) {
    if (size[0] < 2 || size[1] < 2) return false;
    const int a = size[0] <= size[1] ? 0 : 1, b = 1 - a, outer = stride[0] >= stride[1] ? 0 : 1;
    if (stride[outer] - (size[1 - outer] - 1) * stride[1 - outer] >= width) return false;     // all of one between two of the other
    // `e` steps along a against the steps along b that come nearest.
    for (int64_t e = 1; e < size[a]; ++e) {
        const int64_t to = e * stride[a], d = to / stride[b], rest = to - d * stride[b];
        if ((d > 0 && d < size[b] && rest < width) || (d + 1 < size[b] && stride[b] - rest < width)) return true;
    }
    return false;
}

// Checks a cache's description and fills the kernels' view of it.
inline tgemm_status check_cache(const tgemm_kv_cache *c, KvView *view, Extent *k, Extent *v) {
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
inline tgemm_status check_sequences(const tgemm_kv_sequences &q, bool with_lengths, int page_size, KvTable *t) {
    if (q.batch < 0 || q.batch > 65535 || q.pages_width < 0 || q.pages_width > (1 << 30) / page_size ||
        q.pages_stride < 0 || (q.batch > 1 && q.pages_stride < q.pages_width) || q.pages_stride > (int64_t(1) << 40))
        return TGEMM_ERR_INVALID_ARG;
    if (q.batch > 0 && ((q.pages_width > 0 && !q.pages) || (with_lengths && !q.lengths))) return TGEMM_ERR_INVALID_ARG;
    if (!aligned4(q.pages) || !aligned4(q.lengths)) return TGEMM_ERR_ALIGNMENT;
    t->pages = q.pages;
    t->lengths = q.lengths;
    t->stride = q.pages_stride;
    t->head_stride = 0;
    t->width = static_cast<int>(q.pages_width);
    t->batch = static_cast<int>(q.batch);
    return TGEMM_OK;
}

inline tgemm_status check_weights(const tgemm_kv_weights &a, int64_t batch, int64_t heads, KvWeights *w, Extent *e) {
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

inline bool valid_dtype(int64_t d) { return d == TGEMM_F16 || d == TGEMM_BF16; }

inline bool all_device(int device, std::initializer_list<const void *> ps) {
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

inline tgemm_status done(cudaError_t e) {
    if (e == cudaSuccess) return TGEMM_OK;
    cudaGetLastError();
    return TGEMM_ERR_CUDA;
}

}  // namespace tgemm
