// The paged key-value cache as the kernels see it, and the one place that
// turns a position of a sequence into the address of its rows.
//
// A cache is two pools of rows, keys and values.  A row holds `dim` elements of
// one head at one position and lies at
//     page * page_stride + slot * slot_stride + head * head_stride   (bytes),
// with position = 'index into the sequence's page list' * page_size + slot.  An
// e4m3 cache has one fp32 scale per row beside each pool (value = scale *
// element), addressed the same way by its own strides.
//
// Page lists and lengths live on the device, where the host cannot check them:
// every use goes through kv_row() / kv_length(), which refuse what lies outside
// the pool, so that a wrong page number is recorded (TGEMM_ERR_CACHE) and its
// row left out instead of read.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "debug_checks.cuh"
#include "ptx.cuh"

namespace tgemm {

constexpr uint32_t kStatusCache = 9;   // TGEMM_ERR_CACHE

struct KvView {
    unsigned char *k, *v;
    float *k_scale, *v_scale;                                      // e4m3 only
    long long pages;
    long long page_stride, slot_stride, head_stride;               // bytes
    long long scale_page_stride, scale_slot_stride, scale_head_stride;   // floats
    int page_size, heads, dim;
    int row_bytes;                                                 // dim elements
    long long dbg_bytes;                                           // debug builds: a pool's bytes
};

// The sequences' page lists and lengths.
struct KvTable {
    const int *pages;          // [batch, stride], `width` columns used
    const int *lengths;        // [batch]
    long long stride;
    long long head_stride;     // between the lists of a sequence's heads (attention; 0: the heads share one)
    int width;
    int batch;
};

// The accumulated attention weights [batch, heads, width] (base null: none).
struct KvWeights {
    float *base;
    long long batch_stride, head_stride;
    int width;
};

// A sequence's length: what its page list can hold at most, 0 when negative
// (*bad is set when it had to be cut).
__host__ __device__ inline int kv_length(int length, int width, int page_size, bool *bad) {
    const long long room = static_cast<long long>(width) * page_size;
    if (length < 0) {
        *bad = true;
        return 0;
    }
    if (length > room) {
        *bad = true;
        return static_cast<int>(room);
    }
    return length;
}

// Where position `pos` (0 <= pos < width * page_size) of a sequence lies: its
// page and slot; false when the list names a page outside the pool.
__host__ __device__ inline bool kv_row(const int *list, int pos, int page_size, long long pages, int *page,
                                       int *slot) {
    const int i = static_cast<int>(static_cast<unsigned>(pos) / static_cast<unsigned>(page_size));
    *page = list[i];
    *slot = pos - i * page_size;
    return *page >= 0 && *page < pages;
}

__host__ __device__ inline long long kv_offset(const KvView &c, int page, int slot, int head) {
    return page * c.page_stride + slot * c.slot_stride + head * c.head_stride;
}

__host__ __device__ inline long long kv_scale_offset(const KvView &c, int page, int slot, int head) {
    return page * c.scale_page_stride + slot * c.scale_slot_stride + head * c.scale_head_stride;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

}  // namespace tgemm
