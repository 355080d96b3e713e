// The host side of the functions that guard the paged cache's addresses, for
// tests on a machine without a GPU.
#include "../gemm_epilogue_02_gb300/csrc/kv_append.cuh"
#include "../gemm_epilogue_02_gb300/csrc/kv_cache.cuh"
#include "../gemm_epilogue_02_gb300/csrc/kv_evict.cuh"

extern "C" int check_length(int length, int width, int page_size, int *out) {
    bool bad = false;
    *out = tgemm::kv_length(length, width, page_size, &bad);
    return bad ? 1 : 0;
}

extern "C" int check_row(const int *list, int pos, int page_size, long long pages, int *page, int *slot) {
    return tgemm::kv_row(list, pos, page_size, pages, page, slot) ? 1 : 0;
}

extern "C" int check_sequence(const int *starts, int batch, long long t) {
    return tgemm::kv_sequence_of(starts, batch, t);
}

extern "C" unsigned check_key(unsigned bits) { return tgemm::kv_weight_key(bits); }
