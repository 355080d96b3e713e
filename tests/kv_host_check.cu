// The host side of the functions that guard the paged cache's addresses, for
// tests on a machine without a GPU.
#include "../gemm_epilogue_02_gb300/csrc/kv_append.cuh"
#include "../gemm_epilogue_02_gb300/csrc/kv_attend.cuh"
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

extern "C" int check_tiles(int n, int window, int tile, int pad, int *lo) {
    return tgemm::attend_tiles(n, window, tile, pad, lo);
}

extern "C" long long check_first(long long c, long long ctas, long long total) {
    return tgemm::attend_first(c, ctas, total);
}

extern "C" int check_owner(long long t, long long ctas, long long total) { return tgemm::attend_owner(t, ctas, total); }

extern "C" int check_slot(int c, int first, int lane, int lanes) {
    return tgemm::attend_slot(c, first, lane, lanes);
}

extern "C" void check_limits(int *out) {
    out[0] = tgemm::kAttendMaxCtas;
    out[1] = tgemm::kAttendFanIn;
    out[2] = tgemm::kAttendLengths;
}

extern "C" int check_length_of(int k) { return tgemm::attend_length(k); }

extern "C" int check_pad(const long long *units, long long total, int runs) { return tgemm::attend_pad(units, total, runs); }
