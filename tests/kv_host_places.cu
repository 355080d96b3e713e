// The host side of the functions that place the paged cache's outputs, for
// tests on a machine without a GPU.
#include "../gemm_epilogue_02_gb300/csrc/kv_attend.cuh"
#include "../gemm_epilogue_02_gb300/csrc/kv_evict.cuh"

extern "C" int check_kept_place(int larger, int ties, int need, int best, int *at) {
    return tgemm::kv_kept_place(larger, ties, need, best, at) ? 1 : 0;
}

extern "C" long long check_scored(int lo, int tile, int tile_size, int in_tile, long long positions) {
    return tgemm::attend_scored(lo, tile, tile_size, in_tile, positions);
}

extern "C" int check_fan(int parts) { return tgemm::attend_fan(parts); }

extern "C" int check_slot(int c, int first, int lane, int lanes) { return tgemm::attend_slot(c, first, lane, lanes); }

extern "C" void check_join_limits(int *out) {
    out[0] = tgemm::kAttendMaxCtas;
    out[1] = tgemm::kAttendFanIn;
    out[2] = tgemm::kAttendOneLevel;
}
