// The host side of the functions that place the paged cache's outputs, for
// tests on a machine without a GPU.
#include "../gemm_epilogue_02_gb300/csrc/kv_attend.cuh"
#include "../gemm_epilogue_02_gb300/csrc/kv_evict.cuh"

extern "C" int check_kept_place(int larger, int ties, int need, int best, int *at) {
    return tgemm::kv_kept_place(larger, ties, need, best, at) ? 1 : 0;
}
