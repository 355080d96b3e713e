// Eviction's selection alone, for a test of what the compiler makes of it.
#include "../gemm_epilogue_02_gb300/csrc/kv_evict.cuh"

template __global__ void tgemm::kv_select_kernel<256, true>(const tgemm::EvictParams);
template __global__ void tgemm::kv_select_kernel<1024, true>(const tgemm::EvictParams);
template __global__ void tgemm::kv_select_kernel<1024, false>(const tgemm::EvictParams);
