// The host side of the functions that guard the pages' addresses and decide
// their bounds, for tests on a machine without a GPU.
#include "../gemm_epilogue_02_gb300/csrc/page_bounds.cuh"
#include "../gemm_epilogue_02_gb300/csrc/page_pool.cuh"

extern "C" float check_scale(float top) { return tgemm::kv_bounds_scale(top); }

extern "C" int check_completed(int n, long long fresh, int page_size, int *from) {
    return tgemm::kv_completed(n, fresh, page_size, from);
}

extern "C" void check_span(int n, int page_size, int keep, int first, int recent, int *out) {
    const tgemm::ChooseSpan s = tgemm::choose_span(n, page_size, keep, first, recent);
    out[0] = s.count, out[1] = s.keep, out[2] = s.first, out[3] = s.middle, out[4] = s.best;
}

extern "C" int check_fork(const int *lengths, int batch, int parent, int width, int page_size, int to_width, int *bad) {
    bool b = false;
    const int n = tgemm::fork_length(lengths, batch, parent, width, page_size, to_width, &b);
    *bad = b;
    return n;
}

extern "C" int check_pages(int n, int page_size) { return tgemm::kv_pages_of(n, page_size); }
