// What the translation units of the library share on the host: the device's
// properties and status word, and the pointer check of the entry points
// (defined in tgemm_api.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tgemm.h"

namespace tgemm {

struct RuntimeInfo {
    int device = 0;
    int num_sms = 0;
    unsigned int *status = nullptr;   // device address of the status word
};

// The current device, or TGEMM_ERR_UNSUPPORTED_DEVICE.
tgemm_status runtime_current(RuntimeInfo *out);

// While it lives, the thread may make calls that a stream capture in progress
// would otherwise fail at (and be failed by): looking up symbols, setting kernel
// attributes.  None of them is recorded.
class RelaxedCapture {
public:
    RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    RelaxedCapture(const RelaxedCapture &) = delete;
    RelaxedCapture &operator=(const RelaxedCapture &) = delete;

private:
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
};

// Whether the driver knows p as memory that kernels on `device` can use.
bool runtime_is_device_memory(const void *p, int device);

#ifdef TGEMM_DEBUG
// Debug build: reads and clears the first failed check of kv_api.cu's kernels.
int kv_debug_last_check();
#endif

}  // namespace tgemm
