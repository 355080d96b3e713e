// What the translation units of the library share on the host: the device's
// properties and status word, and the pointer check of the entry points
// (defined in tgemm_api.cu).
#pragma once
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

// Whether the driver knows p as memory that kernels on `device` can use.
bool runtime_is_device_memory(const void *p, int device);

#ifdef TGEMM_DEBUG
// Debug build: reads and clears the first failed check of kv_api.cu's kernels.
int kv_debug_last_check();
#endif

}  // namespace tgemm
