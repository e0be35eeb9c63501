// What the C ABI's source files share: the HIP error of the calling thread and
// the current device's size.
#pragma once

#include <hip/hip_runtime.h>

namespace sdt {

struct DeviceInfo {
    int num_cu = 0;
    int nxcd = 1;
};

// Records e for sdt_last_hip_error() and returns SDT_ERR_HIP.
int fail_hip(hipError_t e);

// CU and XCD count of the current device, read once per device; an sdt_status.
int device_info(DeviceInfo* out);

}  // namespace sdt
