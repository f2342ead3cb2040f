// Per-device library state and the watchdog settings, shared by the C entry
// points (host side).  Defined in api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace tmmo {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int num_sms = 0;
    int* status = nullptr;  // the device status word of the bounded waits
    bool ready = false;
};

// Set-up of the current device, once: SM count and the status word address.
cudaError_t device_info(DeviceInfo* out);

// The settings of gemm_debug_config.
long long wait_budget_cycles();
int fault_skip_kblock();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace tmmo
