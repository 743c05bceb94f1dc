// Host helpers shared by the translation units of the C ABI (defined in dg_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg.h"

namespace dg {

constexpr int MAX_ROUTE_EXPERTS = 1024;
constexpr int MAX_ROUTE_K = 32;
constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready = false;
    bool supported = false;
    int sms = 0;
    int l2_bytes = 0;
    int* status = nullptr;
};

// The current device's properties; DG_NO_DEVICE_SUPPORT when it is not compute capability 10.3.
dg_status device_info(DeviceInfo* out);

// device_info, and the tensor-map encoder looked up.
dg_status common_prologue(DeviceInfo* dev);

// Row-major e4m3 matrix [rows, k] (k contiguous) read in boxes of box_rows x 128 with the 128-byte
// swizzle the MMA descriptors expect.
dg_status make_operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t k, int box_rows);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace dg
