// Host helpers shared by the translation units of the C ABI (defined in dg_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dg.h"
#include "dg_tuning.h"

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

// Tuning knobs (dg_tuning.h): the knob's value, or DG_TUNE_AUTO (-1) for the automatic choice.
int tune(int knob);

// A launch that may begin while the previous grid in the stream ends (the kernel waits for it before its first
// access to global memory), unless the DG_TUNE_PDL knob is 0.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tune(DG_TUNE_PDL) != 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace dg
