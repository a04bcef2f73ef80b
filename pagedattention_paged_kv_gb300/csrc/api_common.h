// api_common.h -- host-side pieces shared by the files with extern "C" entry points
// (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

// Facts of the current device and its error word, looked up once per device.
struct DeviceFacts {
    int sms;
    int *err;
};
int current_device(DeviceFacts *out);  // PKV_OK or PKV_ERR_CUDA

// A tiled tensor map with 128-byte swizzle, unit element strides and zero fill.
// dims, box: `rank` entries, innermost first; strides: rank - 1 entries in bytes.
int encode_tiled(CUtensorMap *map, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                 const uint32_t *box);

uint64_t wait_limit_ns();  // pkv_set_wait_limit_ns

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace pkv
