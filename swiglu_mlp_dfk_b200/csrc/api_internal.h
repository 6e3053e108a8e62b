// api_internal.h -- what the entry points outside dfk_api.cu share with it:
// error reporting, the current device, tensor maps, launch attributes.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace dfk {

// Records the formatted text as this thread's dfk_last_error; returns `status`.
int api_fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

// A failed CUDA call as DFK_ERR_CUDA (clears CUDA's own last error).
int api_cuda_error(cudaError_t e, const char *what);

// The current device: DFK_OK with its SM count and status block, or
// DFK_ERR_ARCH.
int api_device(int *sms, unsigned **err);

// 2-D tensor map over bytes: `inner` bytes a row, `outer` rows `pitch` bytes
// apart, box of box_inner x box_outer, 128-byte swizzle, zero fill outside.
// Encoded on every call (a few hundred nanoseconds on the host).
int api_tensor_map_u8(const void *ptr, uint64_t inner, uint64_t outer, uint64_t pitch,
                      uint32_t box_inner, uint32_t box_outer, CUtensorMap *out);

// Lets `fn` use the device's whole shared memory (once per device and kernel).
int api_allow_smem(const void *fn);

// Programmatic dependent launch, unless DFK_PDL=0.
bool api_pdl();

}  // namespace dfk
