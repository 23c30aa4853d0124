// host_device.h -- FP4_HOST_DEVICE marks a function of plain whole-number
// arithmetic that the kernels, the host and the CPU tests all compile.
// Internal header.
#pragma once

#include <cstddef>
#include <cstdint>

#if defined(__HIP__)
#include <hip/hip_runtime.h>
#define FP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FP4_HOST_DEVICE inline
#endif
