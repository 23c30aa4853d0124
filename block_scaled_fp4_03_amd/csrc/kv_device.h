// kv_device.h -- row formats of the paged key-value cache, shared by the
// kernels that write, read and move its rows.  Internal header.
#pragma once

#include "fp4_device.h"

namespace fp4 {

// The C ABI's fp4_kv_fmt values.
constexpr int kKvBf16 = 0, kKvMx8 = 1, kKvMx4 = 2;

// Code bytes of a cache row of D values.
__host__ __device__ constexpr uint32_t kv_row_bytes(int fmt, uint32_t D) {
  return fmt == kKvBf16 ? 2u * D : fmt == kKvMx8 ? D : D / 2u;
}

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

// Two FP32 values rounded to BF16 (nearest even, NaN kept), a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}

}  // namespace fp4
