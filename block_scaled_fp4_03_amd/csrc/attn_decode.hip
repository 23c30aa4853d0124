// attn_decode.hip -- attention of one new token per sequence over the paged
// key-value cache.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"

namespace fp4 {
namespace {


// Element d of cache row `row`.
__device__ __forceinline__ float kv_value(const KvPool& c, const void* pool, const uint8_t* scales, uint64_t row,
                                          uint32_t d) {
  const uint32_t D = (uint32_t)c.head_dim;
  if (c.fmt == kKvBf16) return u2f((uint32_t) static_cast<const uint16_t*>(pool)[row * D + d] << 16);
  const float s = u2f((uint32_t)scales[row * (D / 32u) + d / 32u] << 23);
  if (c.fmt == kKvMx8) {
    const uint32_t b = static_cast<const uint8_t*>(pool)[row * D + d];
    return (b & 0x80u ? -e4m3_value(b & 0x7Fu) : e4m3_value(b)) * s;
  }
  const uint32_t b = (static_cast<const uint8_t*>(pool)[(row * D + d) / 2u] >> (4u * (d & 1u))) & 15u;
  return (b & 8u ? -e2m1_grid(b & 7u) : e2m1_grid(b)) * s;
}

__device__ __forceinline__ float wave_sum(float v) {
  for (int i = 32; i > 0; i >>= 1) v += __shfl_xor(v, i);
  return v;
}

// One workgroup per sequence and kv head; its four waves take every fourth
// token, one query head of the group after the other.
__global__ __launch_bounds__(256) void attn_simple_kernel(KvPool c, const void* q, int q_dtype, int64_t q_stride,
                                                          const int32_t* table, int64_t width, const int32_t* lens,
                                                          int64_t q_heads, int64_t max_len, int64_t window,
                                                          float scale, void* out, int out_dtype, float* lse,
                                                          const float* w_in, float* w_out, int64_t w_stride) {
  __shared__ float part[4][256 + 2];
  const uint32_t h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  const uint32_t D = (uint32_t)c.head_dim, group = (uint32_t)(q_heads / c.kv_heads);
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)c.page_size);
  const int64_t len = lens[b] < 0 ? 0 : (lens[b] < max_len ? lens[b] : max_len);
  const int64_t first = window > 0 && window < len ? len - window : 0;
  for (uint32_t g = 0; g < group; ++g) {
    const uint32_t qh = h * group + g;
    float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.0f;
    for (uint32_t i = 0; i < D / 64u; ++i) {
      const size_t at = (size_t)b * q_stride + qh * D + i * 64u + lane;
      qv[i] = q_dtype == kDtF32 ? static_cast<const float*>(q)[at]
                                : u2f((uint32_t) static_cast<const uint16_t*>(q)[at] << 16);
    }
    for (int pass = 0; pass < (w_out ? 2 : 1); ++pass) {
      for (int64_t t = pass == 0 ? first + wave : wave; t < len; t += 4) {
        const int32_t page = table[(size_t)b * width + (t >> shift)];
        const bool ok = t >= first && page >= 0 && page < c.pages;
        float s = 0.0f;
        const uint64_t row =
            ok ? (((uint64_t)(uint32_t)page * c.kv_heads + h) << shift) + (t & (c.page_size - 1)) : 0u;
        if (ok) {
          for (uint32_t i = 0; i < D / 64u; ++i)
            s = __builtin_fmaf(qv[i], kv_value(c, c.k, c.ks, row, i * 64u + lane), s);
          s = wave_sum(s) * scale;
        }
        if (pass == 1) {
          const size_t at = ((size_t)b * c.kv_heads + h) * w_stride + t;
          const float p = ok ? expf(s - m) / l : 0.0f;
          if (lane == 0) w_out[at] = (g == 0 ? (w_in ? w_in[at] : 0.0f) : w_out[at]) + p;
        } else if (ok) {
          const float m1 = fmaxf(m, s), f = m1 == -INFINITY ? 1.0f : expf(m - m1), p = expf(s - m1);
          l = l * f + p;
          for (uint32_t i = 0; i < D / 64u; ++i)
            acc[i] = acc[i] * f + p * kv_value(c, c.v, c.vs, row, i * 64u + lane);
          m = m1;
        }
      }
      if (pass == 1) break;
      for (uint32_t i = 0; i < D / 64u; ++i) part[wave][2 + i * 64u + lane] = acc[i];
      if (lane == 0) {
        part[wave][0] = m;
        part[wave][1] = l;
      }
      __syncthreads();
      m = fmaxf(fmaxf(part[0][0], part[1][0]), fmaxf(part[2][0], part[3][0]));
      l = 0.0f;
      for (int i = 0; i < 4; ++i)
        if (part[i][1] != 0.0f) l += part[i][1] * expf(part[i][0] - m);
      for (uint32_t d = threadIdx.x; d < D; d += 256u) {
        float o = 0.0f;
        for (int i = 0; i < 4; ++i)
          if (part[i][1] != 0.0f) o += part[i][2 + d] * (expf(part[i][0] - m) / l);
        const size_t at = ((size_t)b * q_heads + qh) * D + d;
        if (out_dtype == kDtF32)
          static_cast<float*>(out)[at] = o;
        else
          static_cast<uint16_t*>(out)[at] = (uint16_t)bf16_pair(o, 0.0f);
      }
      if (threadIdx.x == 0 && lse) lse[(size_t)b * q_heads + qh] = l == 0.0f ? -INFINITY : m + logf(l);
      __syncthreads();
    }
    __syncthreads();
  }
}

}  // namespace

size_t attn_decode_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_attn_decode(const KvPool& c, const void* q, int q_dtype, int64_t q_stride, const int32_t* table,
                              int64_t width, const int32_t* lens, int64_t B, int64_t q_heads, int64_t max_len,
                              int64_t window, float scale, void* out, int out_dtype, float* lse,
                              const float* weights_in, float* weights_out, int64_t weights_stride, void*,
                              hipStream_t stream) {
  attn_simple_kernel<<<dim3((uint32_t)c.kv_heads, (uint32_t)B), 256, 0, stream>>>(
      c, q, q_dtype, q_stride, table, width, lens, q_heads, max_len, window, scale, out, out_dtype, lse, weights_in,
      weights_out, weights_stride);
  return hipGetLastError();
}

}  // namespace fp4
