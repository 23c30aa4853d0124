// logprobs.hip -- log probabilities of given tokens, entropy and the largest
// alternatives, and their gradient.
#include "fp4_device.h"
#include "fp4_launch.h"

namespace fp4 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <int DT>
__device__ __forceinline__ float logit(const void* x, size_t i) {
  if (DT == kDtF32) return static_cast<const float*>(x)[i];
  return u2f((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
}

// 64-bit key ordering (value, lower index first): NaN above all, +0 equal to -0.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t i) {
  uint32_t u = f2u(v + 0.0f);
  u = v != v ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)~i;
}

// m, s, w: the running maximum of y and the sums of e^(y - m) and
// (y - m) e^(y - m); a second set joins the first.
struct Stats {
  float m, s, w;
};
__device__ __forceinline__ Stats join(Stats a, Stats b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == m ? 0.0f : a.m - m, db = b.m == m ? 0.0f : b.m - m;
  const float fa = exp2f(da * kLog2e), fb = exp2f(db * kLog2e);
  Stats r;
  r.m = m;
  r.s = a.s * fa + b.s * fb;
  // A side that vanishes adds nothing, however far below it lies (da may overflow).
  r.w = (fa == 0.0f ? 0.0f : (a.w + da * a.s) * fa) + (fb == 0.0f ? 0.0f : (b.w + db * b.s) * fb);
  return r;
}

template <int DT>
__global__ __launch_bounds__(256) void logprobs_simple_kernel(const void* __restrict__ x, int64_t stride, uint32_t V,
                                                              float scale, const int32_t* __restrict__ tokens,
                                                              int32_t M, float* __restrict__ logp,
                                                              float* __restrict__ entropy, float* __restrict__ lse,
                                                              int32_t top_k, float* __restrict__ top_logp,
                                                              int32_t* __restrict__ top_index) {
  __shared__ Stats part[256];
  __shared__ uint64_t best[256];
  const size_t n = blockIdx.x, row = n * (size_t)stride;
  const uint32_t tid = threadIdx.x;
  Stats a = {-INFINITY, 0.0f, 0.0f};
  for (uint32_t i = tid; i < V; i += 256u) {
    const float y = logit<DT>(x, row + i) * scale;
    a = join(a, Stats{y, y == -INFINITY ? 0.0f : 1.0f, 0.0f});
    if (y != y) a.s = y;
  }
  part[tid] = a;
  __syncthreads();
  for (uint32_t d = 128u; d > 0u; d >>= 1) {
    if (tid < d) part[tid] = join(part[tid], part[tid + d]);
    __syncthreads();
  }
  a = part[0];
  if (a.m == INFINITY) a.s = NAN;  // inf - inf
  const float ls = a.s == 0.0f ? -INFINITY : a.m + logf(a.s);
  if (tid == 0u) {
    if (entropy) entropy[n] = a.s == 0.0f ? 0.0f : logf(a.s) - a.w / a.s;
    if (lse) lse[n] = ls;
  }
  for (int32_t j = (int32_t)tid; j < M; j += 256) {
    const int32_t t = tokens[n * (size_t)M + j];
    float r = 0.0f;
    if (t >= 0 && (uint32_t)t < V) {
      const float y = logit<DT>(x, row + (uint32_t)t) * scale;
      r = y == -INFINITY && ls == ls ? -INFINITY : y - ls;
    }
    logp[n * (size_t)M + j] = r;
  }
  uint64_t below = ~0ull;
  for (int32_t k = 0; k < top_k; ++k) {
    uint64_t most = 0ull;
    for (uint32_t i = tid; i < V; i += 256u) {
      const uint64_t key = top_key(logit<DT>(x, row + i), i);
      if (key < below && key > most) most = key;
    }
    __syncthreads();
    best[tid] = most;
    __syncthreads();
    for (uint32_t d = 128u; d > 0u; d >>= 1) {
      if (tid < d && best[tid + d] > best[tid]) best[tid] = best[tid + d];
      __syncthreads();
    }
    below = best[0];
    if (tid == 0u) {
      const uint32_t i = ~(uint32_t)below;
      float r = -INFINITY;
      if (k < (int32_t)V) {
        const float y = logit<DT>(x, row + i) * scale;
        r = y == -INFINITY && ls == ls ? -INFINITY : y - ls;
      }
      top_index[n * (size_t)top_k + k] = k < (int32_t)V ? (int32_t)i : -1;
      top_logp[n * (size_t)top_k + k] = r;
    }
  }
}

template <int DT>
__device__ __forceinline__ void store_value(void* p, size_t i, float v) {
  if (DT == kDtF32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__bf16*>(p)[i] = (__bf16)v;
}

template <int DT>
__global__ __launch_bounds__(256) void logprobs_backward_simple_kernel(
    const void* __restrict__ x, int64_t stride, uint32_t V, float scale, const int32_t* __restrict__ tokens, int32_t M,
    const float* __restrict__ lse, const float* __restrict__ entropy, const float* __restrict__ g_logp,
    const float* __restrict__ g_entropy, void* __restrict__ dx, int64_t dx_stride) {
  const size_t n = blockIdx.x;
  float g = 0.0f;
  for (int32_t j = 0; j < M; ++j) {
    const int32_t t = tokens[n * (size_t)M + j];
    if (t >= 0 && (uint32_t)t < V) g += g_logp[n * (size_t)M + j];
  }
  const float ge = g_entropy ? g_entropy[n] : 0.0f, h = g_entropy ? entropy[n] : 0.0f, ls = lse[n];
  for (uint32_t i = threadIdx.x; i < V; i += 256u) {
    const float y = logit<DT>(x, n * (size_t)stride + i) * scale;
    const float lp = y == -INFINITY && ls == ls ? -INFINITY : y - ls, p = expf(lp);
    float d = p == 0.0f ? 0.0f : -p * (g + ge * (lp + h));
    for (int32_t j = 0; j < M; ++j)
      if (tokens[n * (size_t)M + j] == (int32_t)i) d += g_logp[n * (size_t)M + j];
    store_value<DT>(dx, n * (size_t)dx_stride + i, d * scale);
  }
}

}  // namespace

size_t logprobs_workspace(int64_t, int64_t, int32_t) { return 0; }

hipError_t launch_logprobs(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale,
                           const int32_t* tokens, int32_t M, float* logp, float* entropy, float* lse, int32_t top_k,
                           float* top_logp, int32_t* top_index, void*, hipStream_t stream) {
  if (dtype == kDtF32)
    logprobs_simple_kernel<kDtF32><<<(uint32_t)N, 256, 0, stream>>>(x, stride, (uint32_t)V, scale, tokens, M, logp,
                                                                    entropy, lse, top_k, top_logp, top_index);
  else
    logprobs_simple_kernel<kDtBF16><<<(uint32_t)N, 256, 0, stream>>>(x, stride, (uint32_t)V, scale, tokens, M, logp,
                                                                     entropy, lse, top_k, top_logp, top_index);
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale,
                                    const int32_t* tokens, int32_t M, const float* lse, const float* entropy,
                                    const float* g_logp, const float* g_entropy, void* dx, int64_t dx_stride,
                                    hipStream_t stream) {
  if (dtype == kDtF32)
    logprobs_backward_simple_kernel<kDtF32><<<(uint32_t)N, 256, 0, stream>>>(
        x, stride, (uint32_t)V, scale, tokens, M, lse, entropy, g_logp, g_entropy, dx, dx_stride);
  else
    logprobs_backward_simple_kernel<kDtBF16><<<(uint32_t)N, 256, 0, stream>>>(
        x, stride, (uint32_t)V, scale, tokens, M, lse, entropy, g_logp, g_entropy, dx, dx_stride);
  return hipGetLastError();
}

}  // namespace fp4
