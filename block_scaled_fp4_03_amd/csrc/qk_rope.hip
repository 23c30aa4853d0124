// qk_rope.hip -- norms of queries and keys for each head with the rotary
// positions in the same pass, and the gradient.
//
//   y = x r w,  r = (mean x^2 + eps)^-1/2 over a head's D values;
//   pair i of the first R values turned by pos freq_i.
//
// A lane holds P pairs of a head: with the halves of a pair R / 2 apart, P
// values at two places, so that no pair crosses lanes; G lanes make a head (a
// DPP sum), 64 / G heads a wave's step.  Values that are not rotated lie in
// pairs of their own with cos 1 and sin 0.  A wave keeps to one row while it
// can: the angles are worked out once for all its heads.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"

#include <algorithm>
#include <type_traits>

namespace fp4 {
namespace {

constexpr uint32_t kWaves = 4;
constexpr uint32_t kMaxGroups = 1024;  // workgroups of the gradient, each with a partial sum

struct Tensor {
  const void* p;
  int64_t stride;  // elements between rows
};

struct Args {
  Tensor q, k, gq, gk;       // inputs; gradients of the outputs
  Tensor oq, ok;             // outputs (written)
  const float* wq;
  const float* wk;
  const float* freq;
  const int32_t* pos;
  float* partial;
  float eps;
  uint32_t rows, hq, heads;  // heads: q's and then k's
  uint32_t D, R, axes;
  uint32_t steps, parts;     // a row's steps of 64 / G heads, and the waves they are cut to
  uint32_t axis[8];          // two bits a pair
};

template <int DT, int P>
struct Chunk;
template <>
struct Chunk<kDtF32, 4> {
  typedef u32x4 T;
};
template <>
struct Chunk<kDtBF16, 8> {
  typedef u32x4 T;
};
template <>
struct Chunk<kDtBF16, 4> {
  typedef u32x2 T;
};

// P values of a chunk.
template <int DT, int P>
__device__ __forceinline__ void unpack(typename Chunk<DT, P>::T w, float* v) {
  if constexpr (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = u2f(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      v[2 * i] = u2f(w[i] << 16);
      v[2 * i + 1] = u2f(w[i] & 0xFFFF0000u);
    }
  }
}
template <int DT, int P>
__device__ __forceinline__ typename Chunk<DT, P>::T pack(const float* v) {
  typename Chunk<DT, P>::T w;
  if constexpr (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = f2u(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  }
  return w;
}

// Sum over the G lanes of a head, in each of them and in a fixed order.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
template <int G>
__device__ __forceinline__ float head_sum(float v) {
  if (G >= 2) v += moved<0xB1>(v);   // lane ^ 1
  if (G >= 4) v += moved<0x4E>(v);   // lane ^ 2
  if (G >= 8) v += moved<0x141>(v);  // 7 - lane of 8: the other four
  if (G >= 16) v += moved<0x140>(v); // 15 - lane of 16: the other eight
  if (G >= 32) v += __shfl_xor(v, 16);
  return v;
}

// A lane's place in its head.
template <int P, int G, bool INTERLEAVED>
struct Lane {
  uint32_t l, a, b;  // its two chunks' first values
  bool live, turns;
  uint32_t axis;     // its pairs' axes, two bits each
  __device__ __forceinline__ explicit Lane(const Args& s) {
    l = threadIdx.x & (G - 1u);
    live = l * 2u * P < s.D;
    turns = l * 2u * P < s.R;
    if (INTERLEAVED) {
      a = l * 2u * P;
      b = a + P;
    } else {
      const uint32_t m = turns ? l : l - s.R / (2u * P);
      a = (turns ? 0u : s.R) + m * P;
      b = a + (turns ? s.R : s.D - s.R) / 2u;
    }
    uint32_t word = 0u;
#pragma unroll
    for (uint32_t i = 0; i < 8u; ++i) word = (l * P) >> 4 == i ? s.axis[i] : word;
    axis = word >> (2u * ((l * P) & 15u));
  }
  // Cosines and sines of the lane's pairs at a row's positions.  The angle in
  // turns, in FP64: its whole part goes before it is rounded (pos freq in
  // FP32 would be off by 2^-24 pos).
  __device__ __forceinline__ void angles(const Args& s, uint32_t row, const float (&freq)[P], float (&c)[P],
                                         float (&n)[P]) const {
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    if (s.R == 0u) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        c[i] = 1.0f;
        n[i] = 0.0f;
      }
      return;
    }
    int32_t at[4];
#pragma unroll
    for (uint32_t x = 0; x < 4u; ++x) at[x] = x < s.axes ? s.pos[(size_t)x * s.rows + row] : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t x = (axis >> (2 * i)) & 3u;
      const int32_t p = x == 0u ? at[0] : x == 1u ? at[1] : x == 2u ? at[2] : at[3];
      double t = (double)p * (double)freq[i] * kTurn;
      t -= __builtin_rint(t);
      float sn, cs;
      sincospif(2.0f * (float)t, &sn, &cs);
      c[i] = turns ? cs : 1.0f;
      n[i] = turns ? sn : 0.0f;
    }
  }
  // Index of the first and the second value of pair i among a lane's 2 P.
  static __device__ __forceinline__ constexpr int first(int i) { return INTERLEAVED ? 2 * i : i; }
  static __device__ __forceinline__ constexpr int second(int i) { return INTERLEAVED ? 2 * i + 1 : P + i; }
};

template <int P>
__device__ __forceinline__ void load_floats(const float* p, uint32_t at, bool live, float otherwise, float* v) {
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = p && live ? p[at + i] : otherwise;
}

// A wave's share of a row: steps [s0, s1).
struct Unit {
  uint32_t row, s0, s1;
};
__device__ __forceinline__ Unit unit_of(const Args& s, uint32_t u) {
  const uint32_t row = u / s.parts, part = u - row * s.parts;
  return Unit{row, part * s.steps / s.parts, (part + 1u) * s.steps / s.parts};
}

template <int DT, int P, int G, bool INTERLEAVED>
__device__ __forceinline__ size_t at_head(const Tensor& q, const Tensor& k, const Args& s, uint32_t row, uint32_t head,
                                          const void** base) {
  const bool is_q = head < s.hq;
  *base = is_q ? q.p : k.p;
  return (size_t)row * (size_t)(is_q ? q.stride : k.stride) + (size_t)(is_q ? head : head - s.hq) * s.D;
}

template <int DT, int P>
__device__ __forceinline__ typename Chunk<DT, P>::T load(const void* base, size_t at) {
  constexpr uint32_t kSize = DT == kDtF32 ? 4u : 2u;
  return *reinterpret_cast<const typename Chunk<DT, P>::T*>(static_cast<const uint8_t*>(base) + at * kSize);
}
template <int DT, int P>
__device__ __forceinline__ void store(const void* base, size_t at, const float* v) {
  constexpr uint32_t kSize = DT == kDtF32 ? 4u : 2u;
  *reinterpret_cast<typename Chunk<DT, P>::T*>(const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + at * kSize) =
      pack<DT, P>(v);
}

template <int DT, int P, int G, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) void forward_kernel(Args s) {
  constexpr uint32_t kHeads = 64u / G;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t u = blockIdx.x * kWaves + wave;
  if (u >= s.rows * s.parts) return;
  const Unit unit = unit_of(s, u);
  const Lane<P, G, INTERLEAVED> lane(s);
  float freq[P], c[P], n[P], wq[2 * P], wk[2 * P];
  load_floats<P>(s.freq, lane.l * P, lane.turns, 0.0f, freq);
  load_floats<P>(s.wq, lane.a, lane.live, 1.0f, wq);
  load_floats<P>(s.wq, lane.b, lane.live, 1.0f, wq + P);
  load_floats<P>(s.wk, lane.a, lane.live, 1.0f, wk);
  load_floats<P>(s.wk, lane.b, lane.live, 1.0f, wk + P);
  lane.angles(s, unit.row, freq, c, n);
  const float inv_d = 1.0f / (float)s.D;
  for (uint32_t step = unit.s0; step < unit.s1; ++step) {
    const uint32_t head = step * kHeads + (threadIdx.x & 63u) / G;
    const bool live = lane.live && head < s.heads, is_q = head < s.hq;
    const void* base;
    const size_t at = at_head<DT, P, G, INTERLEAVED>(s.q, s.k, s, unit.row, head, &base);
    float v[2 * P] = {};
    if (live) {
      unpack<DT, P>(load<DT, P>(base, at + lane.a), v);
      unpack<DT, P>(load<DT, P>(base, at + lane.b), v + P);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) sum = __builtin_fmaf(v[i], v[i], sum);
    sum = head_sum<G>(sum);
    const bool norm = (is_q ? s.wq : s.wk) != nullptr;
    const float r = norm ? __builtin_amdgcn_rsqf(__builtin_fmaf(sum, inv_d, s.eps)) : 1.0f;
    float y[2 * P];
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) v[i] = v[i] * r * (is_q ? wq[i] : wk[i]);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int a = lane.first(i), b = lane.second(i);
      y[a] = __builtin_fmaf(v[a], c[i], -(v[b] * n[i]));
      y[b] = __builtin_fmaf(v[b], c[i], v[a] * n[i]);
    }
    if (live) {
      const size_t to = at_head<DT, P, G, INTERLEAVED>(s.oq, s.ok, s, unit.row, head, &base);
      store<DT, P>(base, to + lane.a, y);
      store<DT, P>(base, to + lane.b, y + P);
    }
  }
}

// g' = the output's gradient turned back; dx = r (w g' - x r^2 mean(x w g'));
// dw = sum of g' x r: in registers over a wave's rows and heads, then over the
// workgroup, then (sum_kernel) over the workgroups, all in a fixed order.
template <int DT, int P, int G, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) void backward_kernel(Args s) {
  constexpr uint32_t kHeads = 64u / G;
  __shared__ float part[kWaves][2][256];
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Lane<P, G, INTERLEAVED> lane(s);
  float freq[P], c[P], n[P], wq[2 * P], wk[2 * P], dq[2 * P] = {}, dk[2 * P] = {};
  load_floats<P>(s.freq, lane.l * P, lane.turns, 0.0f, freq);
  load_floats<P>(s.wq, lane.a, lane.live, 1.0f, wq);
  load_floats<P>(s.wq, lane.b, lane.live, 1.0f, wq + P);
  load_floats<P>(s.wk, lane.a, lane.live, 1.0f, wk);
  load_floats<P>(s.wk, lane.b, lane.live, 1.0f, wk + P);
  const float inv_d = 1.0f / (float)s.D;
  for (uint32_t u = blockIdx.x * kWaves + wave; u < s.rows * s.parts; u += gridDim.x * kWaves) {
    const Unit unit = unit_of(s, u);
    lane.angles(s, unit.row, freq, c, n);
    for (uint32_t step = unit.s0; step < unit.s1; ++step) {
      const uint32_t head = step * kHeads + (threadIdx.x & 63u) / G;
      const bool live = lane.live && head < s.heads, is_q = head < s.hq;
      const bool norm = (is_q ? s.wq : s.wk) != nullptr;
      const void* base;
      float g[2 * P] = {}, x[2 * P] = {}, t[2 * P];
      if (live) {
        const size_t at = at_head<DT, P, G, INTERLEAVED>(s.gq, s.gk, s, unit.row, head, &base);
        unpack<DT, P>(load<DT, P>(base, at + lane.a), g);
        unpack<DT, P>(load<DT, P>(base, at + lane.b), g + P);
      }
      if (live && norm) {
        const size_t at = at_head<DT, P, G, INTERLEAVED>(s.q, s.k, s, unit.row, head, &base);
        unpack<DT, P>(load<DT, P>(base, at + lane.a), x);
        unpack<DT, P>(load<DT, P>(base, at + lane.b), x + P);
      }
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * P; ++i) sum = __builtin_fmaf(x[i], x[i], sum);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int a = lane.first(i), b = lane.second(i);
        t[a] = __builtin_fmaf(g[a], c[i], g[b] * n[i]);
        t[b] = __builtin_fmaf(g[b], c[i], -(g[a] * n[i]));
      }
      sum = head_sum<G>(sum);
      const float r = norm ? __builtin_amdgcn_rsqf(__builtin_fmaf(sum, inv_d, s.eps)) : 1.0f;
#pragma unroll
      for (int i = 0; i < 2 * P; ++i) {
        x[i] *= r;
        const float d = t[i] * x[i];
        if (live && is_q) dq[i] += d;
        if (live && !is_q) dk[i] += d;
        t[i] *= is_q ? wq[i] : wk[i];
        dot = __builtin_fmaf(x[i], t[i], dot);
      }
      dot = head_sum<G>(dot) * inv_d;
#pragma unroll
      for (int i = 0; i < 2 * P; ++i) t[i] = norm ? r * __builtin_fmaf(-x[i], dot, t[i]) : t[i];
      if (live) {
        const size_t to = at_head<DT, P, G, INTERLEAVED>(s.oq, s.ok, s, unit.row, head, &base);
        store<DT, P>(base, to + lane.a, t);
        store<DT, P>(base, to + lane.b, t + P);
      }
    }
  }
  if (!s.partial) return;
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) {
#pragma unroll
    for (int d = G; d < 64; d <<= 1) {
      dq[i] += __shfl_xor(dq[i], d);
      dk[i] += __shfl_xor(dk[i], d);
    }
    if ((threadIdx.x & 63u) < G && lane.live) {
      const uint32_t e = (i < P ? lane.a : lane.b - P) + i;
      part[wave][0][e] = dq[i];
      part[wave][1][e] = dk[i];
    }
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < 2u * s.D; e += 64u * kWaves) {
    const uint32_t w = e >= s.D, at = e - w * s.D;
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kWaves; ++i) sum += part[i][w][at];
    s.partial[(size_t)blockIdx.x * 2u * s.D + e] = sum;
  }
}

// Sums of the workgroups' partial sums: 16 columns a workgroup, 16 threads each.
__global__ __launch_bounds__(256) void sum_kernel(const float* __restrict__ partial, uint32_t groups, uint32_t D,
                                                  float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float part[16][16];
  const uint32_t c = threadIdx.x & 15u, seg = threadIdx.x >> 4, e = blockIdx.x * 16u + c;
  float sum = 0.0f;
  if (e < 2u * D)
    for (uint32_t g = seg; g < groups; g += 16u) sum += partial[(size_t)g * 2u * D + e];
  part[seg][c] = sum;
  __syncthreads();
  if (seg != 0u || e >= 2u * D) return;
  for (uint32_t i = 1; i < 16u; ++i) sum += part[i][c];
  float* out = e < D ? dwq : dwk;
  if (out) out[e < D ? e : e - D] = sum;
}

uint32_t group_lanes(uint32_t D, uint32_t P) {
  uint32_t g = 2u;
  while (g * 2u * P < D) g *= 2u;
  return g;
}

// Pairs of a lane: 16-byte chunks, if the halves divide into them.
int lane_pairs(const QkRope& a) {
  return a.dtype == kDtBF16 && a.R % 16 == 0 && a.D % 16 == 0 ? 8 : 4;
}

template <bool BACKWARD, int DT, int P, int G, bool INTERLEAVED>
hipError_t launch_one(Args& s, const QkRope& a, hipStream_t stream) {
  s.steps = (s.heads + 64u / G - 1u) / (64u / G);
  // Enough waves to fill the chip; beyond that a wave keeps a whole row.
  const uint64_t wanted = 8192u;
  s.parts = (uint32_t)std::min<uint64_t>(s.steps, (wanted + s.rows - 1u) / std::max(s.rows, 1u));
  const uint64_t units = (uint64_t)s.rows * s.parts;
  uint32_t grid = (uint32_t)((units + kWaves - 1u) / kWaves);
  if (BACKWARD) grid = std::min(grid, kMaxGroups);
  if (grid > 0u) {  // (no rows: the weights' gradients are 0)
    if (BACKWARD)
      backward_kernel<DT, P, G, INTERLEAVED><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(s);
    else
      forward_kernel<DT, P, G, INTERLEAVED><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!BACKWARD || !(s.wq || s.wk)) return hipSuccess;
  sum_kernel<<<dim3((2u * s.D + 15u) / 16u), dim3(256), 0, stream>>>(s.partial, grid, s.D, a.dwq, a.dwk);
  return hipGetLastError();
}

template <bool BACKWARD, int DT, int P, bool INTERLEAVED>
hipError_t launch_lanes(Args& s, const QkRope& a, hipStream_t stream) {
  const uint32_t g = group_lanes(s.D, P);
  if constexpr (P == 8)
    if (g == 2u) return launch_one<BACKWARD, DT, P, 2, INTERLEAVED>(s, a, stream);
  if (g == 4u) return launch_one<BACKWARD, DT, P, 4, INTERLEAVED>(s, a, stream);
  if (g == 8u) return launch_one<BACKWARD, DT, P, 8, INTERLEAVED>(s, a, stream);
  if (g == 16u) return launch_one<BACKWARD, DT, P, 16, INTERLEAVED>(s, a, stream);  // (heads of 32 to 256 values)
  if constexpr (P == 4) return launch_one<BACKWARD, DT, P, 32, INTERLEAVED>(s, a, stream);
  return hipErrorInvalidValue;
}

template <bool BACKWARD>
hipError_t launch(const QkRope& a, hipStream_t stream) {
  Args s{};
  s.q = Tensor{a.q, a.q_stride};
  s.k = Tensor{a.k, a.k_stride};
  s.gq = Tensor{a.gq, a.gq_stride};
  s.gk = Tensor{a.gk, a.gk_stride};
  s.oq = Tensor{a.oq, a.oq_stride};
  s.ok = Tensor{a.ok, a.ok_stride};
  s.wq = a.wq;
  s.wk = a.wk;
  s.freq = a.freq;
  s.pos = a.pos;
  s.partial = BACKWARD && (a.wq || a.wk) ? static_cast<float*>(a.workspace) : nullptr;
  s.eps = a.eps;
  s.rows = (uint32_t)a.rows;
  s.hq = (uint32_t)a.hq;
  s.heads = (uint32_t)(a.hq + a.hk);
  s.D = (uint32_t)a.D;
  s.R = (uint32_t)a.R;
  s.axes = (uint32_t)a.axes;
  for (uint32_t i = 0; i < 8u; ++i) s.axis[i] = a.axis[i];
  const auto go = [&](auto interleaved) {
    constexpr bool I = decltype(interleaved)::value;
    if (a.dtype == kDtF32) return launch_lanes<BACKWARD, kDtF32, 4, I>(s, a, stream);
    if (lane_pairs(a) == 8) return launch_lanes<BACKWARD, kDtBF16, 8, I>(s, a, stream);
    return launch_lanes<BACKWARD, kDtBF16, 4, I>(s, a, stream);
  };
  return a.interleaved ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace

size_t qk_rope_workspace(int64_t rows, int64_t heads, int64_t D) {
  return (size_t)std::min<int64_t>(rows * heads, kMaxGroups) * 2u * (size_t)D * 4u;
}
hipError_t launch_qk_rope(const QkRope& a, hipStream_t stream) { return launch<false>(a, stream); }
hipError_t launch_qk_rope_backward(const QkRope& a, hipStream_t stream) { return launch<true>(a, stream); }

}  // namespace fp4
