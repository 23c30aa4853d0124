// qk_rope.hip -- norms of queries and keys for each head with the rotary
// positions in the same pass, and the gradient.
//
//   y = x r w,  r = (mean x^2 + eps)^-1/2 over a head's D values;
//   pair i of the first R values turned by pos freq_i.
//
// A lane holds N consecutive values of a head (16 bytes where the halves divide
// into them: whole lines in one load); G lanes make a head (a DPP sum), 64 / G
// heads a wave's step.  Where the halves of a pair lie R / 2 apart, the other
// half comes from another lane.  A wave keeps to one row of q or of k while it
// can; its lanes work out one pair's angle each and share them in LDS, from where
// each takes the factors of its values, w cos and w' sin.
//
// Memory bounds both directions: 16384 rows of 72 heads of 64 BF16 take 59 us (5.1
// TB/s; a plain copy of the queries alone 47-51), 4099 rows of 32 heads of 128 FP32
// with three axes 22 us; the gradient of 8192 rows of 40 heads of 128 BF16 51 us
// (4.9 TB/s) and 5 for the weights' sums.  Both halves of a pair in one lane read
// half lines: 66 us for the first.  Few rows are cut into a wave for each step.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"
#include "workspace.h"

#include <algorithm>
#include <type_traits>

namespace fp4 {
namespace {

constexpr uint32_t kWaves = 4;
// Workgroups of the gradient, each with a partial sum: as many as run at once (BF16
// heads of 128: 94 registers, five a CU; 8192 x 40 of them take 57 us, 58 with 1024).
constexpr uint32_t kMaxGroups = 1280;
// Waves that few rows are cut to (8192 rows of 40 heads of 128 BF16, a wave a row of q
// and one of k: 31 us; cut to 32768: 39; 2048 to 8192 alike).
constexpr uint64_t kWantedWaves = 8192;

struct Tensor {
  const void* p;
  int64_t stride;  // elements between rows
};

// One of q and k.
struct Heads {
  Tensor x, g, out;    // input; gradient of the output; output (written)
  const float* w;
  float* partial;      // gradient: a row of D sums for each workgroup
  uint32_t heads;
  uint32_t steps, parts;  // a row's steps of 64 / G heads, and the waves they are cut to
  uint32_t groups;     // workgroups
};

struct Args {
  Heads t[2];
  const float* freq;
  const int32_t* pos;
  float eps;
  uint32_t rows, D, R, axes;
  uint32_t axis[8];    // two bits a pair
};

template <int DT, int N>
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

// The N values of a chunk.
template <int DT, int N>
__device__ __forceinline__ void unpack(typename Chunk<DT, N>::T w, float (&v)[N]) {
  if constexpr (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = u2f(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      v[2 * i] = u2f(w[i] << 16);
      v[2 * i + 1] = u2f(w[i] & 0xFFFF0000u);
    }
  }
}
template <int DT, int N>
__device__ __forceinline__ typename Chunk<DT, N>::T pack(const float (&v)[N]) {
  typename Chunk<DT, N>::T w;
  if constexpr (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = f2u(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
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
  if (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

// A lane's place in its head.
template <int DT, int N, int G, bool INTERLEAVED>
struct Lane {
  uint32_t e;      // its first value
  uint32_t other;  // byte address (4 lane) of the lane that holds the other halves
  bool live, turns, second;
  __device__ __forceinline__ explicit Lane(const Args& s) {
    const uint32_t l = threadIdx.x & (G - 1u), half = s.R / 2u;
    e = l * N;
    live = e < s.D;
    turns = e < s.R;
    second = !INTERLEAVED && turns && e >= half;
    const uint32_t o = !turns ? l : second ? l - half / N : l + half / N;
    other = ((threadIdx.x & 63u & ~(G - 1u)) + o) * 4u;
  }
  // The other half of every value's pair (0 where there is none: an infinity that
  // is not turned stays one).
  __device__ __forceinline__ typename Chunk<DT, N>::T others(typename Chunk<DT, N>::T w) const {
#pragma unroll
    for (uint32_t i = 0; i < sizeof(w) / 4u; ++i) {
      if (!INTERLEAVED) w[i] = (uint32_t)__builtin_amdgcn_ds_bpermute((int)other, (int)w[i]);
      w[i] = turns ? w[i] : 0u;
    }
    return w;
  }
  // v's other halves among what others() gave of its chunk.
  static __device__ __forceinline__ float half_of(const float (&o)[N], int i) { return o[INTERLEAVED ? i ^ 1 : i]; }
};

// A wave's cosines and sines, one row's at a time.
struct alignas(16) Turns {
  float c[128], s[128];
};
// What a lane needs of its pairs, lane and lane + 64, for any row.
struct Angles {
  float freq[2];
  uint32_t axis[2];
  __device__ __forceinline__ explicit Angles(const Args& s) {
#pragma unroll
    for (uint32_t h = 0; h < 2u; ++h) {
      const uint32_t i = (threadIdx.x & 63u) + 64u * h;
      freq[h] = 2u * i < s.R ? s.freq[i] : 0.0f;
      uint32_t word = 0u;
#pragma unroll
      for (uint32_t k = 0; k < 8u; ++k) word = i >> 4 == k ? s.axis[k] : word;
      axis[h] = (word >> (2u * (i & 15u))) & 3u;
    }
  }
  // Of the row's positions.  The angle in turns, in FP64: its whole part goes
  // before it is rounded (pos freq in FP32 would be off by 2^-24 pos).
  __device__ __forceinline__ void fill(const Args& s, uint32_t row, Turns& to) const {
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    if (s.R == 0u) return;
    int32_t at[4];
#pragma unroll
    for (uint32_t x = 0; x < 4u; ++x) at[x] = x < s.axes ? s.pos[(size_t)x * s.rows + row] : 0;
    __builtin_amdgcn_wave_barrier();  // (the row before has been read)
#pragma unroll
    for (uint32_t h = 0; h < 2u; ++h) {
      if (h == 1u && s.R <= 128u) break;
      const uint32_t x = axis[h];
      const int32_t p = x == 0u ? at[0] : x == 1u ? at[1] : x == 2u ? at[2] : at[3];
      double t = (double)p * (double)freq[h] * kTurn;
      t -= __builtin_rint(t);
      float sn, cs;
      sincospif(2.0f * (float)t, &sn, &cs);
      to.c[(threadIdx.x & 63u) + 64u * h] = cs;
      to.s[(threadIdx.x & 63u) + 64u * h] = sn;
    }
    // The wave's own LDS writes before its reads: in order, once they are issued.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
};
// Factors of a lane's values: turned, value i is v_i c_i + (its other half) n_i.
template <int DT, int N, int G, bool INTERLEAVED>
__device__ __forceinline__ void read_turns(const Lane<DT, N, G, INTERLEAVED>& lane, const Args& s, const Turns& from,
                                           float (&c)[N], float (&n)[N]) {
  const uint32_t pair = INTERLEAVED ? lane.e / 2u : lane.second ? lane.e - s.R / 2u : lane.e;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t at = (pair + (INTERLEAVED ? i / 2 : i)) & 127u;
    const bool minus = INTERLEAVED ? i % 2 == 0 : !lane.second;
    c[i] = lane.turns ? from.c[at] : 1.0f;
    n[i] = !lane.turns ? 0.0f : minus ? -from.s[at] : from.s[at];
  }
}
template <int N>
__device__ __forceinline__ void load_floats(const float* p, uint32_t at, bool live, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = p && live ? p[at + i] : 1.0f;
}

// A wave's share of a row: steps [s0, s1).
struct Unit {
  uint32_t row, s0, s1;
};
__device__ __forceinline__ Unit unit_of(const Heads& t, uint32_t u) {
  const uint32_t row = u / t.parts, part = u - row * t.parts;
  return Unit{row, part * t.steps / t.parts, (part + 1u) * t.steps / t.parts};
}
// Whether this workgroup has q or k, and its number among those (q's come first).
__device__ __forceinline__ uint32_t which(const Args& s, uint32_t& group) {
  const uint32_t t = blockIdx.x >= s.t[0].groups ? 1u : 0u;
  group = blockIdx.x - (t ? s.t[0].groups : 0u);
  return t;
}

template <int DT>
__device__ __forceinline__ const uint8_t* head_at(const Tensor& x, uint32_t row, uint32_t value) {
  return static_cast<const uint8_t*>(x.p) + ((size_t)row * (size_t)x.stride + value) * (DT == kDtF32 ? 4u : 2u);
}
template <int DT, int N>
__device__ __forceinline__ typename Chunk<DT, N>::T load(const uint8_t* p) {
  return *reinterpret_cast<const typename Chunk<DT, N>::T*>(p);
}
// (Streamed: 16384 x 72 heads of 64 BF16 take 64 us with plain stores, 59 us so.)
template <int DT, int N>
__device__ __forceinline__ void store(const uint8_t* p, const float (&v)[N]) {
  __builtin_nontemporal_store(pack<DT, N>(v), reinterpret_cast<typename Chunk<DT, N>::T*>(const_cast<uint8_t*>(p)));
}

template <int DT, int N, int G, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) void forward_kernel(Args s) {
  constexpr uint32_t kHeads = 64u / G;
  __shared__ Turns turns[kWaves];
  uint32_t group;
  const Heads t = s.t[which(s, group)];
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t u = group * kWaves + wave;
  if (u >= s.rows * t.parts) return;
  const Unit unit = unit_of(t, u);
  const Lane<DT, N, G, INTERLEAVED> lane(s);
  const uint32_t own = (threadIdx.x & 63u) / G;
  const auto fetch = [&](uint32_t step) __attribute__((always_inline)) {
    typename Chunk<DT, N>::T raw{};
    const uint32_t head = step * kHeads + own;
    if (lane.live && head < t.heads) raw = load<DT, N>(head_at<DT>(t.x, unit.row, head * s.D + lane.e));
    return raw;
  };
  typename Chunk<DT, N>::T next = fetch(unit.s0);  // on its way while the angles are worked out
  float c[N], n[N];
  {
    float w[N], o[N];
    load_floats(t.w, lane.e, lane.live, w);
    Angles(s).fill(s, unit.row, turns[wave]);
    read_turns(lane, s, turns[wave], c, n);
#pragma unroll
    for (int i = 0; i < N; ++i)
      o[i] = INTERLEAVED ? w[i] : u2f((uint32_t)__builtin_amdgcn_ds_bpermute((int)lane.other, (int)f2u(w[i])));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      c[i] *= w[i];
      n[i] *= lane.half_of(o, i);
    }
  }
  const float inv_d = 1.0f / (float)s.D;
  for (uint32_t step = unit.s0; step < unit.s1; ++step) {
    const typename Chunk<DT, N>::T raw = next;
    if (step + 1u < unit.s1) next = fetch(step + 1u);
    float v[N], o[N];
    unpack<DT, N>(raw, v);
    unpack<DT, N>(lane.others(raw), o);
    float r = 1.0f;
    if (t.w) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) sum = __builtin_fmaf(v[i], v[i], sum);
      r = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<G>(sum), inv_d, s.eps));
    }
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = r * __builtin_fmaf(v[i], c[i], lane.half_of(o, i) * n[i]);
    const uint32_t head = step * kHeads + own;
    if (lane.live && head < t.heads) store<DT, N>(head_at<DT>(t.out, unit.row, head * s.D + lane.e), y);
  }
}

// g' = the output's gradient turned back; dx = r (w g' - x r^2 mean(x w g'));
// dw = sum of g' x r: in registers over a wave's rows and heads, then over the
// workgroup, then (sum_kernel) over the workgroups, all in a fixed order.
template <int DT, int N, int G, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) void backward_kernel(Args s) {
  constexpr uint32_t kHeads = 64u / G;
  __shared__ union {
    Turns turns[kWaves];
    float part[kWaves][256];
  } sh;
  uint32_t group;
  const Heads t = s.t[which(s, group)];
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Lane<DT, N, G, INTERLEAVED> lane(s);
  const Angles angles(s);
  const uint32_t own = (threadIdx.x & 63u) / G;
  float c[N], n[N], w[N], dw[N] = {};
  load_floats(t.w, lane.e, lane.live, w);
  const float inv_d = 1.0f / (float)s.D;
  for (uint32_t u = group * kWaves + wave; u < s.rows * t.parts; u += t.groups * kWaves) {
    const Unit unit = unit_of(t, u);
    typename Chunk<DT, N>::T next_g{}, next_x{};
    const auto fetch = [&](uint32_t step) __attribute__((always_inline)) {
      const uint32_t head = step * kHeads + own;
      if (lane.live && head < t.heads) {
        next_g = load<DT, N>(head_at<DT>(t.g, unit.row, head * s.D + lane.e));
        if (t.w) next_x = load<DT, N>(head_at<DT>(t.x, unit.row, head * s.D + lane.e));
      }
    };
    fetch(unit.s0);  // on its way while the angles are worked out
    angles.fill(s, unit.row, sh.turns[wave]);
    read_turns(lane, s, sh.turns[wave], c, n);
    for (uint32_t step = unit.s0; step < unit.s1; ++step) {
      const uint32_t head = step * kHeads + own;
      const bool live = lane.live && head < t.heads;
      const typename Chunk<DT, N>::T raw_g = next_g, raw_x = next_x;
      if (step + 1u < unit.s1) fetch(step + 1u);
      float g[N], o[N], d[N];
      unpack<DT, N>(raw_g, g);
      unpack<DT, N>(lane.others(raw_g), o);
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = __builtin_fmaf(g[i], c[i], -(lane.half_of(o, i) * n[i]));
      if (t.w) {
        float x[N], sum = 0.0f, dot = 0.0f;
        unpack<DT, N>(raw_x, x);
#pragma unroll
        for (int i = 0; i < N; ++i) sum = __builtin_fmaf(x[i], x[i], sum);
        sum = head_sum<G>(sum);
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, inv_d, s.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) {
          x[i] *= r;
          const float p = d[i] * x[i];
          dw[i] += live ? p : 0.0f;
          d[i] *= w[i];
          dot = __builtin_fmaf(p, w[i], dot);
        }
        dot = head_sum<G>(dot) * inv_d;
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = r * __builtin_fmaf(-x[i], dot, d[i]);
      }
      if (live) store<DT, N>(head_at<DT>(t.out, unit.row, head * s.D + lane.e), d);
    }
  }
  if (!t.w) return;
  __syncthreads();  // (the turns have been read)
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int k = G; k < 64; k <<= 1) dw[i] += __shfl_xor(dw[i], k);
    if ((threadIdx.x & 63u) < G && lane.live) sh.part[wave][lane.e + i] = dw[i];
  }
  __syncthreads();
  const uint32_t e = threadIdx.x;
  if (e < s.D)
    t.partial[(size_t)group * s.D + e] = (sh.part[0][e] + sh.part[1][e]) + (sh.part[2][e] + sh.part[3][e]);
}

// Sums of the workgroups' partial sums: 16 columns a workgroup, 64 threads
// each.
__global__ __launch_bounds__(1024) void sum_kernel(const float* __restrict__ partial_q,
                                                  const float* __restrict__ partial_k, uint32_t groups_q,
                                                  uint32_t groups_k, uint32_t D, float* __restrict__ dwq,
                                                  float* __restrict__ dwk) {
  __shared__ float part[64][17];
  const uint32_t columns = (D + 15u) / 16u;
  const bool is_q = blockIdx.x < columns;
  const float* partial = is_q ? partial_q : partial_k;
  float* out = is_q ? dwq : dwk;
  if (!out) return;
  const uint32_t groups = is_q ? groups_q : groups_k;
  const uint32_t c = threadIdx.x & 15u, seg = threadIdx.x >> 4, e = (is_q ? blockIdx.x : blockIdx.x - columns) * 16u + c;
  float sum = 0.0f;
  if (e < D) {
    uint32_t g = seg;
    for (; g + 448u < groups; g += 512u) {  // eight loads at a time
      float v[8];
#pragma unroll
      for (uint32_t i = 0; i < 8u; ++i) v[i] = partial[(size_t)(g + 64u * i) * D + e];
#pragma unroll
      for (uint32_t i = 0; i < 8u; ++i) sum += v[i];
    }
    for (; g < groups; g += 64u) sum += partial[(size_t)g * D + e];
  }
  part[seg][c] = sum;
  __syncthreads();
  if (seg != 0u || e >= D) return;
#pragma unroll
  for (uint32_t i = 1; i < 64u; ++i) sum += part[i][c];
  out[e] = sum;
}

uint32_t group_lanes(uint32_t D, uint32_t N) {
  uint32_t g = 4u;
  while (g * N < D) g *= 2u;
  return g;
}

// Values of a lane: 16 bytes, if the halves divide into them (8 bytes: 60 us instead of
// 57 for 16384 rows of 72 heads of 64, alike for heads of 128).
int lane_values(const QkRope& a) { return a.dtype == kDtBF16 && (a.interleaved || a.R % 16 == 0) ? 8 : 4; }

template <bool BACKWARD, int DT, int N, int G, bool INTERLEAVED>
hipError_t launch_one(Args& s, const QkRope& a, hipStream_t stream) {
  uint32_t grid = 0u;
  const uint32_t all = s.t[0].heads + s.t[1].heads;
  for (Heads& t : s.t) {
    if (t.heads == 0u || s.rows == 0u) continue;
    t.steps = (t.heads + 64u / G - 1u) / (64u / G);
    // Enough waves to fill the chip; beyond that a wave keeps a whole row.
    t.parts = (uint32_t)std::min<uint64_t>(t.steps, (kWantedWaves + s.rows - 1u) / s.rows);
    t.groups = (uint32_t)(((uint64_t)s.rows * t.parts + kWaves - 1u) / kWaves);
    // (The gradient's keep their sums over many rows.)
    if (BACKWARD) t.groups = std::min(t.groups, std::max(kMaxGroups * t.heads / all, 1u));
    grid += t.groups;
  }
  if (s.t[0].partial) s.t[1].partial = s.t[0].partial + (size_t)s.t[0].groups * s.D;
  if (grid > 0u) {
    if (BACKWARD)
      backward_kernel<DT, N, G, INTERLEAVED><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(s);
    else
      forward_kernel<DT, N, G, INTERLEAVED><<<dim3(grid), dim3(64 * kWaves), 0, stream>>>(s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!BACKWARD || !(s.t[0].w || s.t[1].w)) return hipSuccess;
  // (Without rows the weights' gradients are 0.)
  sum_kernel<<<dim3(2u * ((s.D + 15u) / 16u)), dim3(1024), 0, stream>>>(s.t[0].partial, s.t[1].partial, s.t[0].groups,
                                                                      s.t[1].groups, s.D, a.dwq, a.dwk);
  return hipGetLastError();
}

template <bool BACKWARD, int DT, int N, bool INTERLEAVED>
hipError_t launch_lanes(Args& s, const QkRope& a, hipStream_t stream) {
  const uint32_t g = group_lanes(s.D, N);  // (heads of 32 to 256 values)
  if constexpr (N == 8)
    if (g == 4u) return launch_one<BACKWARD, DT, N, 4, INTERLEAVED>(s, a, stream);
  if (g == 8u) return launch_one<BACKWARD, DT, N, 8, INTERLEAVED>(s, a, stream);
  if (g == 16u) return launch_one<BACKWARD, DT, N, 16, INTERLEAVED>(s, a, stream);
  if (g == 32u) return launch_one<BACKWARD, DT, N, 32, INTERLEAVED>(s, a, stream);
  if constexpr (N == 4) return launch_one<BACKWARD, DT, N, 64, INTERLEAVED>(s, a, stream);
  return hipErrorInvalidValue;
}

template <bool BACKWARD>
hipError_t launch(const QkRope& a, hipStream_t stream) {
  Args s{};
  float* partial = a.workspace ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kControlBytes) : nullptr;
  s.t[0] = Heads{{a.q, a.q_stride}, {a.gq, a.gq_stride}, {a.oq, a.oq_stride}, a.wq,
                 partial, (uint32_t)a.hq, 0u, 0u, 0u};
  s.t[1] = Heads{{a.k, a.k_stride}, {a.gk, a.gk_stride}, {a.ok, a.ok_stride}, a.wk, nullptr, (uint32_t)a.hk, 0u, 0u, 0u};
  s.freq = a.freq;
  s.pos = a.pos;
  s.eps = a.eps;
  s.rows = (uint32_t)a.rows;
  s.D = (uint32_t)a.D;
  s.R = (uint32_t)a.R;
  s.axes = (uint32_t)a.axes;
  for (uint32_t i = 0; i < 8u; ++i) s.axis[i] = a.axis[i];
  const auto go = [&](auto interleaved) {
    constexpr bool I = decltype(interleaved)::value;
    if (a.dtype == kDtF32) return launch_lanes<BACKWARD, kDtF32, 4, I>(s, a, stream);
    if (lane_values(a) == 8) return launch_lanes<BACKWARD, kDtBF16, 8, I>(s, a, stream);
    return launch_lanes<BACKWARD, kDtBF16, 4, I>(s, a, stream);
  };
  return a.interleaved ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace

// Room for a sum of each workgroup, behind the control words: they are no more than heads
// of all rows, nor than kMaxGroups and one (of q or of k, where that would have none).
size_t qk_rope_workspace(int64_t rows, int64_t heads, int64_t D) {
  constexpr size_t kRoom = 2048, kLeast = 32 * 4;  // sums, and bytes of one (D is 32 at least)
  static_assert((kRoom - (kMaxGroups + 1u)) * kLeast >= kControlBytes);
  const size_t all = (size_t)(rows * heads), sum = (size_t)D * 4u;
  return all == 0u ? 0u : std::min(kControlBytes + all * 2u * sum, kRoom * sum);
}
hipError_t launch_qk_rope(const QkRope& a, hipStream_t stream) { return launch<false>(a, stream); }
hipError_t launch_qk_rope_backward(const QkRope& a, hipStream_t stream) { return launch<true>(a, stream); }

}  // namespace fp4
