// moe.hip -- around the grouped expert GEMM: the router's choice of experts,
// the tokens' order by expert, rows taken there and joined back, and the
// gradients.
//
// Route.  The k largest logits of a token (ties to the lower expert) and their
// softmax.  16 lanes hold a token (one DPP row), expert e in lane e % 16: the
// largest of a lane's keys, then of the 16, k times.  A BF16 key and its expert
// fit one word; of an FP32 key the expert is found after the largest.  16384
// tokens, 8 of 128 experts, BF16: 5.9 us, of it 58% vector ALU issue (7.8 with
// 64-bit keys); 16 tokens 2 us.
//
// Sort.  A stable counting sort.  A wave ranks 64 entries at a time among
// equal ids by one ballot for each bit of the id, and adds their number to its
// own counters in LDS; the waves' counters, and the workgroups' where there
// are several, are then summed over the entries before.  64 entries 3.5 us;
// 131072 entries of 128 experts 3.1 us to count and 7.5 to place: launches and
// dependent memory latencies (16 us with chunks of 8192, on 16 CUs).
//
// Gather, combine and the gradient move rows of 16-byte vectors; a wave takes
// 64 of them of one token (in the gradient every second or all 64 of a token's).
// Rows in expert order are streamed past the caches: 16384 tokens of 2880 BF16,
// four experts each, take 78 us there (86 us without) and 78 us back (88 us), 6.0
// TB/s, and the gradient 154 us, 5.5 TB/s (169 us with plain stores, 164 loads).
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"
#include "workspace.h"

#include <algorithm>
#include <type_traits>

namespace fp4 {
namespace {

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// ---- router ----------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float element(const void* x, size_t i) {
  if (DT == kDtF32) return static_cast<const float*>(x)[i];
  return u2f((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
}

// Keys in the order of the values, NaN above all, +0 equal to -0; 0 is below
// every value's key.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = f2u(v + 0.0f);
  return v != v ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 0xFFFFFFFFu ? NAN : u2f((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Rotations inside each row of 16 lanes (DPP row_ror): the largest and the least
// word and the sum over the row, in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t ror_word(uint32_t a) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)a, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t row_max(uint32_t a) {
  a = max(a, ror_word<0x121>(a));
  a = max(a, ror_word<0x122>(a));
  a = max(a, ror_word<0x124>(a));
  return max(a, ror_word<0x128>(a));
}
__device__ __forceinline__ uint32_t row_min(uint32_t a) {
  a = min(a, ror_word<0x121>(a));
  a = min(a, ror_word<0x122>(a));
  a = min(a, ror_word<0x124>(a));
  return min(a, ror_word<0x128>(a));
}
template <int CTRL>
__device__ __forceinline__ float ror(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_sum(float v) {
  v += ror<0x121>(v);
  v += ror<0x122>(v);
  v += ror<0x124>(v);
  return v + ror<0x128>(v);
}
__device__ __forceinline__ float row_fmax(float v) {
  v = fmaxf(v, ror<0x121>(v));
  v = fmaxf(v, ror<0x122>(v));
  v = fmaxf(v, ror<0x124>(v));
  return fmaxf(v, ror<0x128>(v));
}

// e^(v - m), 0 for v = -inf whatever m is.
__device__ __forceinline__ float weight_of(float v, float m) { return v == -INFINITY ? 0.0f : expf(v - m); }

// The key of expert e's logit v; of BF16 the upper half (all there is) and, so
// that the lower expert of equals is first, e's complement below.
template <int DT>
__device__ __forceinline__ uint32_t choice_key(float v, uint32_t e) {
  const uint32_t k = order_key(v);
  return DT == kDtF32 ? k : (k & 0xFFFF0000u) | (0xFFFFu - e);
}
template <int DT>
__device__ __forceinline__ float choice_value(uint32_t k) {
  return key_value(DT == kDtF32 ? k : (k & 0x80000000u) ? k & 0xFFFF0000u : k | 0xFFFFu);
}

// N: values a lane holds (16 N >= E).
template <int DT, int N>
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ x, int64_t stride, uint32_t T, uint32_t E,
                                                    uint32_t k, bool renormalise, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const uint32_t lane = threadIdx.x & 15u, t = blockIdx.x * 16u + (threadIdx.x >> 4);
  const uint32_t row = t < T ? t : T - 1u;  // (every lane takes part in the moves)
  uint32_t key[N];  // 0: none, or chosen already
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t e = 16u * i + lane;
    key[i] = e < E ? choice_key<DT>(element<DT>(x, (size_t)row * (size_t)stride + e), e) : 0u;
  }
  float rest = 0.0f, top = 0.0f, value = -INFINITY;
  uint32_t mine = 0u;       // lane j keeps the j-th choice
  for (uint32_t j = 0; j < k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) best = max(best, key[i]);
    best = row_max(best);
    uint32_t e;
    if (DT == kDtF32) {
      e = 0xFFFFFFFFu;
#pragma unroll
      for (int i = N - 1; i >= 0; --i) e = key[i] == best ? 16u * i + lane : e;
      e = row_min(e);
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = 16u * i + lane == e ? 0u : key[i];
    } else {
      e = 0xFFFFu - (best & 0xFFFFu);
    }
    const float v = choice_value<DT>(best);
    if (j == 0u) {
      top = v;
      if (!renormalise) {
        rest = weight_of(DT == kDtF32 && (e & 15u) == lane ? v : -INFINITY, top);  // (gone from key[] already)
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (key[i] != 0u) rest += weight_of(choice_value<DT>(key[i]), top);
      }
    }
    if (lane == j) {
      mine = e;
      value = v;
    }
    if (DT != kDtF32) {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = key[i] == best ? 0u : key[i];
    }
  }
  const float w = weight_of(value, top), sum = row_sum(renormalise ? w : rest);
  if (t < T && lane < k) {
    ids[(size_t)t * k + lane] = (int32_t)mine;
    weights[(size_t)t * k + lane] = sum == 0.0f ? 0.0f : w / sum;
  }
}

// dx = p (full - sum p full), p the softmax over the chosen experts or over
// all, full the gradient of the weights at the chosen experts and 0 elsewhere.
template <int DT, int N>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ x, int64_t stride, uint32_t T,
                                                             uint32_t E, uint32_t k, bool renormalise,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ g, void* __restrict__ dx) {
  const uint32_t lane = threadIdx.x & 15u, t = blockIdx.x * 16u + (threadIdx.x >> 4);
  const uint32_t row = t < T ? t : T - 1u;
  float p[N], full[N];
  uint32_t chosen = 0u;  // bit i: expert 16 i + lane is
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t e = 16u * i + lane;
    p[i] = e < E ? element<DT>(x, (size_t)row * (size_t)stride + e) : -INFINITY;
    full[i] = 0.0f;
  }
  const int32_t my_id = lane < k ? ids[(size_t)row * k + lane] : -1;
  const float my_g = lane < k ? g[(size_t)row * k + lane] : 0.0f;
  for (uint32_t j = 0; j < k; ++j) {
    const int32_t id = __shfl(my_id, (int)j, 16);
    const float gj = __shfl(my_g, (int)j, 16);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool hit = id == (int32_t)(16u * i + lane);
      full[i] += hit ? gj : 0.0f;
      chosen |= hit ? 1u << i : 0u;
    }
  }
  if (renormalise) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!((chosen >> i) & 1u)) p[i] = -INFINITY;
  }
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmaxf(m, p[i]);
    nan |= p[i] != p[i];
  }
  m = row_fmax(m);
  float z = nan ? NAN : 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = weight_of(p[i], m);
    z += p[i];
  }
  z = row_sum(z);
  const float inv = z == 0.0f ? 0.0f : 1.0f / z;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] *= inv;
    s = __builtin_fmaf(p[i], full[i], s);
  }
  s = row_sum(s);
  if (t >= T) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t e = 16u * i + lane;
    if (e >= E) continue;
    const float v = p[i] * (full[i] - s);
    if (DT == kDtF32)
      static_cast<float*>(dx)[(size_t)t * E + e] = v;
    else
      static_cast<__bf16*>(dx)[(size_t)t * E + e] = (__bf16)v;
  }
}

template <template <int, int> class F, typename... A>
hipError_t by_experts(int dtype, uint32_t E, A... a) {
  const uint32_t n = (E + 15u) / 16u;
  const auto go = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (n <= 1u) return F<DT, 1>::go(a...);
    if (n <= 2u) return F<DT, 2>::go(a...);
    if (n <= 4u) return F<DT, 4>::go(a...);
    if (n <= 8u) return F<DT, 8>::go(a...);
    if (n <= 16u) return F<DT, 16>::go(a...);
    return F<DT, 32>::go(a...);
  };
  if (dtype == kDtF32) return go(std::integral_constant<int, kDtF32>{});
  return go(std::integral_constant<int, kDtBF16>{});
}

template <int DT, int N>
struct Route {
  static hipError_t go(const void* x, int64_t stride, uint32_t T, uint32_t E, uint32_t k, bool renormalise,
                       int32_t* ids, float* weights, hipStream_t s) {
    route_kernel<DT, N><<<dim3((T + 15u) / 16u), dim3(256), 0, s>>>(x, stride, T, E, k, renormalise, ids, weights);
    return hipGetLastError();
  }
};
template <int DT, int N>
struct RouteBackward {
  static hipError_t go(const void* x, int64_t stride, uint32_t T, uint32_t E, uint32_t k, bool renormalise,
                       const int32_t* ids, const float* g, void* dx, hipStream_t s) {
    route_backward_kernel<DT, N><<<dim3((T + 15u) / 16u), dim3(256), 0, s>>>(x, stride, T, E, k, renormalise, ids, g,
                                                                              dx);
    return hipGetLastError();
  }
};

// ---- sort ------------------------------------------------------------------
// A chunk of entries is a workgroup's: small ones while their counters can be
// summed where they are needed (256 chunks: 524288 entries of 128 experts 14.7 us, 20
// the other way), large ones beyond, with a launch of its own for the sums (1048576
// entries 22.6 us, 30 the other way).
constexpr uint32_t kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr uint32_t kFewRounds = 2, kManyRounds = 8;              // of 64 entries, a wave
constexpr uint32_t kFewChunks = 256;
static_assert(kFewChunks * kFewRounds >= kManyRounds, "large chunks are two at least");
constexpr uint32_t kAhead = 16;                                  // counts of chunks asked for together
constexpr uint32_t kMaxBins = 512 + 2;                           // experts, unrouted, past the end

// Bin of entry i: its expert, E for an id that is none, E + 1 past the end.
__device__ __forceinline__ uint32_t bin_of(const int32_t* ids, uint32_t i, uint32_t N, uint32_t E) {
  if (i >= N) return E + 1u;
  const uint32_t id = (uint32_t)ids[i];
  return id < E ? id : E;
}

// How many entries of each bin every chunk has: counts[chunk][E + 1].
template <uint32_t ROUNDS>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids, uint32_t N,
                                                                  uint32_t E, uint32_t* __restrict__ counts) {
  __shared__ uint32_t count[kMaxBins];
  const uint32_t base = blockIdx.x * (kSortThreads * ROUNDS) + threadIdx.x;
  uint32_t bin[ROUNDS];
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) bin[r] = bin_of(ids, base + r * kSortThreads, N, E);
  for (uint32_t e = threadIdx.x; e < E + 2u; e += kSortThreads) count[e] = 0u;
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) atomicAdd(&count[bin[r]], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E + 1u; e += kSortThreads) counts[(size_t)blockIdx.x * (E + 1u) + e] = count[e];
}

// counts[chunk][bin] to the sums over the chunks before, and row `chunks` to the
// sums over all: 16 bins a workgroup, 64 runs of chunks each.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(uint32_t* __restrict__ counts, uint32_t chunks,
                                                                 uint32_t bins) {
  __shared__ uint32_t run_sum[64][16];
  const uint32_t e = blockIdx.x * 16u + (threadIdx.x & 15u), run = threadIdx.x >> 4, len = (chunks + 63u) / 64u;
  const uint32_t b0 = min(run * len, chunks), b1 = e < bins ? min(b0 + len, chunks) : b0;
  uint32_t sum = 0u;
  for (uint32_t b = b0; b < b1; ++b) sum += counts[(size_t)b * bins + e];
  run_sum[run][threadIdx.x & 15u] = sum;
  __syncthreads();
  uint32_t before = 0u;
  for (uint32_t i = 0; i < run; ++i) before += run_sum[i][threadIdx.x & 15u];
  for (uint32_t b = b0; b < b1; ++b) {
    const uint32_t c = counts[(size_t)b * bins + e];
    counts[(size_t)b * bins + e] = before;
    before += c;
  }
  if (run == 63u && e < bins) counts[(size_t)chunks * bins + e] = before;
}

// Places of a chunk's entries.  counts: sort_count_kernel's (kFewRounds),
// sort_scan_kernel's (kManyRounds), or NULL where there is one chunk.  Dynamic
// LDS: kSortWaves x (E + 2) counters.
template <uint32_t ROUNDS>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids, uint32_t N,
                                                                  uint32_t k, uint32_t E, uint32_t bits,
                                                                  const uint32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ group_off,
                                                                  int32_t* __restrict__ row_idx,
                                                                  int32_t* __restrict__ pos) {
  extern __shared__ uint32_t wave_count[];
  __shared__ uint32_t start[kMaxBins], wave_sum[kSortWaves], part[2][kSortThreads];
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, bins = E + 2u;
  const uint32_t base = blockIdx.x * (kSortThreads * ROUNDS) + wave * 64u * ROUNDS + lane;
  uint32_t bin[ROUNDS], rank[ROUNDS];
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) bin[r] = bin_of(ids, base + 64u * r, N, E);
  for (uint32_t i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) wave_count[i] = 0u;
  // Few chunks: a bin's counts of every `runs`-th chunk, all and those before this one.
  const uint32_t runs = kSortThreads / (E + 1u), run = threadIdx.x / (E + 1u);
  if (ROUNDS == kFewRounds && counts != nullptr && run < runs) {
    const uint32_t at = threadIdx.x - run * (E + 1u);
    uint32_t all = 0u, before = 0u;
    for (uint32_t b0 = run; b0 < gridDim.x; b0 += kAhead * runs) {
      uint32_t c[kAhead];
#pragma unroll
      for (uint32_t i = 0; i < kAhead; ++i) c[i] = counts[(size_t)min(b0 + i * runs, gridDim.x - 1u) * (E + 1u) + at];
#pragma unroll
      for (uint32_t i = 0; i < kAhead; ++i) {
        all += b0 + i * runs < gridDim.x ? c[i] : 0u;
        before += b0 + i * runs < blockIdx.x ? c[i] : 0u;
      }
    }
    part[0][threadIdx.x] = all;
    part[1][threadIdx.x] = before;
  }
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) {
    uint64_t same = ~0ull;  // lanes with this lane's bin
    for (uint32_t b = 0; b < bits; ++b) {
      const bool set = (bin[r] >> b) & 1u;
      const uint64_t all = __ballot(set);
      same &= set ? all : ~all;
    }
    const uint32_t first = (uint32_t)__builtin_ctzll(same);
    uint32_t before = 0u;
    if (lane == first) before = atomicAdd(&wave_count[wave * bins + bin[r]], (uint32_t)__popcll(same));
    rank[r] = (uint32_t)__shfl((int)before, (int)first) + (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
  }
  __syncthreads();
  // Of every bin (one thread each): the waves' counts before each wave, the
  // chunks' before this one, and all of them.
  const uint32_t e = threadIdx.x;
  uint32_t total = 0u, mine = 0u;
  if (e <= E) {
    uint32_t c[kSortWaves];
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) c[w] = wave_count[w * bins + e];
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; ++w) {
      wave_count[w * bins + e] = total;
      total += c[w];
    }
    if (counts != nullptr) {
      total = 0u;
      if (ROUNDS == kFewRounds) {
        for (uint32_t i = 0; i < runs; ++i) {
          total += part[0][i * (E + 1u) + e];
          mine += part[1][i * (E + 1u) + e];
        }
      } else {
        total = counts[(size_t)gridDim.x * (E + 1u) + e];
        mine = counts[(size_t)blockIdx.x * (E + 1u) + e];
      }
    }
  }
  // Exclusive sums over the bins.
  uint32_t sum = total;
#pragma unroll
  for (uint32_t d = 1; d < 64u; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 63u) wave_sum[wave] = sum;
  __syncthreads();
  uint32_t at = sum - total;
  for (uint32_t w = 0; w < wave; ++w) at += wave_sum[w];
  if (e <= E) start[e] = at + mine;
  if (blockIdx.x == 0u && e <= E) group_off[e] = (int32_t)(e < E ? at : N);
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < ROUNDS; ++r) {
    const uint32_t i = base + 64u * r, b = bin[r];
    if (i >= N) continue;
    const uint32_t p = start[b] + wave_count[wave * bins + b] + rank[r];
    pos[i] = b < E ? (int32_t)p : (int32_t)~p;
    row_idx[p] = (int32_t)(i / k);
  }
}

// ---- rows ------------------------------------------------------------------
// The row an entry of pos names, routed or not.
__device__ __forceinline__ uint32_t row_of(int32_t p) { return (uint32_t)(p < 0 ? ~p : p); }

template <int DT>
constexpr uint32_t kVec = DT == kDtF32 ? 4u : 8u;

template <int DT>
__device__ __forceinline__ void unpack(u32x4 w, float (&v)[kVec<DT>]) {
  if constexpr (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u2f(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = u2f(w[i] << 16);
      v[2 * i + 1] = u2f(w[i] & 0xFFFF0000u);
    }
  }
}
template <int DT>
__device__ __forceinline__ u32x4 pack(const float (&v)[kVec<DT>]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kDtF32)
      w[i] = f2u(v[i]);
    else
      w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  }
  return w;
}

// A wave's place: token and first vector.
struct Place {
  uint32_t t, v;
  bool live;
};
__device__ __forceinline__ Place place(uint32_t T, uint32_t nv) {
  const uint32_t segs = (nv + 63u) / 64u, w = blockIdx.x * 4u + uniform(threadIdx.x >> 6);
  const uint32_t t = w / segs;
  return Place{t, (w - t * segs) * 64u + (threadIdx.x & 63u), t < T};
}

// Row t of x (16-byte vectors, `stride` apart) to the rows of its k entries.
__global__ __launch_bounds__(256) void gather_kernel(const u32x4* __restrict__ x, int64_t stride,
                                                     const int32_t* __restrict__ pos, uint32_t T, uint32_t k,
                                                     uint32_t nv, uint32_t rows, u32x4* __restrict__ out) {
  const Place at = place(T, nv);
  if (!at.live || at.v >= nv) return;
  const u32x4 w = x[(size_t)at.t * (size_t)stride + at.v];
  for (uint32_t j = 0; j < k; ++j) {
    const uint32_t r = row_of(pos[(size_t)at.t * k + j]);
    if (r < rows) __builtin_nontemporal_store(w, out + (size_t)r * nv + at.v);
  }
}

// J entries of a token, from the j0-th: rows (past every row of y where there is
// none) and weights.
template <uint32_t J>
struct Entries {
  int32_t p[J];
  float w[J];
  bool all;  // every one is a row of y
  __device__ __forceinline__ Entries(const int32_t* __restrict__ pos, const float* __restrict__ weights, size_t at,
                                     uint32_t rows) {
    all = true;
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      p[j] = pos[at + j];
      w[j] = weights ? weights[at + j] : 1.0f;
      all &= (uint32_t)p[j] < rows;
    }
  }
};

// acc += w y over J entries, in order; their loads together.
template <int DT, uint32_t J>
__device__ __forceinline__ void combine_some(const u32x4* __restrict__ y, const Entries<J>& e, uint32_t nv, uint32_t v,
                                             uint32_t rows, float (&acc)[kVec<DT>]) {
  u32x4 raw[J];
  if (e.all) {
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) raw[j] = __builtin_nontemporal_load(y + (size_t)(uint32_t)e.p[j] * nv + v);
  }
#pragma unroll
  for (uint32_t j = 0; j < J; ++j) {
    if ((uint32_t)e.p[j] >= rows) continue;
    float x[kVec<DT>];
    unpack<DT>(e.all ? raw[j] : __builtin_nontemporal_load(y + (size_t)(uint32_t)e.p[j] * nv + v), x);
#pragma unroll
    for (uint32_t i = 0; i < kVec<DT>; ++i) acc[i] = __builtin_fmaf(e.w[j], x[i], acc[i]);
  }
}

template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(const u32x4* __restrict__ y, const int32_t* __restrict__ pos,
                                                      const float* __restrict__ weights, uint32_t T, uint32_t k,
                                                      uint32_t nv, uint32_t rows, u32x4* __restrict__ out,
                                                      int64_t stride) {
  const Place at = place(T, nv);
  if (!at.live || at.v >= nv) return;
  float acc[kVec<DT>] = {};
  const size_t entry = (size_t)at.t * k;
  uint32_t j = 0;
  for (; j + 4u <= k; j += 4u) combine_some<DT>(y, Entries<4>(pos, weights, entry + j, rows), nv, at.v, rows, acc);
  for (; j < k; ++j) combine_some<DT>(y, Entries<1>(pos, weights, entry + j, rows), nv, at.v, rows, acc);
  __builtin_nontemporal_store(pack<DT>(acc), out + (size_t)at.t * (size_t)stride + at.v);
}

// dy[pos] = w g, dw = g . y[pos]; entries that no expert takes: zeros.  W waves
// have a token, every W-th 64 vectors of it each; g is read once for J entries.
template <int DT, uint32_t W, uint32_t J>
__device__ __forceinline__ void backward_some(const u32x4* __restrict__ g, const u32x4* __restrict__ y,
                                              const Entries<J>& e, uint32_t nv, uint32_t rows, u32x4* __restrict__ dy,
                                              float* __restrict__ dw, bool live, float (&part)[4][4]) {
  const uint32_t lane = threadIdx.x & 63u, wave = uniform(threadIdx.x >> 6), own = wave % W;
  float sum[J] = {};
  for (uint32_t v = own * 64u + lane; live && v < nv; v += 64u * W) {
    u32x4 raw[J];
    float gv[kVec<DT>];
    if (e.all) {
#pragma unroll
      for (uint32_t j = 0; j < J; ++j) raw[j] = __builtin_nontemporal_load(y + (size_t)(uint32_t)e.p[j] * nv + v);
    }
    unpack<DT>(g[v], gv);
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) {
      const uint32_t r = row_of(e.p[j]);
      if (r >= rows) continue;
      float o[kVec<DT>] = {};
      if (e.p[j] >= 0) {
        float x[kVec<DT>];
        unpack<DT>(e.all ? raw[j] : __builtin_nontemporal_load(y + (size_t)r * nv + v), x);
#pragma unroll
        for (uint32_t i = 0; i < kVec<DT>; ++i) {
          sum[j] = __builtin_fmaf(gv[i], x[i], sum[j]);
          o[i] = e.w[j] * gv[i];
        }
      }
      __builtin_nontemporal_store(pack<DT>(o), dy + (size_t)r * nv + v);
    }
  }
#pragma unroll
  for (uint32_t j = 0; j < J; ++j) sum[j] = wave_fsum(sum[j]);
  if (W > 1u) {
    __syncthreads();  // (the sums before have been read)
    if (lane == 0u) {
#pragma unroll
      for (uint32_t j = 0; j < J; ++j) part[wave][j] = sum[j];
    }
    __syncthreads();
  }
  if (!live || own != 0u || lane >= J) return;
  float all = 0.0f;
  if (W > 1u) {
    for (uint32_t i = 0; i < W; ++i) all += part[wave + i][lane];
  } else {
#pragma unroll
    for (uint32_t j = 0; j < J; ++j) all = lane == j ? sum[j] : all;
  }
  dw[lane] = all;
}

template <int DT, uint32_t W>
__global__ __launch_bounds__(256) void combine_backward_kernel(const u32x4* __restrict__ g, int64_t stride,
                                                               const u32x4* __restrict__ y,
                                                               const int32_t* __restrict__ pos,
                                                               const float* __restrict__ weights, uint32_t T,
                                                               uint32_t k, uint32_t nv, uint32_t rows,
                                                               u32x4* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float part[4][4];
  const uint32_t at = blockIdx.x * (4u / W) + uniform(threadIdx.x >> 6) / W;
  const bool live = at < T;
  const uint32_t t = live ? at : T - 1u;  // (every wave comes to the barriers)
  const u32x4* row = g + (size_t)t * (size_t)stride;
  const size_t entry = (size_t)t * k;
  uint32_t j = 0;
  for (; j + 4u <= k; j += 4u)
    backward_some<DT, W>(row, y, Entries<4>(pos, weights, entry + j, rows), nv, rows, dy, dw + entry + j, live, part);
  for (; j < k; ++j)
    backward_some<DT, W>(row, y, Entries<1>(pos, weights, entry + j, rows), nv, rows, dy, dw + entry + j, live, part);
}

constexpr uint32_t kFewVectors = 128;

uint32_t vectors(int64_t H, int dtype) { return (uint32_t)(H / (dtype == kDtF32 ? 4 : 8)); }

}  // namespace

hipError_t launch_moe_route(const void* x, int dtype, int64_t stride, int64_t T, int64_t E, int32_t k,
                            bool renormalise, int32_t* ids, float* weights, hipStream_t s) {
  return by_experts<Route>(dtype, (uint32_t)E, x, stride, (uint32_t)T, (uint32_t)E, (uint32_t)k, renormalise, ids,
                           weights, s);
}

hipError_t launch_moe_route_backward(const void* x, int dtype, int64_t stride, int64_t T, int64_t E, int32_t k,
                                     bool renormalise, const int32_t* ids, const float* g, void* dx, hipStream_t s) {
  return by_experts<RouteBackward>(dtype, (uint32_t)E, x, stride, (uint32_t)T, (uint32_t)E, (uint32_t)k, renormalise,
                                   ids, g, dx, s);
}

// Entries of a chunk, and the chunks.
static bool sort_few(int64_t entries) { return entries <= (int64_t)kFewChunks * kSortThreads * kFewRounds; }
static uint32_t sort_chunks(int64_t entries) {
  const int64_t chunk = (int64_t)kSortThreads * (sort_few(entries) ? kFewRounds : kManyRounds);
  return (uint32_t)((entries + chunk - 1) / chunk);
}

// What any call of as many entries or fewer takes (small chunks are more than the first large ones).
size_t moe_sort_workspace(int64_t entries, int64_t E) {
  const int64_t few = std::min(entries, (int64_t)kFewChunks * kSortThreads * kFewRounds);
  const size_t chunks = std::max(sort_chunks(entries), sort_chunks(few));
  return chunks <= 1u ? 0u : kControlBytes + (chunks + 1u) * (size_t)(E + 1) * 4u;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t T, int32_t k, int64_t E, int32_t* group_off, int32_t* row_idx,
                           int32_t* pos, void* workspace, hipStream_t s) {
  const int64_t entries = T * k;
  const uint32_t n = (uint32_t)entries, bins = (uint32_t)E + 1u, chunks = sort_chunks(entries);
  uint32_t* counts = chunks > 1u ? reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kControlBytes) : nullptr;
  uint32_t bits = 1u;
  while ((1u << bits) < (uint32_t)E + 2u) ++bits;
  const size_t lds = kSortWaves * (size_t)(E + 2) * 4u;
  const auto go = [&](auto rounds) {
    constexpr uint32_t R = decltype(rounds)::value;
    if (counts) {
      sort_count_kernel<R><<<dim3(chunks), dim3(kSortThreads), 0, s>>>(ids, n, (uint32_t)E, counts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (R == kManyRounds && counts) {
      sort_scan_kernel<<<dim3((bins + 15u) / 16u), dim3(kSortThreads), 0, s>>>(counts, chunks, bins);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    sort_place_kernel<R><<<dim3(chunks ? chunks : 1u), dim3(kSortThreads), lds, s>>>(
        ids, n, (uint32_t)k, (uint32_t)E, bits, counts, group_off, row_idx, pos);
    return hipGetLastError();
  };
  if (sort_few(entries)) return go(std::integral_constant<uint32_t, kFewRounds>{});
  return go(std::integral_constant<uint32_t, kManyRounds>{});
}

// Workgroups of four waves, one wave to 64 vectors of a token.
static dim3 row_grid(int64_t T, uint32_t nv) { return dim3((uint32_t)((T * ((nv + 63u) / 64u) + 3) / 4)); }

hipError_t launch_moe_gather(const void* x, int dtype, int64_t stride, const int32_t* pos, int64_t T, int32_t k,
                             int64_t H, int64_t rows, void* out, hipStream_t s) {
  const uint32_t nv = vectors(H, dtype), per = dtype == kDtF32 ? 4u : 8u;
  gather_kernel<<<row_grid(T, nv), dim3(256), 0, s>>>(static_cast<const u32x4*>(x), stride / per, pos, (uint32_t)T,
                                                      (uint32_t)k, nv, (uint32_t)rows, static_cast<u32x4*>(out));
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int dtype, const int32_t* pos, const float* weights, int64_t T, int32_t k,
                              int64_t H, int64_t rows, void* out, int64_t stride, hipStream_t s) {
  const uint32_t nv = vectors(H, dtype), per = dtype == kDtF32 ? 4u : 8u;
  const auto go = [&](auto kernel) {
    kernel<<<row_grid(T, nv), dim3(256), 0, s>>>(static_cast<const u32x4*>(y), pos, weights, (uint32_t)T, (uint32_t)k,
                                                 nv, (uint32_t)rows, static_cast<u32x4*>(out), stride / per);
    return hipGetLastError();
  };
  return dtype == kDtF32 ? go(combine_kernel<kDtF32>) : go(combine_kernel<kDtBF16>);
}

hipError_t launch_moe_combine_backward(const void* g, int64_t stride, const void* y, int dtype, const int32_t* pos,
                                       const float* weights, int64_t T, int32_t k, int64_t H, int64_t rows, void* dy,
                                       float* dw, hipStream_t s) {
  const uint32_t nv = vectors(H, dtype), per = dtype == kDtF32 ? 4u : 8u;
  const auto go = [&](auto kernel, uint32_t tokens) {  // tokens of a workgroup
    kernel<<<dim3((uint32_t)((T + tokens - 1) / tokens)), dim3(256), 0, s>>>(
        static_cast<const u32x4*>(g), stride / per, static_cast<const u32x4*>(y), pos, weights, (uint32_t)T,
        (uint32_t)k, nv, (uint32_t)rows, static_cast<u32x4*>(dy), dw);
    return hipGetLastError();
  };
  // Four waves to a token's row while each has vectors of it to take (rows of 256: 102
  // us, 144 with one wave; of 128: 130 and 125; of 32: 82 and 36; 40000 and 16384 tokens).
  if (nv > kFewVectors)
    return dtype == kDtF32 ? go(combine_backward_kernel<kDtF32, 4>, 1u) : go(combine_backward_kernel<kDtBF16, 4>, 1u);
  return dtype == kDtF32 ? go(combine_backward_kernel<kDtF32, 1>, 4u) : go(combine_backward_kernel<kDtBF16, 1>, 4u);
}

}  // namespace fp4
