// logprobs.hip -- log probabilities of given tokens, entropy and the largest
// alternatives, in one pass over the logits; and their gradient.
//
// Forward.  With a running reference r (a logit), t_i = scale (x_i - r):
//   S = sum e^t_i,  W = sum t_i e^t_i;  lse = scale r + log S,
//   entropy = log S - W / S.
// Moving r to r' multiplies S by f = e^(scale (r - r')) and turns W into
// f (W + scale (r - r') S).  Each thread keeps its own (r, S, W) and moves r
// only when a logit passes it by 2^kLazy, so the common step is six VALU
// operations, one of them the exponential, for an element.  All in base 2 (t
// times log2 e), FP32.  Their issue (about 100 us) and the memory (130 us at
// 6.3 TB/s) bound it together: 4096 rows of 100003 BF16 take 138 us with the
// top 8 (5.9 TB/s), 133 us without; 1024 rows of 131072 FP32 86 us (6.2 TB/s).
//
// The top k in the same pass: the first 16 KB give a threshold with at least
// k elements at or above it (the k-th largest of 64 groups' maxima).  16-byte
// blocks that reach it, and later blocks that pass it, are noted in LDS (one
// ballot; looking at their elements there and then cost a quarter of the
// kernel's time).  The threshold rises as the row goes on (after 5, 17, 65,
// ... steps, from the groups' maxima so far): the number of blocks noted grows
// with the logarithm of V.  At the end the noted blocks' elements at or above
// the last threshold are ranked, a wave's first 64 blocks' from LDS (read once
// more they cost 2% for 6413 rows of 39381 BF16, which take 107 us), later
// ones' from memory.  An element equal to
// the threshold in a later block is never among the k: k elements before it
// are as large.  A row that overflows a buffer (a rising row, or one of few
// values) is read again for elements above the k-th largest of the groups'
// maxima over everything, and filled up with the first elements equal to
// that; one that overflows again, or holds a NaN, is searched k times.
//
// Few rows are split over workgroups; the last to arrive joins them.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"
#include "logit_rows.h"

#include <cfloat>

namespace fp4 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr uint32_t kThreads = 256, kWaves = 4;
constexpr uint32_t kUnroll = 4;                      // 16-byte blocks of a thread's step
constexpr uint32_t kStepBlocks = kThreads * kUnroll;  // 16 KB
constexpr uint32_t kGroups = 64;                     // groups of four threads
constexpr uint32_t kNoted = 512;                     // blocks a wave can note
constexpr uint32_t kKept = 64;                       // of which it keeps the elements
constexpr uint32_t kFew = 1024;                      // elements a workgroup can hold to rank them
constexpr uint32_t kMaxSplits = 64, kMaxTop = 32;
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int DT>
constexpr uint32_t kElem = DT == kDtF32 ? 4u : 8u;  // elements of a 16-byte block

template <int DT>
__device__ __forceinline__ float logit(const void* x, size_t i) {
  if (DT == kDtF32) return static_cast<const float*>(x)[i];
  return u2f((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
}

// A row and its 16-byte blocks (logit_rows.h says which can be loaded whole).
template <int DT>
struct Row : RowBlocks {
  static constexpr uint32_t kSize = DT == kDtF32 ? 4u : 2u, E = kElem<DT>;
  const uint8_t* p;  // the row's first element
  uint32_t V;
  __device__ __forceinline__ Row(const void* x, int64_t stride, size_t n, uint32_t rows, uint32_t V_)
      : p(static_cast<const uint8_t*>(x) + n * (size_t)stride * kSize), V(V_) {
    static_cast<RowBlocks&>(*this) = row_blocks<kSize>(reinterpret_cast<uintptr_t>(p), (uint32_t)n, rows, (uint32_t)stride, V_);
  }
  // Whether blocks [j, j + n) lie wholly inside the row.
  __device__ __forceinline__ bool inside(uint32_t j, uint32_t n) const {
    return j * E >= head && (uint64_t)(j + n) * E <= (uint64_t)V + head;
  }
  // Block j as it lies in memory, or the nearest that can be loaded (lo < hi).
  __device__ __forceinline__ u32x4 raw(uint32_t j) const {
    const uint8_t* at = p + ((int64_t)min(max(j, lo), hi - 1u) * E - head) * kSize;
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at));  // a logit is read once
  }
  // A step's blocks from j0 on, a thread's every 256th, as raw() gives them
  // (offsets in 32 bits from the step's first).
  __device__ __forceinline__ void raw_step(uint32_t j0, u32x4 (&w)[kUnroll]) const {
    if (lo >= hi) return;  // a matrix without a whole block
    const uint32_t from = min(j0, hi - 1u), least = max(lo, from) - from, most = hi - 1u - from;
    const uint8_t* at = p - head * kSize + (size_t)from * 16u;
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u) {
      const uint32_t j = min(max(u * kThreads + threadIdx.x, least), most);
      w[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(at + j * 16u));
    }
  }
  static __device__ __forceinline__ void values(u32x4 w, float (&v)[E]) {
    if constexpr (DT == kDtF32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = u2f(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = u2f(w[k] << 16);
        v[2 * k + 1] = u2f(w[k] & 0xFFFF0000u);
      }
    }
  }
  // The block that values() took apart.
  static __device__ __forceinline__ u32x4 block(const float (&v)[E]) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == kDtF32)
        w[k] = f2u(v[k]);
      else
        w[k] = (f2u(v[2 * k]) >> 16) | f2u(v[2 * k + 1]);
    }
    return w;
  }
  // Elements that blocks before `end` hold, counted from the row's first.
  __device__ __forceinline__ uint32_t limit(uint32_t end) const { return end == blocks ? V : end * E - head; }
  // Elements of block j from what raw(j) gave; -inf for those before the row
  // (their numbers wrap) and from `limit` on.
  __device__ __forceinline__ void edge_values(u32x4 w, uint32_t j, uint32_t limit, float (&v)[E]) const {
    values(w, v);
    const uint32_t i0 = j * E - head;
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) v[e] = i0 + e < limit ? v[e] : -INFINITY;
    if (j < lo || j >= hi) {
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        const bool in = i0 + e < limit;
        const float x = at(in ? i0 + e : 0u);
        v[e] = in ? x : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ float at(uint32_t i) const { return logit<DT>(p, i); }
};

// 64-bit key in the order (value, lower index first): NaN above all, +0 equal
// to -0.  0 is below every key.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t i) {
  uint32_t u = f2u(v + 0.0f);
  u = v != v ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)u << 32) | (uint32_t)~i;
}

struct Stats {
  float r, s, w;  // reference (a logit), S, W (base 2)
};
// c2 = scale log2 e.
__device__ __forceinline__ Stats join(Stats a, Stats b, float c2) {
  const float r = fmaxf(a.r, b.r);
  const float da = a.r == r ? 0.0f : (a.r - r) * c2, db = b.r == r ? 0.0f : (b.r - r) * c2;
  const float fa = exp2_fast(da), fb = exp2_fast(db);
  // A side that vanishes adds nothing, however far below it lies (da may overflow).
  return Stats{r, a.s * fa + b.s * fb,
               (fa == 0.0f ? 0.0f : (a.w + da * a.s) * fa) + (fb == 0.0f ? 0.0f : (b.w + db * b.s) * fb)};
}
// The wavefront's statistics joined, in every lane.
__device__ __forceinline__ Stats wave_join(Stats a, float c2) {
  const float r = wave_fmax(a.r);
  const float d = a.r == r ? 0.0f : (a.r - r) * c2, f = exp2_fast(d);
  return Stats{r, wave_fsum(a.s * f), wave_fsum(f == 0.0f ? 0.0f : (a.w + d * a.s) * f)};
}

// A step's t is v c2 + ref2 in one operation, ref2 = -r c2 rounded: (v - r) c2
// and what that rounding leaves, which is the same for every logit until the
// reference moves and is taken out then.  (Left in, threads whose references
// differ would weigh differently: 2^-24 |ref2|, 3e-3 for logits of 4e4, and the
// entropy is a mean over them.)  Beyond kFarRef, and where ref2 is not finite,
// differences come first and nothing is left over.
constexpr float kFarRef = 65536.0f;
__device__ __forceinline__ float ref_rest(float r, float c2) {
  const float ref = r == -INFINITY ? 0.0f : r, ref2 = -ref * c2;
  return fabsf(ref2) > kFarRef ? 0.0f : __builtin_fmaf(ref, c2, ref2);
}

struct Args {
  const void* x;
  int64_t stride;
  uint32_t rows;
  uint32_t V;
  float scale;
  const int32_t* tokens;
  int32_t M;
  float* logp;
  float* entropy;
  float* lse;
  int32_t top_k;
  float* top_logp;
  int32_t* top_index;
  uint32_t* done;   // arrival counters, one a row
  float* stats;     // rows x splits x 4
  uint64_t* keys;   // rows x splits x top_k
};

struct Shared {
  uint32_t noted[kWaves][kNoted];  // a wave's blocks, in no order
  u32x4 kept[kWaves][kKept];       // the first of them
  uint64_t few[kFew];              // keys to rank, in no order
  uint64_t best[kMaxTop];
  alignas(16) uint64_t group_key[kGroups];
  alignas(16) float group[kGroups];
  float tau;
  uint64_t tau_key;
  uint32_t wave_count[kWaves], few_count, flag;
  Stats part[kWaves];
  uint64_t wave_key[kWaves];
};

// The larger of a lane's key and its neighbour's (lane ^ 1, lane ^ 2), by DPP;
// the sum of a lane's count and its neighbour's.
template <int CTRL>
__device__ __forceinline__ uint64_t max_key_dpp(uint64_t a) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)a, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(a >> 32), CTRL, 0xF, 0xF, false);
  const uint64_t b = ((uint64_t)hi << 32) | lo;
  return a > b ? a : b;
}
template <int CTRL>
__device__ __forceinline__ uint32_t add_dpp(uint32_t a) {
  return a + (uint32_t)__builtin_amdgcn_mov_dpp((int)a, CTRL, 0xF, 0xF, false);
}

// The k-th largest of the 64 groups' maxima: every group of four threads gives
// its own (`mine` in all four) and counts those above it and those not below
// it, a quarter each.  (The largest with fewer than k above and k or more not
// below: every group that holds it writes it.)  Every thread of the workgroup
// calls it.
template <typename T>
__device__ __forceinline__ T kth_of_groups(T (&group)[kGroups], T& result, T mine, uint32_t k) {
  const uint32_t g = threadIdx.x >> 2, q0 = (threadIdx.x & 3u) * (kGroups / 4u);
  if ((threadIdx.x & 3u) == 0u) group[g] = mine;
  __syncthreads();
  uint32_t above = 0u, upto = 0u;
#pragma unroll
  for (uint32_t i = 0u; i < kGroups / 4u; ++i) {
    const T u = group[q0 + i];
    above += u > mine ? 1u : 0u;
    upto += u >= mine ? 1u : 0u;
  }
  above = add_dpp<0x4E>(add_dpp<0xB1>(above));
  upto = add_dpp<0x4E>(add_dpp<0xB1>(upto));
  if (above < k && k <= upto && (threadIdx.x & 3u) == 0u) result = mine;
  __syncthreads();
  return result;
}
__device__ __forceinline__ float threshold(Shared& sh, float mine, uint32_t k) {
  mine = fmaxf(mine, lane_xor1(mine));
  mine = fmaxf(mine, lane_xor2(mine));
  return kth_of_groups(sh.group, sh.tau, mine, k);
}

// Notes the lane's block j (elements v) where `is`; `count` goes on past their number.
template <int DT>
__device__ __forceinline__ void note(Shared& sh, bool is, uint32_t j, const float (&v)[kElem<DT>], uint32_t& count) {
  const uint64_t all = __ballot(is);
  const uint32_t at = count + (uint32_t)__popcll(all & ((1ull << (threadIdx.x & 63u)) - 1ull));
  if (is && at < kNoted) sh.noted[threadIdx.x >> 6][at] = j;
  if (is && at < kKept) sh.kept[threadIdx.x >> 6][at] = Row<DT>::block(v);
  count += (uint32_t)__popcll(all);
}

// Adds a key to those to rank; their number goes on past the array.
__device__ __forceinline__ void push(Shared& sh, uint64_t key) {
  const uint32_t at = atomicAdd(&sh.few_count, 1u);
  if (at < kFew) sh.few[at] = key;
}

// The value a key stands for (-0 as +0).
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return u == 0xFFFFFFFFu ? NAN : u2f((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}

// The largest k of few[0 .. n), n <= kFew, into best, in order (fewer: the
// rest 0).  Many: the k-th largest of 64 groups' maxima bounds the k-th
// largest from below first, which leaves little more than k; each of those is
// then ranked by counting the ones above it.
__device__ __forceinline__ void rank_few(Shared& sh, uint32_t n, uint32_t k) {
  const uint32_t tid = threadIdx.x;
  if (tid < k) sh.best[tid] = 0ull;
  __syncthreads();
  if (n > 64u) {
    uint64_t key[kFew / kThreads], mine = 0ull;
#pragma unroll
    for (uint32_t i = 0; i < kFew / kThreads; ++i) {
      key[i] = i * kThreads + tid < n ? sh.few[i * kThreads + tid] : 0ull;
      mine = key[i] > mine ? key[i] : mine;
    }
    mine = max_key_dpp<0xB1>(mine);
    mine = max_key_dpp<0x4E>(mine);
    if (tid == 0u) sh.few_count = 0u;
    const uint64_t kth = kth_of_groups(sh.group_key, sh.tau_key, mine, k);
#pragma unroll
    for (uint32_t i = 0; i < kFew / kThreads; ++i)
      if (key[i] != 0ull && key[i] >= kth) push(sh, key[i]);
    __syncthreads();
    n = sh.few_count;
  }
  for (uint32_t i = tid; i < n; i += kThreads) {
    const uint64_t v = sh.few[i];
    uint32_t rank = 0u;
#pragma unroll 8
    for (uint32_t j = 0u; j < n; ++j) rank += sh.few[j] > v ? 1u : 0u;
    if (v != 0ull && rank < k) sh.best[rank] = v;
  }
  __syncthreads();
}

// k searches of blocks [b0, b1) for the largest key below the last (the first
// takes any: a NaN at index 0 has the largest key there is).
template <int DT>
__device__ __forceinline__ void search(Shared& sh, const Row<DT>& row, uint32_t b0, uint32_t b1, uint32_t k) {
  constexpr uint32_t E = kElem<DT>;
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint64_t below = 0ull;
  for (uint32_t n = 0u; n < k; ++n) {
    uint64_t most = 0ull;
    for (uint32_t j = b0 + threadIdx.x; j < b1; j += kThreads) {
      for (uint32_t e = 0u; e < E; ++e) {
        const int64_t i = (int64_t)j * E + e - row.head;
        if (i < 0 || i >= row.V) continue;
        const uint64_t key = top_key(row.at((uint32_t)i), (uint32_t)i);
        if ((n == 0u || key < below) && key > most) most = key;
      }
    }
    for (int d = 32; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)most, d);
      most = o > most ? o : most;
    }
    if (lane == 0u) sh.wave_key[wave] = most;
    __syncthreads();
    for (uint32_t w = 0u; w < kWaves; ++w) most = sh.wave_key[w] > most ? sh.wave_key[w] : most;
    __syncthreads();
    below = most;
    if (threadIdx.x == 0u) sh.best[n] = most;
  }
  __syncthreads();
}

// best[have .. k): the first elements of blocks [b0, b1) equal to tau.
template <int DT>
__device__ __forceinline__ void fill_ties(Shared& sh, const Row<DT>& row, uint32_t b0, uint32_t b1, float tau,
                                       uint32_t have, uint32_t k) {
  if (threadIdx.x < 64u) {
    const int64_t first = (int64_t)b0 * kElem<DT> - row.head, end = (int64_t)b1 * kElem<DT> - row.head;
    const int64_t lo = first < 0 ? 0 : first, hi = end < row.V ? end : row.V;
    for (int64_t i0 = lo; i0 < hi && have < k; i0 += 64) {
      const int64_t i = i0 + threadIdx.x;
      const float v = i < hi ? row.at((uint32_t)i) : 0.0f;
      const bool eq = i < hi && v == tau;
      const uint64_t all = __ballot(eq);
      const uint32_t at = have + (uint32_t)__popcll(all & ((1ull << threadIdx.x) - 1ull));
      if (eq && at < k) sh.best[at] = top_key(v, (uint32_t)i);
      have += (uint32_t)__popcll(all);
    }
  }
  __syncthreads();
}

// lse and entropy of joined statistics.  Nothing but -inf: -inf and 0; a NaN
// or +inf logit: NaN.
__device__ __forceinline__ void finish(Stats a, float scale, float& lse, float& entropy) {
  if (a.r == INFINITY) a.s = NAN;  // inf - inf
  const float ls = logf(a.s);
  lse = a.s == 0.0f ? -INFINITY : __builtin_fmaf(a.r, scale, ls);
  entropy = a.s == 0.0f ? 0.0f : ls - kLn2 * a.w / a.s;
}

__device__ __forceinline__ float log_prob(float x, float scale, float lse) {
  const float y = x * scale;
  return y == -INFINITY && lse == lse ? -INFINITY : y - lse;
}

// The logit of the row's token j, and whether it is one (else padding).
template <int DT>
__device__ __forceinline__ float token_logit(const Args& a, const Row<DT>& row, size_t n, int32_t j, bool& is) {
  const int32_t t = j < a.M ? a.tokens[n * (size_t)a.M + j] : -1;
  is = t >= 0 && (uint32_t)t < a.V;
  return is ? row.at((uint32_t)t) : 0.0f;
}

// One row's outputs: statistics in every thread, the top keys in sh.best, the
// thread's first token's logit in x0 (asked for before the statistics were).
template <int DT>
__device__ __forceinline__ void write_row(const Args& a, Shared& sh, const Row<DT>& row, size_t n, Stats st, float x0,
                                          bool is0) {
  float lse, entropy;
  finish(st, a.scale, lse, entropy);
  if (threadIdx.x == 0u) {
    if (a.lse) a.lse[n] = lse;
    if (a.entropy) a.entropy[n] = entropy;
  }
  for (int32_t j = (int32_t)threadIdx.x; j < a.M; j += (int32_t)kThreads) {
    if (j >= (int32_t)kThreads) x0 = token_logit<DT>(a, row, n, j, is0);
    a.logp[n * (size_t)a.M + j] = is0 ? log_prob(x0, a.scale, lse) : 0.0f;
  }
  if ((int32_t)threadIdx.x < a.top_k) {
    const bool some = threadIdx.x < a.V;
    const uint64_t key = sh.best[threadIdx.x];
    const size_t at = n * (size_t)a.top_k + threadIdx.x;
    a.top_index[at] = some ? (int32_t)~(uint32_t)key : -1;
    a.top_logp[at] = some ? log_prob(key_value(key), a.scale, lse) : -INFINITY;
  }
}

template <int DT>
__global__ __launch_bounds__(256) void logprobs_kernel(Args a) {
  constexpr uint32_t E = kElem<DT>;
  __shared__ Shared sh;
  const uint32_t split = blockIdx.x, splits = gridDim.x, tid = threadIdx.x;
  const size_t n = blockIdx.y;
  const Row<DT> row(a.x, a.stride, n, a.rows, a.V);
  const uint32_t per = (row.blocks + splits - 1u) / splits;
  const uint32_t b0 = min(split * per, row.blocks), b1 = min(b0 + per, row.blocks);
  const uint32_t k = (uint32_t)a.top_k;
  const float c2 = a.scale * kLog2e;

  Stats st = {-INFINITY, 0.0f, 0.0f};
  float mine = -INFINITY, tau = INFINITY;  // this thread's largest; nothing passes until the threshold is known
  uint32_t count = 0u;                     // blocks this wave has noted
  const bool only = b1 - b0 <= kStepBlocks;
  if (tid == 0u) sh.few_count = 0u;
  u32x4 next[kUnroll] = {};
  const uint32_t limit = row.limit(b1);
  if (b0 < b1) row.raw_step(b0, next);
  for (uint32_t s0 = b0; s0 < b1; s0 += kStepBlocks) {
    float v[kUnroll][E];
    const uint32_t used = min((b1 - s0 + kThreads - 1u) / kThreads, kUnroll);  // blocks of a thread
    if (s0 + kStepBlocks <= b1 && row.inside(s0, kStepBlocks)) {
#pragma unroll
      for (uint32_t u = 0; u < kUnroll; ++u) Row<DT>::values(next[u], v[u]);
    } else {
#pragma unroll
      for (uint32_t u = 0; u < kUnroll; ++u) row.edge_values(next[u], s0 + u * kThreads + tid, limit, v[u]);
    }
    if (s0 + kStepBlocks < b1) row.raw_step(s0 + kStepBlocks, next);
    float hi[kUnroll], top = -INFINITY;
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u) {
      hi[u] = v[u][0];
#pragma unroll
      for (uint32_t e = 1; e < E; ++e) hi[u] = fmaxf(hi[u], v[u][e]);
      top = fmaxf(top, hi[u]);
    }
    mine = fmaxf(mine, top);
    if (__any((top - st.r) * c2 > kLazy || st.r == -INFINITY)) {
      const float r = fmaxf(st.r, top);
      const float d = st.r == r ? 0.0f : (st.r - r) * c2 + (ref_rest(r, c2) - ref_rest(st.r, c2)), f = exp2_fast(d);
      st.w = f == 0.0f ? 0.0f : (st.w + d * st.s) * f;
      st.s *= f;
      st.r = r;
    }
    const float ref = st.r == -INFINITY ? 0.0f : st.r, ref2 = -ref * c2;
    float s = st.s, w = st.w;
#pragma unroll
    for (uint32_t u = 0; u < kUnroll; ++u) {
      if (u >= used) continue;  // (also parts the code so that it takes 92 registers, not 141)
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        const float t = __builtin_fmaf(v[u][e], c2, ref2), p = exp2_fast(t);
        s += p;
        w = __builtin_fmaf(t, p, w);
      }
    }
    constexpr int kNanOrInf = 0x207;
    if (__any(__builtin_amdgcn_classf(w, kNanOrInf) || fabsf(ref2) > kFarRef)) {
      // A masked logit (-inf, or so low that t is): e^t is 0, and t e^t has
      // to be too.  (Or a NaN, which stays one in s.)  Or logits so large that
      // the product's rounding shows in t (or that ref2 overflows).  Again, with
      // care, and with differences first.
      const float rest = ref_rest(st.r, c2);
      s = st.s;
      w = st.w;
#pragma unroll
      for (uint32_t u = 0; u < kUnroll; ++u)
#pragma unroll
        for (uint32_t e = 0; e < E; ++e) {
          const float t = __builtin_fmaf(v[u][e] - ref, c2, rest), p = exp2_fast(t);
          s += p;
          w = __builtin_fmaf(fmaxf(t, -1000.0f), p, w);
        }
    }
    st.s = s;
    st.w = w;
    if (k > 0u) {
      const uint32_t step = (s0 - b0) / kStepBlocks;
      if (step == 0u) {
        // (Masked logits, -inf, are not noted; fill_ties finds the first where they are needed.)
        tau = threshold(sh, mine, k);
        if (only) {
          // A workgroup's one step: its elements are still at hand.
          const float least = fmaxf(tau, -FLT_MAX);
#pragma unroll
          for (uint32_t u = 0; u < kUnroll; ++u) {
            if (!(hi[u] >= least)) continue;
            const uint32_t i0 = (s0 + u * kThreads + tid) * E - row.head;
#pragma unroll
            for (uint32_t e = 0; e < E; ++e)
              if (v[u][e] >= least) push(sh, top_key(v[u][e], i0 + e));
          }
          continue;
        }
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u)
          note<DT>(sh, hi[u] >= tau && hi[u] > -INFINITY, s0 + u * kThreads + tid, v[u], count);
      } else {
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u)
          if (__any(hi[u] > tau)) note<DT>(sh, hi[u] > tau, s0 + u * kThreads + tid, v[u], count);
        if (step == 4u || step == 16u || step == 64u || step == 256u) tau = threshold(sh, mine, k);
      }
    }
  }

  // The workgroup's statistics, in a fixed order, relative to the references themselves.
  const float rest = ref_rest(st.r, c2), less = exp2_fast(-rest);
  st.w = (st.w - rest * st.s) * less;
  st.s *= less;
  st = wave_join(st, c2);
  if ((tid & 63u) == 0u) {
    sh.part[tid >> 6] = st;
    sh.wave_count[tid >> 6] = count;
  }
  __syncthreads();
  st = join(join(sh.part[0], sh.part[1], c2), join(sh.part[2], sh.part[3], c2), c2);

  if (k > 0u) {
    const bool special = !(st.s == st.s) || st.r == INFINITY;
    const uint32_t most = max(max(sh.wave_count[0], sh.wave_count[1]), max(sh.wave_count[2], sh.wave_count[3]));
    bool over = special || most > kNoted;
    if (!over) {
      // The noted blocks' elements.
      const float least = fmaxf(tau, -FLT_MAX);
      for (uint32_t i = tid & 63u; i < count; i += 64u) {
        const uint32_t j = sh.noted[tid >> 6][i];
        float v[E];
        if (i < kKept)
          Row<DT>::values(sh.kept[tid >> 6][i], v);
        else
          row.edge_values(row.lo < row.hi ? row.raw(j) : u32x4{}, j, limit, v);
#pragma unroll
        for (uint32_t e = 0; e < E; ++e)
          if (v[e] >= least) push(sh, top_key(v[e], j * E - row.head + e));
      }
      __syncthreads();
      over = sh.few_count > kFew;
    }
    if (over && !special) {
      // Too many: again, above the k-th largest of the groups' maxima over all.
      tau = threshold(sh, mine, k);  // (its barriers end the reading of few_count)
      if (tid == 0u) sh.few_count = 0u;
      __syncthreads();
      for (uint32_t j = b0 + tid; j < b1; j += kThreads) {
        float v[E];
        row.edge_values(row.lo < row.hi ? row.raw(j) : u32x4{}, j, limit, v);
#pragma unroll
        for (uint32_t e = 0; e < E; ++e)
          if (v[e] > tau) push(sh, top_key(v[e], j * E - row.head + e));
      }
      __syncthreads();
      over = sh.few_count > kFew;
    }
    if (over) {
      search<DT>(sh, row, b0, b1, k);
    } else {
      const uint32_t n_few = sh.few_count;
      rank_few(sh, n_few, k);
      if (n_few < k) fill_ties<DT>(sh, row, b0, b1, tau, n_few, k);
    }
  }
  float x0 = 0.0f;
  bool is0 = false;
  if (splits == 1u) {
    x0 = token_logit<DT>(a, row, n, (int32_t)tid, is0);
    write_row<DT>(a, sh, row, n, st, x0, is0);
    return;
  }

  // ---- the splits' results, written through; the last to arrive joins them ----
  const size_t part = n * splits;
  if (tid < k)
    __hip_atomic_store(a.keys + (part + split) * k + tid, sh.best[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (tid < 3u)
    __hip_atomic_store(a.stats + (part + split) * 4u + tid, tid == 0u ? st.r : tid == 1u ? st.s : st.w,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's results have reached the coherence point
  __syncthreads();
  if (tid == 0u) {
    const uint32_t before = __hip_atomic_fetch_add(a.done + n, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh.flag = before == splits - 1u;
    if (sh.flag) __hip_atomic_store(a.done + n, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!sh.flag) return;
  x0 = token_logit<DT>(a, row, n, (int32_t)tid, is0);
  Stats all = {-INFINITY, 0.0f, 0.0f};
  if ((tid & 63u) < splits) {
    const float* from = a.stats + (part + (tid & 63u)) * 4u;
    all.r = __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    all.s = __hip_atomic_load(from + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    all.w = __hip_atomic_load(from + 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  all = wave_join(all, c2);
  if (k > 0u) {
    // splits x k <= kFew (the host's choice of splits); those of splits with
    // fewer than k elements are 0, none.
    for (uint32_t i = tid; i < splits * k; i += kThreads)
      sh.few[i] = __hip_atomic_load(a.keys + part * k + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    rank_few(sh, splits * k, k);
  }
  write_row<DT>(a, sh, row, n, all, x0, is0);
}

// ---------------------------------------------------------------------------
// Gradient: dx_i = scale (hot_i - p_i (G + ge (log p_i + H))), one pass, 16
// bytes a step, bound by the memory (4096 rows of 100003 BF16: 264 us, 6.2 TB/s
// read and written; 256 rows of 32768 FP32 12.5 us, 5.3 TB/s).  The tokens' own
// terms are rare: a bitmap marks the blocks that hold one, and only those look
// through the row's tokens.
// ---------------------------------------------------------------------------
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
__global__ __launch_bounds__(256) void logprobs_backward_kernel(
    const void* __restrict__ x, int64_t stride, uint32_t V, float scale, const int32_t* __restrict__ tokens, int32_t M,
    const float* __restrict__ lse, const float* __restrict__ entropy, const float* __restrict__ g_logp,
    const float* __restrict__ g_entropy, void* __restrict__ dx, int64_t dx_stride, uint32_t rows) {
  constexpr uint32_t E = kElem<DT>;
  __shared__ uint32_t marked[kStepBlocks / 32u];
  __shared__ float sums[kWaves];
  const size_t n = blockIdx.y;
  const uint32_t tid = threadIdx.x;
  const Row<DT> row(x, stride, n, rows, V);
  const uint32_t b0 = blockIdx.x * kStepBlocks;
  if (b0 >= row.blocks) return;
  float v[kUnroll][E];
  u32x4 raw[kUnroll] = {};
  row.raw_step(b0, raw);
  if (tid < kStepBlocks / 32u) marked[tid] = 0u;
  __syncthreads();
  const int32_t* tok = tokens + n * (size_t)M;
  const float* gl = g_logp + n * (size_t)M;
  float g = 0.0f;
  for (int32_t j = (int32_t)tid; j < M; j += (int32_t)kThreads) {
    const int32_t t = tok[j];
    if (t < 0 || (uint32_t)t >= V) continue;
    g += gl[j];
    const uint32_t blk = ((uint32_t)t + row.head) / E - b0;
    if (blk < kStepBlocks) atomicOr(&marked[blk >> 5], 1u << (blk & 31u));
  }
  g = wave_fsum(g);
  if ((tid & 63u) == 0u) sums[tid >> 6] = g;
  __syncthreads();
  g = (sums[0] + sums[1]) + (sums[2] + sums[3]);

  const float ge = g_entropy ? g_entropy[n] : 0.0f, h = g_entropy ? entropy[n] : 0.0f;
  // A row of -inf logits: every p is 0 (its lse of -inf would give NaN).
  const float ls = lse[n] == -INFINITY ? INFINITY : lse[n];
  const float A = -(g + ge * h), B = -ge;
  const bool whole = row.inside(b0, kStepBlocks);
#pragma unroll
  for (uint32_t u = 0; u < kUnroll; ++u) {
    if (whole)
      Row<DT>::values(raw[u], v[u]);
    else
      row.edge_values(raw[u], b0 + u * kThreads + tid, V, v[u]);
  }
  uint8_t* out = static_cast<uint8_t*>(dx) + n * (size_t)dx_stride * (DT == kDtF32 ? 4u : 2u);
#pragma unroll
  for (uint32_t u = 0; u < kUnroll; ++u) {
    const uint32_t blk = u * kThreads + tid, j = b0 + blk;
    if (j >= row.blocks) continue;
    const int64_t i0 = (int64_t)j * E - row.head;
    float d[E];
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) {
      const float lp = __builtin_fmaf(v[u][e], scale, -ls), p = exp2_fast(lp * kLog2e);
      // p = 0 from lp = -inf must not meet an infinite factor.
      d[e] = p * __builtin_fmaf(B, fmaxf(lp, -1000.0f), A);
    }
    if (marked[blk >> 5] & (1u << (blk & 31u))) {
      for (int32_t q = 0; q < M; ++q) {
        const int64_t e = (int64_t)tok[q] - i0;
        if (tok[q] < 0 || (uint32_t)tok[q] >= V || e < 0 || e >= E) continue;
#pragma unroll
        for (uint32_t f = 0; f < E; ++f) d[f] += f == (uint32_t)e ? gl[q] : 0.0f;
      }
    }
#pragma unroll
    for (uint32_t e = 0; e < E; ++e) d[e] *= scale;
    if (i0 >= 0 && i0 + E <= V) {
      u32x4_any w;
      if constexpr (DT == kDtF32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = f2u(d[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = bf16_pair(d[2 * k], d[2 * k + 1]);
      }
      // (The output's rows may be aligned otherwise than the input's.  Marked
      // as not read again here, which takes 9% off 4096 x 100003 BF16.)
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(out + i0 * (DT == kDtF32 ? 4 : 2)));
    } else {
#pragma unroll
      for (uint32_t e = 0; e < E; ++e) {
        if (i0 + e < 0 || i0 + e >= V) continue;
        if constexpr (DT == kDtF32)
          reinterpret_cast<float*>(out)[i0 + e] = d[e];
        else
          reinterpret_cast<__bf16*>(out)[i0 + e] = (__bf16)d[e];
      }
    }
  }
}

// Workgroups of a row: one where the rows alone fill the chip, else pieces of
// at least 2048 logits (8 a thread), as many as give about 512 workgroups,
// with all their top keys within one workgroup's candidates.  (64 rows of
// 131072 FP32, top 20: 17 us in 512 workgroups, 18 in 256 or 1024; 300 rows of
// 131072 BF16, top 8: 23 us, 27 in 300, 25 in 1200.)
constexpr int64_t kRowGroups = 512;
// The counters take the same place whatever the sizes, so that no other
// call's data ever lies where a call expects zeros.  (Rows are split only
// where there are fewer than kRowGroups.)
constexpr size_t kDoneBytes = (size_t)kRowGroups * 4;
uint32_t splits_of(int64_t N, int64_t V, int32_t top_k) {
  int64_t s = (kRowGroups + N - 1) / N;
  const int64_t most = (V + 2047) / 2048;
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  if (top_k > 0 && s > (int64_t)kFew / top_k) s = kFew / top_k;
  return (uint32_t)(s < 1 ? 1 : s);
}

}  // namespace

size_t logprobs_workspace(int64_t N, int64_t V, int32_t top_k) {
  if (N == 0) return 0;
  const size_t s = splits_of(N, V, top_k);
  return s == 1 ? 0 : kDoneBytes + (size_t)N * s * (16 + 8 * (size_t)top_k);
}

hipError_t launch_logprobs(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale,
                           const int32_t* tokens, int32_t M, float* logp, float* entropy, float* lse, int32_t top_k,
                           float* top_logp, int32_t* top_index, void* workspace, hipStream_t stream) {
  const uint32_t s = splits_of(N, V, top_k);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a{x, stride, 0u, (uint32_t)V, scale, tokens, M, logp, entropy, lse, top_k, top_logp, top_index, nullptr, nullptr,
         nullptr};
  if (s > 1) {
    a.done = reinterpret_cast<uint32_t*>(ws);
    a.stats = reinterpret_cast<float*>(ws + kDoneBytes);
    a.keys = reinterpret_cast<uint64_t*>(ws + kDoneBytes + (size_t)N * s * 16);
  }
  // Rows in the grid's y, at most 65535 a launch.
  for (int64_t n0 = 0; n0 < N; n0 += 65535) {
    const int64_t rows = N - n0 < 65535 ? N - n0 : 65535;
    Args b = a;
    b.x = static_cast<const uint8_t*>(x) + (size_t)n0 * (size_t)stride * (dtype == kDtF32 ? 4 : 2);
    b.rows = (uint32_t)rows;
    b.tokens = tokens + n0 * M;
    b.logp = logp + n0 * M;
    b.entropy = entropy ? entropy + n0 : nullptr;
    b.lse = lse ? lse + n0 : nullptr;
    b.top_logp = top_logp + n0 * top_k;
    b.top_index = top_index + n0 * top_k;
    const dim3 grid(s, (uint32_t)rows);
    if (dtype == kDtF32)
      logprobs_kernel<kDtF32><<<grid, kThreads, 0, stream>>>(b);
    else
      logprobs_kernel<kDtBF16><<<grid, kThreads, 0, stream>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_logprobs_backward(const void* x, int dtype, int64_t stride, int64_t N, int64_t V, float scale,
                                    const int32_t* tokens, int32_t M, const float* lse, const float* entropy,
                                    const float* g_logp, const float* g_entropy, void* dx, int64_t dx_stride,
                                    hipStream_t stream) {
  const size_t size = dtype == kDtF32 ? 4 : 2;
  const int64_t step = kStepBlocks * (16 / (int64_t)size);
  // A row that does not begin a line may reach into one step more than its length takes.
  const uint32_t steps = (uint32_t)((V + (int64_t)(128 / size) - 1 + step - 1) / step);
  for (int64_t n0 = 0; n0 < N; n0 += 65535) {
    const int64_t rows = N - n0 < 65535 ? N - n0 : 65535;
    const void* xr = static_cast<const uint8_t*>(x) + (size_t)n0 * (size_t)stride * size;
    void* dr = static_cast<uint8_t*>(dx) + (size_t)n0 * (size_t)dx_stride * size;
    const dim3 grid(steps, (uint32_t)rows);
    const float* ent = entropy ? entropy + n0 : nullptr;
    const float* ge = g_entropy ? g_entropy + n0 : nullptr;
    if (dtype == kDtF32)
      logprobs_backward_kernel<kDtF32><<<grid, kThreads, 0, stream>>>(
          xr, stride, (uint32_t)V, scale, tokens + n0 * M, M, lse + n0, ent, g_logp + n0 * M, ge, dr, dx_stride,
          (uint32_t)rows);
    else
      logprobs_backward_kernel<kDtBF16><<<grid, kThreads, 0, stream>>>(
          xr, stride, (uint32_t)V, scale, tokens + n0 * M, M, lse + n0, ent, g_logp + n0 * M, ge, dr, dx_stride,
          (uint32_t)rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4
