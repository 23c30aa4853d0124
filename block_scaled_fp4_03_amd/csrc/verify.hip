// verify.hip -- verification of drafted tokens against the target's
// probabilities, and the draw that follows, from given random numbers.
//
//   p, q: softmaxes of the target's and the draft's logits over the temperature;
//   draft d is kept while u q(d) < p(d); at the first that is not, the smallest
//   t with sum_{s <= t} r_s > u sum r, r = max(p - q, 0), is drawn (r = p past
//   the last draft).
//
// Exponentials and sums in FP64: the borders of a draw lie 1 / V apart, and
// FP32's 2^-24 would move one draw in a hundred at V = 131072.  2^z from a table
// of 2^(j / 256) and a cubic (relative error 2e-13).
//
// Two launches.  The sums of every row's parts, a wave each: the last workgroup of
// a sequence to arrive joins them and decides.  Then, of the row drawn from, the
// sums of chunks of r, a wave each: the last workgroup to arrive finds the token
// among the chunks, and within one.
//
// 64 sequences x 7 drafts over 100003 BF16 logits, a quarter of them greedy: 54 us
// for the rows (173 MB; 21.3 M vector instructions, 9 of 15 a logit FP64, are 35 us
// at 2.4 GHz) and 16 for the draws.  One sequence x 4 over 131072 FP32: 11 + 9 us,
// two chains of about seven memory latencies.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "workspace.h"

#include <algorithm>

namespace fp4 {
namespace {

constexpr uint32_t kThreads = 256, kWaves = 4;            // of the draw's workgroups
constexpr uint32_t kRowThreads = 256, kRowWaves = 4;      // of the rows'
static_assert(kRowWaves == kVerifyRowWaves);
constexpr uint32_t kRounds = 8;               // tokens of a chunk a lane has
constexpr uint32_t kChunk = 64u * kRounds;
static_assert(kChunk == kVerifyChunk);
constexpr uint32_t kRun = 4;                  // chunks' sums that a lane keeps (V up to 131072)
constexpr uint32_t kLaneParts = kVerifyMaxSplits * kRowWaves / 64u;  // a row's parts that a lane joins
constexpr uint32_t kMaxDrafts = 32;
// Waves for the draw, of a launch (64 x 15 rows of 100003 BF16: 4096 waves +3%).
constexpr int64_t kWantedWaves = 16384;
constexpr double kLog2e = 1.4426950408889634074;

// A wave's part of a row: the sum of 2^(c (x - r) / 256), r a logit; where the
// sequence is greedy, the largest logit's key.
struct Part {
  uint64_t value;   // the sum's bits, or the key
  uint64_t r_bad;   // r's bits; above them, whether there is a NaN
};
static_assert(sizeof(Part) == kVerifyPartBytes);

// What the draw needs of the row drawn from.
struct Chosen {
  double inv_p, inv_q;  // 1 / sum
  float rp, rq;
  uint32_t row;         // of the sequence's target rows
  int32_t q;            // kQNone, kQDraft, or the token that holds all of q
};
static_assert(sizeof(Chosen) == kVerifyChosenBytes);
constexpr int32_t kQNone = -1, kQDraft = -2, kNoDraw = -3;

struct Args {
  Verify v;
  uint32_t B, G, V, rows, splits, chunks;
  uint32_t per, groups;  // chunks of a wave, and workgroups of a sequence, in the draw
  Part* parts;       // B x rows x splits x kRowWaves; rows: G + 1 of the target, G of the draft
  double* sums;      // B x chunks
  Chosen* chosen;    // B
  uint32_t* arrived; // B counters, counter_words apart, zero before and after each launch
  uint32_t counter_words;
  uint32_t* drawn;   // the draw's, a line apart; zeroed where the sequence is decided
};
constexpr uint32_t kLineWords = kLineBytes / 4u;

template <int DT>
constexpr uint32_t kSize = DT == kDtF32 ? 4u : 2u;

template <int DT>
__device__ __forceinline__ float logit(const void* p, size_t i) {
  if (DT == kDtF32) return static_cast<const float*>(p)[i];
  return u2f((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ const uint8_t* row_at(const Args& a, uint32_t b, uint32_t row) {
  const bool target = row <= a.G;
  const uint8_t* p = static_cast<const uint8_t*>(target ? a.v.target : a.v.draft);
  const int64_t at = target ? b * a.v.target_seq + row * a.v.target_row
                            : b * a.v.draft_seq + (row - a.G - 1u) * a.v.draft_row;
  return p + at * kSize<DT>;
}

__device__ __forceinline__ uint64_t order_key(float v, uint32_t i) {
  const uint32_t u = f2u(v + 0.0f);
  return ((uint64_t)((u & 0x80000000u) ? ~u : u | 0x80000000u) << 32) | (uint32_t)~i;
}

__device__ __forceinline__ float temperature_of(const Args& a, uint32_t b) {
  return a.v.temperature ? a.v.temperature[b] : 1.0f;
}
// 256 log2 e / temperature; -1 where the sequence is greedy.
__device__ __forceinline__ double units_of(float t) { return t > 0.0f ? 256.0 * kLog2e / (double)t : -1.0; }

// 2^(j / 256), less j in the upper word's bits from 12 on: with k << 12 added
// there, entry k % 256 gives 2^(k / 256) at once.
constexpr uint32_t kTable = 256;
struct Table {
  uint64_t v[kTable];
};
constexpr Table make_table() {
  Table t{};
  for (uint32_t j = 0; j < kTable; ++j) {
    const double x = 0.69314718055994530942 * j / kTable;
    double sum = 0.0;
    for (int n = 1; n < 24; ++n) {  // e^x - 1, the small terms first
      double p = 1.0;
      for (int m = 24 - n; m > 0; --m) p *= x / m;
      sum += p;
    }
    t.v[j] = __builtin_bit_cast(uint64_t, 1.0 + sum) - ((uint64_t)j << 44);
  }
  return t;
}
__constant__ const Table kPowers = make_table();
typedef u32x2 Powers[kTable];

// 2^(k / 256).
__device__ __forceinline__ double power(const Powers& table, uint32_t k) {
  const u32x2 e = table[k & (kTable - 1u)];
  return __builtin_bit_cast(double, u32x2{e[0], e[1] + (k << 12)});
}

// A thread's entry, asked for before it is needed, and the table from them.
template <uint32_t THREADS>
struct TableEntries {
  static constexpr uint32_t N = (kTable + THREADS - 1u) / THREADS;
  u32x2 e[N];
  __device__ __forceinline__ TableEntries() {
#pragma unroll
    for (uint32_t i = 0; i < N; ++i) e[i] = __builtin_bit_cast(u32x2, kPowers.v[(threadIdx.x + i * THREADS) & (kTable - 1u)]);
  }
  __device__ __forceinline__ void fill(Powers& table) const {
#pragma unroll
    for (uint32_t i = 0; i < N; ++i)
      if (threadIdx.x + i * THREADS < kTable) table[threadIdx.x + i * THREADS] = e[i];
    __syncthreads();
  }
};

// 2^(f / 256) = 1 + kC1 f + kC2 f^2 + kC3 f^3 for |f| <= 1/2.
constexpr double kC1 = 0.69314718055994530942 / kTable, kC2 = kC1 * kC1 / 2.0, kC3 = kC1 * kC1 * kC1 / 6.0;

// 2^(y / 256), y <= 256 * 512; below -256 * 1000, and for a NaN, 2^-1000.
__device__ __forceinline__ double exp_units(double y, const Powers& table) {
  constexpr double kRound = 0x1.8p52;  // its last place is 1
  y = __builtin_fmax(y, -256.0 * 1000.0);
  const double t = y + kRound;
  const double f = y - (t - kRound);
  const double p = f * __builtin_fma(f, __builtin_fma(f, kC3, kC2), kC1);
  const double e = power(table, (uint32_t)__builtin_bit_cast(uint64_t, t));
  return __builtin_fma(e, p, e);
}
// The same, 0 below.
__device__ __forceinline__ double weight(float x, float r, double c, const Powers& table) {
  const double y = ((double)x - (double)r) * c, v = exp_units(y, table);
  return y > -256.0 * 1000.0 ? v : 0.0;
}

// Sum over the wavefront, in every lane and in a fixed order: rotations inside
// each row of 16 lanes (DPP), then the four rows' results.
template <int CTRL>
__device__ __forceinline__ double ror(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double from_lane(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += ror<0x121>(v);
  v += ror<0x122>(v);
  v += ror<0x124>(v);
  v += ror<0x128>(v);
  return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// What one workgroup hands to another is written through to the coherence point,
// and read from there.
template <typename T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether this workgroup is the last of n to come here (which resets the counter).
__device__ __forceinline__ bool last_of(uint32_t* arrived, uint32_t n, uint32_t& flag) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's results have reached the coherence point
  __syncthreads();
  if (threadIdx.x == 0u) {
    const uint32_t before = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    flag = before == n - 1u;
    if (flag) put(arrived, 0u);
  }
  __syncthreads();
  return flag != 0u;
}

struct RowSum {
  double inv;  // 1 / sum of the row
  float r;
  bool ok;     // it has a distribution: no NaN, no +inf, not all -inf
  uint32_t best;
};
// A draft: its token, the two models' logits of it, and its random number.
struct Draft {
  int32_t token;
  float xp, xq, u;
};
struct Shared {
  Powers table;
  Draft draft[kMaxDrafts];
  RowSum row[2 * kMaxDrafts + 1];
  uint32_t flag;
};
struct Running {
  double sum;
  float r;
  bool bad;
  uint64_t key;
};

// ---- the rows' sums ----------------------------------------------------------
// A wave's sum against a reference r that its lanes share, moved (to the lanes'
// largest logit) when a logit passes it by 2^500.  Of each logit, with R the
// whole number nearest c r:
//   t = c x - R to the nearest whole number, f = c x - R - t,
// both from an FMA's exact product.  Logits far below r are first raised to one
// whose term is 2^-900.  Where |c r| reaches 2^38 (a temperature near 0, a large
// finite mask as the reference), where that logit would lie below FP32's lowest value
// and where c vanishes, differences come first instead.
struct WaveSum {
  static constexpr double kRound = 0x1.8p52;
  double sum = 0.0, c, shift = 0.0;  // shift: kRound - R
  float r = -INFINITY, passes, low = 0.0f, c_passes;
  bool fast = false, bad = false;

  __device__ __forceinline__ explicit WaveSum(double c_) : c(c_), passes(-INFINITY) {
    c_passes = (float)(256.0 * 500.0 / c_);
  }
  // Factor from sums against R to sums against r.
  __device__ __forceinline__ double rest(const Powers& table) const {
    return fast ? exp_units(__builtin_fma(-(double)r, c, kRound - shift), table) : 1.0;
  }
  __device__ __forceinline__ void move(float m, const Powers& table) {
    bad |= m != m;
    m = wave_fmax(m);  // (a NaN left out)
    if (!(m > r)) return;
    const bool some = r != -INFINITY;
    if (some) sum *= rest(table) * weight(r, m, c, table);
    r = m;
    passes = fminf(r + c_passes, 0x1.fffffep127f);  // (a +inf logit passes it at every temperature)
    const double rc = (double)r * c;
    low = (float)((double)r - 256.0 * 900.0 / c);  // (FP32's rounding is 2^14 of those units at most)
    fast = c > 1e-30 && __builtin_fabs(rc) < 0x1p38 && low > -INFINITY;
    if (!fast) return;
    shift = kRound - __builtin_rint(rc);
    // From against r to against R: rest()'s inverse.
    if (some) sum *= exp_units(__builtin_fma((double)r, c, shift - kRound), table);
  }
  template <int N>
  __device__ __forceinline__ void add_fast(const float (&v)[N], const Powers& table) {
    double f[N], e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const double x = (double)__builtin_amdgcn_fmed3f(v[i], low, INFINITY);  // (a NaN gives low)
      const double t = __builtin_fma(x, c, shift);
      e[i] = power(table, (uint32_t)__builtin_bit_cast(uint64_t, t));
      f[i] = __builtin_fma(x, c, shift - t);  // t - shift: the whole number nearest c x
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      sum += __builtin_fma(e[i], f[i] * __builtin_fma(f[i], __builtin_fma(f[i], kC3, kC2), kC1), e[i]);
  }
  __device__ __forceinline__ void add(float v, const Powers& table) {
    if (v != -INFINITY) sum += exp_units(fast ? __builtin_fma((double)v, c, shift - kRound) : ((double)v - (double)r) * c, table);
  }
};

// The largest; a NaN if there is one.
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = __builtin_elementwise_maximum(m, v[i]);
  return m;
}

template <int DT, int N>
__device__ __forceinline__ void values(const u32x4& w, float (&v)[N]) {
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

// A wave's part of a split: blocks [b0, b1) of 16 bytes that lie wholly in the
// row, every fourth 1 KB of them, and, in split 0, the elements beside them.
template <int DT>
struct RowPart {
  static constexpr uint32_t E = 16u / kSize<DT>, U = 2u;
  static constexpr uint32_t kStep = U * kRowThreads;  // a split has whole steps, but the last
  static constexpr uint32_t kLowest = DT == kDtF32 ? 0xFF800000u : 0xFF80FF80u;  // -inf
  const uint8_t* p;
  const u32x4* from;
  uint32_t head, b0, b1, edge_at;
  bool first, edge;
  u32x4 next[U];  // the first step's blocks, on their way

  __device__ __forceinline__ RowPart(const uint8_t* p_, uint32_t V, uint32_t split, uint32_t splits) : p(p_) {
    head = min((uint32_t)(-reinterpret_cast<intptr_t>(p) & 15) / kSize<DT>, V);
    const uint32_t blocks = (V - head) / E, tail = head + blocks * E, steps = (blocks + kStep - 1u) / kStep;
    b0 = steps * split / splits * kStep;
    b1 = min(steps * (split + 1u) / splits * kStep, blocks);
    from = reinterpret_cast<const u32x4*>(p + (size_t)head * kSize<DT>);
    first = split == 0u;
    edge = first && threadIdx.x < head + (V - tail);
    edge_at = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    if (b0 < b1) load(b0, next);
  }
  // Blocks of the step at j0 (those past the end: the last one).
  __device__ __forceinline__ void load(uint32_t j0, u32x4 (&w)[U]) const {
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) w[u] = from[min(j0 + u * kRowThreads + threadIdx.x, b1 - 1u)];
  }
  __device__ __forceinline__ Running run(double c, const Powers& table);
};

template <int DT>
__device__ __forceinline__ Running RowPart<DT>::run(double c, const Powers& table) {
  Running s{0.0, -INFINITY, false, 0ull};
  if (c < 0.0) {
    float best = -INFINITY;
    uint32_t at = 0u;
    for (uint32_t j0 = b0; j0 < b1; j0 += U * kRowThreads) {
      u32x4 w[U];
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) w[u] = next[u];
      load(j0 + U * kRowThreads, next);
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        float v[E];
        values<DT, E>(w[u], v);
        const float m = largest(v);
        if (!(m <= best)) {  // (rarely)
          s.bad |= m != m;
          best = m;
#pragma unroll
          for (int i = (int)E - 1; i >= 0; --i)
            at = v[i] == m ? head + min(j0 + u * kRowThreads + threadIdx.x, b1 - 1u) * E + i : at;
        }
      }
    }
    if (best > -INFINITY) s.key = order_key(best, at);
    if (edge) {
      const float v = logit<DT>(p, edge_at);
      const uint64_t key = order_key(v, edge_at);
      s.bad |= v != v;
      s.key = key > s.key ? key : s.key;
    }
    return s;
  }
  WaveSum sum(c);
  uint32_t j0 = b0;
  for (; j0 < b1; j0 += U * kRowThreads) {  // (the same steps for every lane)
    u32x4 w[U];
    float m = -INFINITY;  // the lane's largest logit of this step
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) w[u] = next[u];
    load(j0 + U * kRowThreads, next);  // (past the end: the last block)
    if (j0 + U * kRowThreads > b1) {
#pragma unroll
      for (uint32_t u = 0; u < U; ++u)
        if (j0 + u * kRowThreads + threadIdx.x >= b1) w[u] = u32x4{kLowest, kLowest, kLowest, kLowest};
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      float v[E];
      values<DT, E>(w[u], v);
      m = __builtin_elementwise_maximum(m, largest(v));
    }
    if (__any(!(m <= sum.passes))) {
      sum.move(m, table);
      if (!sum.fast && sum.r > -INFINITY) break;
    }
    if (!sum.fast) continue;  // nothing but masked logits so far
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      float v[E];
      values<DT, E>(w[u], v);
      if constexpr (DT == kDtF32) {
        sum.add_fast(v, table);
      } else {  // (four at a time: fewer registers, more waves)
        const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
        sum.add_fast(lo, table);
        sum.add_fast(hi, table);
      }
    }
  }
  // A temperature at the edge of its range, or a part that begins with nothing but a large
  // finite mask (-1e9 at temperature 1, the type's lowest value): a logit at a time, from the
  // step that showed it to the part's end (64 x 15 rows of 100003 BF16, the first 90% masked
  // so: 142 us with the draw, 56 with -inf).
  for (; j0 < b1; j0 += kRowThreads) {
    const bool in = j0 + threadIdx.x < b1;
    const u32x4 w = from[min(j0 + threadIdx.x, b1 - 1u)];
    float v[E];
    values<DT, E>(w, v);
    const float m = in ? largest(v) : -INFINITY;
    if (__any(!(m <= sum.passes))) sum.move(m, table);
#pragma unroll 1
    for (uint32_t i = 0; i < E; ++i)
      if (in) sum.add(logit<DT>(from + j0 + threadIdx.x, i), table);
  }
  if (first) {
    const float v = edge ? logit<DT>(p, edge_at) : -INFINITY;
    if (__any(!(v <= sum.passes))) sum.move(v, table);
    sum.add(v, table);
  }
  s.sum = sum.sum * sum.rest(table);
  s.r = sum.r;
  s.bad = sum.bad;
  return s;
}

// ---- the decision ------------------------------------------------------------
// Every row's sum, a wave a row at a time; a lane has kLaneParts of its parts.
__device__ __forceinline__ void join_rows(const Args& a, Shared& sh, uint32_t b, double c) {
  constexpr uint32_t kAhead = 4;  // rows whose parts are asked for together
  const uint32_t lane = threadIdx.x & 63u, rows = c < 0.0 ? a.G + 1u : a.rows, parts = a.splits * kRowWaves;
  for (uint32_t row0 = threadIdx.x >> 6; row0 < rows; row0 += kRowWaves * kAhead) {
    uint64_t value[kAhead][kLaneParts], r_bad[kAhead][kLaneParts];
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      const Part* from = a.parts + ((size_t)b * a.rows + row0 + i * kRowWaves) * parts;
#pragma unroll
      for (uint32_t k = 0; k < kLaneParts; ++k) {
        const bool in = row0 + i * kRowWaves < rows && lane + 64u * k < parts;
        value[i][k] = in ? get(&from[lane + 64u * k].value) : 0ull;
        r_bad[i][k] = in ? get(&from[lane + 64u * k].r_bad) : (uint64_t)0xFF800000u;  // -inf
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kAhead; ++i) {
      if (row0 + i * kRowWaves >= rows) break;
      bool bad = false;
      RowSum s{};
      if (c < 0.0) {
        uint64_t key = 0ull;
#pragma unroll
        for (uint32_t k = 0; k < kLaneParts; ++k) {
          key = value[i][k] > key ? value[i][k] : key;
          bad |= (r_bad[i][k] >> 32) != 0ull;
        }
        key = wave_max(key);
        const uint32_t top = (uint32_t)(key >> 32);  // the keys of -inf and +inf bound those of finite values
        s.best = ~(uint32_t)key;
        s.ok = __ballot(bad) == 0ull && top > 0x007FFFFFu && top < 0xFF800000u;
      } else {
        float r[kLaneParts], m = -INFINITY;
#pragma unroll
        for (uint32_t k = 0; k < kLaneParts; ++k) {
          r[k] = u2f((uint32_t)r_bad[i][k]);
          m = fmaxf(m, r[k]);
          bad |= (r_bad[i][k] >> 32) != 0ull;
        }
        s.r = wave_fmax(m);
        double sum = 0.0;
#pragma unroll
        for (uint32_t k = 0; k < kLaneParts; ++k)
          if (r[k] != -INFINITY) sum += __builtin_bit_cast(double, value[i][k]) * weight(r[k], s.r, c, sh.table);
        s.inv = 1.0 / wave_sum(sum);
        s.ok = __ballot(bad) == 0ull && s.r > -INFINITY && s.r < INFINITY;
      }
      if (lane == 0u) sh.row[row0 + i * kRowWaves] = s;
    }
  }
  __syncthreads();
}

// Decides over a sequence's drafts (wave 0, a lane a position) and writes all
// but a drawn token.
__device__ __forceinline__ void decide(const Args& a, const Shared& sh, uint32_t b, double c) {
  const bool greedy = c < 0.0;
  const uint32_t i = threadIdx.x;
  const Draft own = sh.draft[min(i, kMaxDrafts - 1u)];  // (of lanes past the drafts: not used)
  const int32_t d = i < a.G ? own.token : -1;
  bool keep = false;
  double odds = 0.0;
  if (i < a.G && (uint32_t)d < a.V && sh.row[i].ok) {
    const RowSum& p = sh.row[i];
    if (greedy) {
      keep = (uint32_t)d == p.best;
      odds = keep ? 1.0 : 0.0;
    } else if (!a.v.draft || sh.row[a.G + 1u + i].ok) {
      const RowSum& q = sh.row[a.v.draft ? a.G + 1u + i : i];
      const double pd = weight(own.xp, p.r, c, sh.table) * p.inv;
      const double qd = a.v.draft ? weight(own.xq, q.r, c, sh.table) * q.inv : 1.0;
      keep = (double)own.u * qd < pd;
      odds = pd >= qd ? (pd > 0.0 ? 1.0 : 0.0) : pd / qd;
    }
  }
  const uint32_t n = (uint32_t)__builtin_ctzll(__ballot(!keep));  // drafts kept (lane G keeps none)
  const RowSum& p = sh.row[n];
  if (i < a.G) a.v.chance[(size_t)b * a.G + i] = (float)odds;
  if (i <= a.G) a.v.out[(size_t)b * (a.G + 1u) + i] = i < n ? d : i == n && greedy && p.ok ? (int32_t)p.best : -1;
  const int32_t dn = __shfl(d, (int)n);
  if (i != 0u) return;
  put(a.drawn + (size_t)b * kLineWords, 0u);
  a.v.accepted[b] = (int32_t)n;
  Chosen s{p.inv, 0.0, p.r, 0.0f, n, kQNone};
  if (n < a.G && (uint32_t)dn < a.V) {
    if (!a.v.draft) {
      s.q = dn;
    } else if (!greedy && sh.row[a.G + 1u + n].ok) {
      s.q = kQDraft;
      s.inv_q = sh.row[a.G + 1u + n].inv;
      s.rq = sh.row[a.G + 1u + n].r;
    }
  }
  if (!p.ok || greedy) s.q = kNoDraw;
  a.chosen[b] = s;
}

template <int DT>
__global__ __launch_bounds__(kRowThreads) void stats_kernel(Args a) {
  __shared__ Shared sh;
  const uint32_t split = blockIdx.x % a.splits, n = blockIdx.x / a.splits, b = n / a.rows, row = n - b * a.rows;
  const float temperature = temperature_of(a, b);
  const TableEntries<kRowThreads> entries;
  RowPart<DT> part(row_at<DT>(a, b, row), a.V, split, a.splits);
  // The drafts' own logits: the last workgroup decides with them, and which that is
  // shows only when there is nothing left to hide their latency.
  if (threadIdx.x < a.G) {
    const uint32_t i = threadIdx.x;
    Draft d{a.v.tokens[(size_t)b * a.G + i], 0.0f, 0.0f, a.v.u[(size_t)b * (a.G + 1u) + i]};
    if ((uint32_t)d.token < a.V) {
      d.xp = logit<DT>(row_at<DT>(a, b, i), (uint32_t)d.token);
      if (a.v.draft) d.xq = logit<DT>(row_at<DT>(a, b, a.G + 1u + i), (uint32_t)d.token);
    }
    sh.draft[i] = d;
  }
  const double c = units_of(temperature);
  const bool greedy = c < 0.0;
  if (greedy && row > a.G) return;  // the draft's distribution is not asked for
  entries.fill(sh.table);
  const Running s = part.run(c, sh.table);
  {
    const uint64_t value = greedy ? wave_max(s.key) : __builtin_bit_cast(uint64_t, wave_sum(s.sum));  // (lanes share r)
    const uint64_t bad = __ballot(s.bad) != 0ull ? 1ull : 0ull;
    if ((threadIdx.x & 63u) == 0u) {
      Part* to = a.parts + ((size_t)n * a.splits + split) * kRowWaves + (threadIdx.x >> 6);
      put(&to->value, value);
      put(&to->r_bad, bad << 32 | f2u(s.r));
    }
  }
  if (!last_of(a.arrived + (size_t)b * a.counter_words, (greedy ? a.G + 1u : a.rows) * a.splits, sh.flag)) return;
  join_rows(a, sh, b, c);
  if (threadIdx.x < 64u) decide(a, sh, b, c);
}

// ---- the draw ----------------------------------------------------------------
__device__ __forceinline__ double scan(double v, uint32_t lane) {
#pragma unroll
  for (uint32_t d = 1; d < 64u; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// r of a chunk's tokens, 64 apart in a lane, and its sum.  The logits are all asked
// for before the first is used (tokens past the end: the last one, without weight).
template <int DT>
__device__ __forceinline__ double chunk_sum(const Args& a, const Chosen& s, const uint8_t* p, const uint8_t* q,
                                            uint32_t chunk, double c, const Powers& table,
                                            double (&w)[kRounds]) {
  const uint32_t t0 = chunk * kChunk + (threadIdx.x & 63u);
  float x[kRounds], y[kRounds];
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) x[r] = logit<DT>(p, min(t0 + 64u * r, a.V - 1u));
  if (s.q == kQDraft) {
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r) y[r] = logit<DT>(q, min(t0 + 64u * r, a.V - 1u));
  }
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) w[r] = weight(x[r], s.rp, c, table) * s.inv_p;
  if (s.q == kQDraft) {
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r) w[r] = __builtin_fmax(w[r] - weight(y[r], s.rq, c, table) * s.inv_q, 0.0);
  }
  double sum = 0.0;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const uint32_t t = t0 + 64u * r;
    // (A token that holds all of q has p < 1 there, or no weight is left in any.)
    if (t >= a.V || (s.q >= 0 && (uint32_t)s.q == t)) w[r] = 0.0;
    sum += w[r];
  }
  return wave_sum(sum);
}

// The token of a chunk at which the sum (`before` it) first passes `border`; the
// last that has any weight, if rounding leaves none; -1 if none has.
__device__ __forceinline__ int32_t pick(const double (&w)[kRounds], uint32_t chunk, double before, double border) {
  const uint32_t lane = threadIdx.x & 63u;
  int32_t token = -1;
  bool found = false;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const double upto = before + scan(w[r], lane);
    const uint64_t some = __ballot(w[r] > 0.0), past = __ballot(upto > border) & some;
    if (some && !found) {
      token = (int32_t)(chunk * kChunk + 64u * r + (past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(some)));
      found = past != 0ull;
    }
    before = from_lane(upto, 63);
  }
  return token;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void draw_kernel(Args a) {
  __shared__ Shared sh;
  const uint32_t group = blockIdx.x % a.groups, b = blockIdx.x / a.groups, lane = threadIdx.x & 63u;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const float temperature = temperature_of(a, b);
  const TableEntries<kThreads> entries;
  const double u = (double)a.v.u[(size_t)b * (a.G + 1u) + a.G];
  Chosen s = a.chosen[b];
  if (s.q == kNoDraw) return;
  // (In a workspace that was not zero-filled the rows may never have been decided:
  // whatever lies there then leads to none outside the tensors.)
  if (s.row > a.G || (s.q == kQDraft && (s.row == a.G || !a.v.draft))) return;
  const double c = units_of(temperature);
  entries.fill(sh.table);
  const uint8_t* p = row_at<DT>(a, b, s.row);
  const uint8_t* q = s.q == kQDraft ? row_at<DT>(a, b, a.G + 1u + s.row) : nullptr;
  double* sums = a.sums + (size_t)b * a.chunks;
  double w[kRounds];
  const uint32_t c0 = (group * kWaves + wave) * a.per, c1 = min(c0 + a.per, a.chunks);
  for (uint32_t i = c0; i < c1; ++i) {
    const double sum = chunk_sum<DT>(a, s, p, q, i, c, sh.table, w);
    if (lane == 0u) put(sums + i, sum);
  }
  if (!last_of(a.drawn + (size_t)b * kLineWords, a.groups, sh.flag)) return;
  if (wave != 0u) return;
  // A lane has a run of the chunks: the run, then the chunk, that passes the border;
  // the last with any weight, if none does.
  const uint32_t run = (a.chunks + 63u) / 64u, i0 = min(lane * run, a.chunks), i1 = min(i0 + run, a.chunks);
  double own_parts[kRun], mine = 0.0;  // the first of the run
#pragma unroll
  for (uint32_t i = 0; i < kRun; ++i) own_parts[i] = i0 + i < i1 ? get(sums + i0 + i) : 0.0;
#pragma unroll
  for (uint32_t i = 0; i < kRun; ++i) mine += own_parts[i];
  for (uint32_t i = i0 + kRun; i < i1; ++i) mine += get(sums + i);
  double upto = scan(mine, lane);
  const double total = from_lane(upto, 63), border = u * total;
  int32_t token = -1;
  if (total > 0.0) {
    const uint64_t some = __ballot(mine > 0.0), past = __ballot(upto > border) & some;
    const uint32_t l = past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(some);
    double before = __shfl(upto - mine, (int)l), chunk_before = before;
    uint32_t chunk = l * run;
    const uint32_t end = min((l + 1u) * run, a.chunks);
    if (run <= kRun) {
      bool hit = false;
#pragma unroll
      for (uint32_t i = 0; i < kRun; ++i) {
        const double part = __shfl(own_parts[i], (int)l);
        if (part > 0.0 && !hit) {
          chunk = l * run + i;
          chunk_before = before;
          hit = before + part > border;
        }
        before += part;
      }
    }
    for (uint32_t i = l * run; run > kRun && i < end; i += 64u) {
      const double part = i + lane < end ? get(sums + i + lane) : 0.0;
      upto = before + scan(part, lane);
      const uint64_t any = __ballot(part > 0.0), hit = __ballot(upto > border) & any;
      if (any) {
        const uint32_t at = hit ? (uint32_t)__builtin_ctzll(hit) : 63u - (uint32_t)__builtin_clzll(any);
        chunk = i + at;
        chunk_before = __shfl(upto - part, (int)at);
        if (hit) break;
      }
      before = from_lane(upto, 63);
    }
    chunk_sum<DT>(a, s, p, q, chunk, c, sh.table, w);
    token = pick(w, chunk, chunk_before, border);
  } else {
    // p and q alike to the last bit: nothing is left over, and p itself is drawn from.
    s.q = kQNone;
    double before = 0.0;
    for (uint32_t i = 0; i < a.chunks; ++i) {
      const double sum = chunk_sum<DT>(a, s, p, q, i, c, sh.table, w);
      if (sum > 0.0) token = pick(w, i, before, u);
      if (before + sum > u) break;
      before += sum;
    }
  }
  if (lane == 0u) a.v.out[(size_t)b * (a.G + 1u) + s.row] = token;
}

template <int DT>
hipError_t launch(const Args& a, hipStream_t stream) {
  stats_kernel<DT><<<dim3(a.B * a.rows * a.splits), dim3(kRowThreads), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  draw_kernel<DT><<<dim3(a.B * a.groups), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// For calls with and without draft logits, and any smaller ones.
size_t verify_workspace(int64_t B, int64_t G, int64_t V) {
  const int64_t n = std::min(B, kVerifyBatch);
  return n == 0 ? 0u : verify_bytes(n, 2 * G + 1, V);
}

hipError_t launch_verify(const Verify& v, hipStream_t stream) {
  Args a{};
  const int64_t most = std::min(v.B, kVerifyBatch), size = v.dtype == kDtF32 ? 4 : 2;
  a.G = (uint32_t)v.G;
  a.V = (uint32_t)v.V;
  a.rows = (uint32_t)(v.draft ? 2 * v.G + 1 : v.G + 1);
  const VerifyLayout w = verify_layout(most, a.rows, v.V);
  a.splits = w.splits;
  a.chunks = w.chunks;
  // A wave has one chunk while the chip has room, and more in a large batch.
  a.per = std::max<uint32_t>(1u, (uint32_t)(most * a.chunks / kWantedWaves));
  a.groups = (a.chunks + a.per * kWaves - 1u) / (a.per * kWaves);
  uint8_t* ws = static_cast<uint8_t*>(v.workspace);
  a.arrived = reinterpret_cast<uint32_t*>(ws);
  a.counter_words = w.counter_words;
  a.drawn = reinterpret_cast<uint32_t*>(ws + w.drawn);
  a.chosen = reinterpret_cast<Chosen*>(ws + w.chosen);
  a.sums = reinterpret_cast<double*>(ws + w.sums);
  a.parts = reinterpret_cast<Part*>(ws + w.parts);
  for (int64_t b = 0; b < v.B; b += kVerifyBatch) {
    a.v = v;
    a.B = (uint32_t)std::min(v.B - b, kVerifyBatch);
    a.v.target = static_cast<const uint8_t*>(v.target) + b * v.target_seq * size;
    if (v.draft) a.v.draft = static_cast<const uint8_t*>(v.draft) + b * v.draft_seq * size;
    if (v.tokens) a.v.tokens = v.tokens + b * v.G;
    a.v.u = v.u + b * (v.G + 1);
    if (v.temperature) a.v.temperature = v.temperature + b;
    a.v.out = v.out + b * (v.G + 1);
    a.v.accepted = v.accepted + b;
    if (v.chance) a.v.chance = v.chance + b * v.G;
    const hipError_t e = v.dtype == kDtF32 ? launch<kDtF32>(a, stream) : launch<kDtBF16>(a, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4
