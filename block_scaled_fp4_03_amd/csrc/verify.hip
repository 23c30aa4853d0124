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
// Three launches: the sums of every row's splits; of the row drawn from, the
// sums of chunks of r; and the token, found among the chunks, then within one.
#include "fp4_device.h"
#include "fp4_launch.h"

#include <algorithm>

namespace fp4 {
namespace {

constexpr uint32_t kThreads = 256, kWaves = 4;
constexpr uint32_t kTable = 256;              // 2^(j / 256)
constexpr uint32_t kRounds = 16;              // tokens of a chunk a thread has
constexpr uint32_t kChunk = kThreads * kRounds;
constexpr uint32_t kMaxSplits = 64, kMaxDrafts = 32;
constexpr double kLog2e = 1.4426950408889634074;

// A split's part of a row: sum of 2^(c (x - r)) / 256, r a logit; the largest
// logit's key where the sequence is greedy.
struct Part {
  double sum;
  float r;
  uint32_t bad;  // a NaN or +inf
  uint64_t key;
  uint64_t unused;
};

// What the draw needs of the row drawn from.
struct Chosen {
  double inv_p, inv_q;  // 1 / sum
  float rp, rq;
  uint32_t row;         // of the sequence's target rows
  int32_t q;            // kQNone, kQDraft, or the token that holds all of q
};
constexpr int32_t kQNone = -1, kQDraft = -2, kNoDraw = -3;

struct Args {
  Verify v;
  uint32_t B, G, V, rows, splits, chunks;
  Part* parts;     // B x rows x splits; rows: G + 1 of the target, G of the draft
  double* sums;    // B x chunks
  Chosen* chosen;  // B
};

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

// 256 log2 e / temperature; 0 where the sequence is greedy.
__device__ __forceinline__ double units_of(const Args& a, uint32_t b) {
  const float t = a.v.temperature ? a.v.temperature[b] : 1.0f;
  return t > 0.0f ? (double)kTable * kLog2e / (double)t : -1.0;
}

__device__ __forceinline__ void fill_table(double (&table)[kTable]) {
  table[threadIdx.x] = exp2((double)threadIdx.x / (double)kTable);
  __syncthreads();
}
static_assert(kTable == kThreads, "a thread fills one entry");

// 2^(y / 256), y <= 256 * 512; below -256 * 1000, and for a NaN, 2^-1000.
__device__ __forceinline__ double exp_units(double y, const double (&table)[kTable]) {
  constexpr double kRound = 0x1.8p52;  // its last place is 1
  constexpr double kC1 = 0.69314718055994530942 / kTable, kC2 = kC1 * kC1 / 2.0, kC3 = kC1 * kC1 * kC1 / 6.0;
  y = __builtin_fmax(y, -256.0 * 1000.0);
  const double t = y + kRound;
  const int32_t k = (int32_t)(uint32_t)__builtin_bit_cast(uint64_t, t);
  const double f = y - (t - kRound);
  const double p = f * __builtin_fma(f, __builtin_fma(f, kC3, kC2), kC1);
  const double e = table[(uint32_t)k & (kTable - 1u)];
  const uint64_t v = __builtin_bit_cast(uint64_t, __builtin_fma(e, p, e));
  return __builtin_bit_cast(double, v + ((uint64_t)(uint32_t)((k >> 8) << 20) << 32));
}
// The same, 0 below.
__device__ __forceinline__ double weight(float x, float r, double c, const double (&table)[kTable]) {
  const double y = ((double)x - (double)r) * c, v = exp_units(y, table);
  return y > -256.0 * 1000.0 ? v : 0.0;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// ---- the rows' sums ----------------------------------------------------------
struct Running {
  double sum;
  float r;  // reference, moved when a logit passes it by 2^500
  bool bad;
  uint64_t key;
};

template <int N>
__device__ __forceinline__ void take(Running& a, const float (&v)[N], double c, float c32,
                                     const double (&table)[kTable]) {
  float m = v[0];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmaxf(m, v[i]);
    a.bad |= v[i] != v[i];
  }
  if ((m - a.r) * c32 > 256.0f * 500.0f || a.r == -INFINITY) {
    a.sum = a.r == -INFINITY ? 0.0 : a.sum * weight(a.r, m, c, table);
    a.r = m;
  }
  const double r = (double)a.r;
#pragma unroll
  for (int i = 0; i < N; ++i) a.sum += exp_units(((double)v[i] - r) * c, table);
}

template <int N>
__device__ __forceinline__ void take_best(Running& a, const float (&v)[N], uint32_t i0) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a.bad |= v[i] != v[i];
    const uint64_t k = order_key(v[i], i0 + i);
    a.key = k > a.key ? k : a.key;
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void stats_kernel(Args a) {
  constexpr uint32_t E = 16u / kSize<DT>, U = 4u;
  __shared__ double table[kTable];
  __shared__ Running part[kWaves];
  const uint32_t split = blockIdx.x % a.splits, n = blockIdx.x / a.splits, b = n / a.rows, row = n - b * a.rows;
  const double c = units_of(a, b);
  const bool greedy = c < 0.0;
  if (greedy && row > a.G) return;  // the draft's distribution is not asked for
  fill_table(table);
  const uint8_t* p = row_at<DT>(a, b, row);
  // Blocks of 16 bytes that lie wholly in the row, and the elements beside them.
  const uint32_t head = min((uint32_t)(-reinterpret_cast<intptr_t>(p) & 15) / kSize<DT>, a.V);
  const uint32_t blocks = (a.V - head) / E;
  const uint32_t b0 = (uint32_t)((uint64_t)blocks * split / a.splits);
  const uint32_t b1 = (uint32_t)((uint64_t)blocks * (split + 1u) / a.splits);
  const u32x4* from = reinterpret_cast<const u32x4*>(p + (size_t)head * kSize<DT>);
  const float c32 = (float)c;
  Running s{0.0, -INFINITY, false, 0ull};
  const auto one = [&](const u32x4& w, uint32_t j) __attribute__((always_inline)) {
    float v[E];
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
    if (greedy)
      take_best(s, v, head + j * E);
    else
      take(s, v, c, c32, table);
  };
  uint32_t j = b0 + threadIdx.x;
  for (; j + (U - 1u) * kThreads < b1; j += U * kThreads) {
    u32x4 w[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) w[u] = from[j + u * kThreads];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) one(w[u], j + u * kThreads);
  }
  for (; j < b1; j += kThreads) one(from[j], j);
  // The elements before the first block and behind the last: split 0's threads.
  const uint32_t tail = head + blocks * E;
  if (split == 0u && threadIdx.x < head + (a.V - tail)) {
    const uint32_t i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    const float v[1] = {logit<DT>(p, i)};
    if (greedy)
      take_best(s, v, i);
    else
      take(s, v, c, c32, table);
  }
  // Joined over the workgroup.
  const float r = wave_fmax(s.r);
  double sum = s.r == -INFINITY ? 0.0 : s.r == r ? s.sum : s.sum * weight(s.r, r, c, table);
  sum = wave_sum(sum);
  const uint64_t key = wave_max(s.key);
  const bool bad = __ballot(s.bad) != 0ull;
  if ((threadIdx.x & 63u) == 0u) {
    Running& w = part[threadIdx.x >> 6];
    w.r = r;
    w.sum = sum;
    w.bad = bad;
    w.key = key;
  }
  __syncthreads();
  if (threadIdx.x != 0u) return;
  Part out{};
  out.r = fmaxf(fmaxf(part[0].r, part[1].r), fmaxf(part[2].r, part[3].r));
  for (uint32_t w = 0; w < kWaves; ++w) {
    if (part[w].r != -INFINITY) out.sum += part[w].sum * weight(part[w].r, out.r, c, table);
    out.bad |= part[w].bad ? 1u : 0u;
    out.key = part[w].key > out.key ? part[w].key : out.key;
  }
  a.parts[(size_t)n * a.splits + split] = out;
}

// ---- the decision ------------------------------------------------------------
struct RowSum {
  double inv;  // 1 / sum of the row
  float r;
  bool ok;     // it has a distribution: no NaN, no +inf, not all -inf
  uint32_t best;
};
struct Shared {
  double table[kTable];
  RowSum row[2 * kMaxDrafts + 1];
  Chosen chosen;
  double part[kRounds * kWaves];
  uint32_t found;
};

// Every row's sum, a wave a row, a lane a split.
__device__ __forceinline__ void join_rows(const Args& a, Shared& sh, uint32_t b, double c) {
  const uint32_t lane = threadIdx.x & 63u;
  for (uint32_t row = threadIdx.x >> 6; row < a.rows; row += kWaves) {
    if (c < 0.0 && row > a.G) break;
    Part p{};
    p.r = -INFINITY;
    if (lane < a.splits) p = a.parts[((size_t)b * a.rows + row) * a.splits + lane];
    const float r = wave_fmax(p.r);
    const double sum = wave_sum(p.r == -INFINITY ? 0.0 : p.sum * weight(p.r, r, c, sh.table));
    const uint64_t key = wave_max(p.key);
    const bool bad = __ballot(p.bad != 0u) != 0ull;
    if (lane == 0u) {
      RowSum& s = sh.row[row];
      s.inv = 1.0 / sum;
      s.r = r;
      s.best = ~(uint32_t)key;
      const uint32_t top = (uint32_t)(key >> 32);  // the keys of -inf and +inf bound those of finite values
      s.ok = !bad && (c < 0.0 ? top > 0x007FFFFFu && top < 0xFF800000u : r > -INFINITY && r < INFINITY);
    }
  }
  __syncthreads();
}

// Decides over a sequence's drafts (wave 0, a lane a position) and, in its first
// workgroup, writes all but a drawn token.
template <int DT>
__device__ __forceinline__ void decide(const Args& a, Shared& sh, uint32_t b, double c, bool first) {
  const bool greedy = c < 0.0;
  const int32_t* tokens = a.v.tokens + (size_t)b * a.G;
  if (threadIdx.x < 64u) {
    const uint32_t i = threadIdx.x;
    bool keep = false;
    double odds = 0.0;
    int32_t d = -1;
    if (i < a.G) {
      d = tokens[i];
      const RowSum& p = sh.row[i];
      if (p.ok && (uint32_t)d < a.V) {
        if (greedy) {
          keep = (uint32_t)d == p.best;
          odds = keep ? 1.0 : 0.0;
        } else {
          const double pd = weight(logit<DT>(row_at<DT>(a, b, i), (uint32_t)d), p.r, c, sh.table) * p.inv;
          double qd = 1.0;
          bool ok = true;
          if (a.v.draft) {
            const RowSum& q = sh.row[a.G + 1u + i];
            ok = q.ok;
            if (ok) qd = weight(logit<DT>(row_at<DT>(a, b, a.G + 1u + i), (uint32_t)d), q.r, c, sh.table) * q.inv;
          }
          if (ok) {
            keep = (double)a.v.u[(size_t)b * (a.G + 1u) + i] * qd < pd;
            odds = pd >= qd ? (pd > 0.0 ? 1.0 : 0.0) : pd / qd;
          }
        }
      }
    }
    const uint32_t n = (uint32_t)__builtin_ctzll(__ballot(!keep));  // drafts kept (lane G keeps none)
    if (first) {
      if (i < a.G) a.v.chance[(size_t)b * a.G + i] = (float)odds;
      const int32_t last = greedy && sh.row[n].ok ? (int32_t)sh.row[n].best : -1;
      if (i <= a.G) a.v.out[(size_t)b * (a.G + 1u) + i] = i < n ? d : i == n ? last : -1;
      if (i == 0u) a.v.accepted[b] = (int32_t)n;
    }
    if (i == 0u) {
      const RowSum& p = sh.row[n];
      Chosen& s = sh.chosen;
      s.row = n;
      s.inv_p = p.inv;
      s.rp = p.r;
      s.q = kQNone;
      if (n < a.G && (uint32_t)tokens[n] < a.V) {
        if (!a.v.draft) {
          s.q = tokens[n];
        } else if (!greedy && sh.row[a.G + 1u + n].ok) {
          s.q = kQDraft;
          s.inv_q = sh.row[a.G + 1u + n].inv;
          s.rq = sh.row[a.G + 1u + n].r;
        }
      }
      if (!p.ok || greedy) s.q = kNoDraw;
      if (first) a.chosen[b] = s;
    }
  }
  __syncthreads();
}

// r of token t.
template <int DT>
__device__ __forceinline__ double residual(const Args& a, const Chosen& s, const uint8_t* p, const uint8_t* q,
                                           uint32_t t, double c, const double (&table)[kTable]) {
  if (t >= a.V) return 0.0;
  const double w = weight(logit<DT>(p, t), s.rp, c, table) * s.inv_p;
  if (s.q == kQNone) return w;
  const double o = s.q == kQDraft ? weight(logit<DT>(q, t), s.rq, c, table) * s.inv_q : (uint32_t)s.q == t ? 1.0 : 0.0;
  return w > o ? w - o : 0.0;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sums_kernel(Args a) {
  __shared__ Shared sh;
  const uint32_t chunk = blockIdx.x % a.chunks, b = blockIdx.x / a.chunks;
  const double c = units_of(a, b);
  if (c < 0.0 && chunk != 0u) return;
  fill_table(sh.table);
  join_rows(a, sh, b, c);
  decide<DT>(a, sh, b, c, chunk == 0u);
  const Chosen s = sh.chosen;
  if (s.q == kNoDraw) return;
  const uint8_t* p = row_at<DT>(a, b, s.row);
  const uint8_t* q = s.q == kQDraft ? row_at<DT>(a, b, a.G + 1u + s.row) : nullptr;
  double sum = 0.0;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r)
    sum += residual<DT>(a, s, p, q, chunk * kChunk + r * kThreads + threadIdx.x, c, sh.table);
  sum = wave_sum(sum);
  if ((threadIdx.x & 63u) == 0u) sh.part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0u) a.sums[(size_t)b * a.chunks + chunk] = (sh.part[0] + sh.part[1]) + (sh.part[2] + sh.part[3]);
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

// The token of chunk `chunk` at which the sum (`before` it) first passes `border`; the
// last that has any weight, if rounding leaves none; -1 if none has.
template <int DT>
__device__ __forceinline__ int32_t pick(const Args& a, Shared& sh, const Chosen& s, const uint8_t* p, const uint8_t* q,
                                        uint32_t chunk, double before, double border, double c) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, t0 = chunk * kChunk + threadIdx.x;
  double w[kRounds];
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) w[r] = residual<DT>(a, s, p, q, t0 + r * kThreads, c, sh.table);
  if (threadIdx.x == 0u) sh.found = 0u;
#pragma unroll
  for (uint32_t r = 0; r < kRounds; ++r) {
    const double sum = wave_sum(w[r]);
    if (lane == 0u) sh.part[r * kWaves + wave] = sum;
  }
  __syncthreads();
  static_assert(kRounds * kWaves == 64u, "a lane of the scan for each segment");
  const double upto = before + scan(sh.part[lane], lane);  // every wave alike
  const uint64_t some = __ballot(sh.part[lane] > 0.0), past = __ballot(upto > border) & some;
  if (some == 0ull) return -1;
  const uint32_t seg = past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(some);
  const double start = __shfl(upto - sh.part[lane], (int)seg);
  if (seg % kWaves == wave) {
    double mine = 0.0;
#pragma unroll
    for (uint32_t r = 0; r < kRounds; ++r) mine = seg / kWaves == r ? w[r] : mine;
    const double at = start + scan(mine, lane);
    const uint64_t hit = __ballot(at > border && mine > 0.0), any = __ballot(mine > 0.0);
    const uint32_t l = hit ? (uint32_t)__builtin_ctzll(hit) : any ? 63u - (uint32_t)__builtin_clzll(any) : 0u;
    if (lane == 0u) sh.found = chunk * kChunk + seg * 64u + l;
  }
  __syncthreads();
  return (int32_t)sh.found;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void pick_kernel(Args a) {
  __shared__ Shared sh;
  const uint32_t b = blockIdx.x, lane = threadIdx.x & 63u;
  const double c = units_of(a, b);
  Chosen s = a.chosen[b];
  if (s.q == kNoDraw) return;
  fill_table(sh.table);
  const uint8_t* p = row_at<DT>(a, b, s.row);
  const uint8_t* q = s.q == kQDraft ? row_at<DT>(a, b, a.G + 1u + s.row) : nullptr;
  const double* sums = a.sums + (size_t)b * a.chunks;
  double total = 0.0;
  for (uint32_t i = 0; i < a.chunks; i += 64u) total += wave_sum(i + lane < a.chunks ? sums[i + lane] : 0.0);
  const double border = (double)a.v.u[(size_t)b * (a.G + 1u) + a.G] * total;
  // The chunk that passes the border; the last with any weight, if none does.
  uint32_t chunk = 0u;
  double before = 0.0, chunk_before = 0.0;
  bool found = false;
  for (uint32_t i = 0; i < a.chunks && !found; i += 64u) {
    const double mine = i + lane < a.chunks ? sums[i + lane] : 0.0, upto = before + scan(mine, lane);
    const uint64_t some = __ballot(mine > 0.0), past = __ballot(upto > border) & some;
    if (some) {
      const uint32_t l = past ? (uint32_t)__builtin_ctzll(past) : 63u - (uint32_t)__builtin_clzll(some);
      chunk = i + l;
      chunk_before = __shfl(upto - mine, (int)l);
      found = past != 0ull;
    }
    before = __shfl(upto, 63);
  }
  int32_t token = -1;
  if (total > 0.0) {
    token = pick<DT>(a, sh, s, p, q, chunk, chunk_before, border, c);
  } else {
    // p and q alike to the last bit: nothing is left over, and p itself is drawn from.
    s.q = kQNone;
    const double u = (double)a.v.u[(size_t)b * (a.G + 1u) + a.G];
    double upto = 0.0;
    for (uint32_t i = 0; i < a.chunks; ++i) {
      double sum = 0.0;
#pragma unroll
      for (uint32_t r = 0; r < kRounds; ++r)
        sum += residual<DT>(a, s, p, q, i * kChunk + r * kThreads + threadIdx.x, c, sh.table);
      sum = wave_sum(sum);
      __syncthreads();
      if (lane == 0u) sh.part[threadIdx.x >> 6] = sum;
      __syncthreads();
      sum = (sh.part[0] + sh.part[1]) + (sh.part[2] + sh.part[3]);
      __syncthreads();
      const bool last = upto + sum > u;
      if (sum > 0.0 && (last || i + 1u == a.chunks)) {
        token = pick<DT>(a, sh, s, p, q, i, upto, u, c);
        break;
      }
      upto += sum;
    }
  }
  if (threadIdx.x == 0u) a.v.out[(size_t)b * (a.G + 1u) + s.row] = token;
}

// Splits of a row: enough workgroups for the chip, each with 4096 logits or more.
uint32_t splits_of(int64_t B, int64_t rows, int64_t V) {
  const int64_t n = B * rows, wanted = (2048 + n - 1) / n, most = std::max<int64_t>(V / 4096, 1);
  return (uint32_t)std::min<int64_t>({wanted, most, kMaxSplits});
}
uint32_t chunks_of(int64_t V) { return (uint32_t)((V + kChunk - 1) / kChunk); }

template <int DT>
hipError_t launch(const Args& a, hipStream_t stream) {
  stats_kernel<DT><<<dim3(a.B * a.rows * a.splits), dim3(kThreads), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sums_kernel<DT><<<dim3(a.B * a.chunks), dim3(kThreads), 0, stream>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  pick_kernel<DT><<<dim3(a.B), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// For a call with draft logits; one without needs less.
size_t verify_workspace(int64_t B, int64_t G, int64_t V) {
  const int64_t with = B * (2 * G + 1) * splits_of(B, 2 * G + 1, V), without = B * (G + 1) * splits_of(B, G + 1, V);
  return (size_t)std::max(with, without) * sizeof(Part) + (size_t)B * chunks_of(V) * 8u + (size_t)B * sizeof(Chosen);
}

hipError_t launch_verify(const Verify& v, hipStream_t stream) {
  Args a{};
  a.v = v;
  a.B = (uint32_t)v.B;
  a.G = (uint32_t)v.G;
  a.V = (uint32_t)v.V;
  a.rows = (uint32_t)(v.draft ? 2 * v.G + 1 : v.G + 1);
  a.splits = splits_of(v.B, a.rows, v.V);
  a.chunks = chunks_of(v.V);
  a.chosen = static_cast<Chosen*>(v.workspace);
  a.sums = reinterpret_cast<double*>(a.chosen + a.B);
  a.parts = reinterpret_cast<Part*>(a.sums + (size_t)a.B * a.chunks);
  return v.dtype == kDtF32 ? launch<kDtF32>(a, stream) : launch<kDtBF16>(a, stream);
}

}  // namespace fp4
