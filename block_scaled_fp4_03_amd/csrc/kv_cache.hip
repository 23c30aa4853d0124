// kv_cache.hip -- the paged key-value cache: writing new keys and values into
// it in its row format, and evicting tokens by accumulated attention weight.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"

namespace fp4 {
namespace {

// ---------------------------------------------------------------------------
// Append.  One thread per 16 values of a new key row and the same 16 of the
// value row; in the MX formats the two threads of a 32-value block share its
// maximum by DPP (blocks never straddle a wave: a row is a multiple of 64
// values).  Bound by the bytes: 16384 rows of 8 x 128 to MXFP8 take 18.0 us
// (5.7 TB/s); with 8 values a thread 20.4, and with stores not marked as
// streaming 20.9 (loads marked so made it slower).
// ---------------------------------------------------------------------------
constexpr uint32_t kPiece = 16;  // values of a thread
template <int DT>
__device__ __forceinline__ void load_piece(const void* x, size_t i, float (&v)[kPiece]) {
  if (DT == kDtF32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + i);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 a = p[q];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[4 * q + k] = u2f(a[k]);
    }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const u32x4 a = p[q];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[8 * q + 2 * k] = u2f(a[k] << 16);
        v[8 * q + 2 * k + 1] = u2f(a[k] & 0xFFFF0000u);
      }
    }
  }
}

// The 16 values of `v` as elements d0 .. d0 + 15 of cache row `row`.  Every
// lane of the wavefront takes part (the block maximum); `valid` writes.
template <int FMT>
__device__ __forceinline__ void store_piece(void* pool, uint8_t* scales, uint64_t row, uint32_t D, uint32_t d0,
                                            const float (&v)[kPiece], bool valid) {
  uint8_t* out = static_cast<uint8_t*>(pool) + row * kv_row_bytes(FMT, D) + kv_row_bytes(FMT, d0);
  if (FMT == kKvBf16) {
    u32x4 w[2];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k / 4][k % 4] = bf16_pair(v[2 * k], v[2 * k + 1]);
    if (valid) {
      __builtin_nontemporal_store(w[0], reinterpret_cast<u32x4*>(out));
      __builtin_nontemporal_store(w[1], reinterpret_cast<u32x4*>(out) + 1);
    }
    return;
  }
  float am = 0.0f;
#pragma unroll
  for (uint32_t k = 0; k < kPiece; ++k) am = fmaxf(am, fabsf(v[k]));
  am = fmaxf(am, lane_xor1(am));
  const uint32_t byte = FMT == kKvMx8 ? mx8_scale_byte<kFmtMX8>(am) : mx_scale_byte<kFmtMX>(am);
  const float inv = u2f((254u - byte) << 23);
  float y[kPiece];
#pragma unroll
  for (uint32_t k = 0; k < kPiece; ++k) y[k] = v[k] * inv;
  if (!valid) return;
  if (FMT == kKvMx8) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = e4m3x4_sat(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(out));
  } else {
    float lo[8], hi[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = y[k];
      hi[k] = y[8 + k];
    }
    __builtin_nontemporal_store(u32x2{pack8(lo), pack8(hi)}, reinterpret_cast<u32x2*>(out));
  }
  if ((d0 & 31u) == 0u) scales[row * (D / 32u) + d0 / 32u] = (uint8_t)byte;
}

template <int FMT, int DT>
__global__ __launch_bounds__(256) void kv_append_kernel(KvPool c, const void* __restrict__ k,
                                                        const void* __restrict__ v, int64_t k_stride,
                                                        int64_t v_stride, const int32_t* __restrict__ table,
                                                        int64_t width, int64_t seqs, const int32_t* __restrict__ seq,
                                                        const int32_t* __restrict__ pos, uint32_t per_row,
                                                        uint32_t total) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const bool in = at < total;
  const uint32_t i = (in ? at : 0u) / per_row, e = ((in ? at : 0u) % per_row) * kPiece;
  const uint32_t D = (uint32_t)c.head_dim, h = e / D, d0 = e % D;
  float a[kPiece], b[kPiece];
  load_piece<DT>(k, (size_t)i * (size_t)k_stride + e, a);
  load_piece<DT>(v, (size_t)i * (size_t)v_stride + e, b);
  const int32_t s = seq[i], t = pos[i];
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)c.page_size);
  bool ok = in && s >= 0 && s < seqs && t >= 0 && (int64_t)(t >> shift) < width;
  const int32_t page = ok ? table[(size_t)s * (size_t)width + (uint32_t)(t >> shift)] : -1;
  ok = ok && page >= 0 && page < c.pages;
  const uint64_t row =
      ok ? (((uint64_t)(uint32_t)page * (uint32_t)c.kv_heads + h) << shift) + ((uint32_t)t & (c.page_size - 1u)) : 0u;
  store_piece<FMT>(c.k, c.ks, row, D, d0, a, ok);
  store_piece<FMT>(c.v, c.vs, row, D, d0, b, ok);
}

template <int FMT>
hipError_t append_fmt(const KvPool& c, const void* k, const void* v, int in_dtype, int64_t k_stride, int64_t v_stride,
                      const int32_t* table, int64_t width, int64_t seqs, const int32_t* seq, const int32_t* pos,
                      int64_t rows, hipStream_t stream) {
  const uint32_t per_row = (uint32_t)(c.kv_heads * c.head_dim / (int)kPiece);
  const uint32_t total = (uint32_t)(rows * per_row), grid = (total + 255u) / 256u;
  if (in_dtype == kDtF32)
    kv_append_kernel<FMT, kDtF32><<<grid, 256, 0, stream>>>(c, k, v, k_stride, v_stride, table, width, seqs, seq, pos,
                                                           per_row, total);
  else
    kv_append_kernel<FMT, kDtBF16><<<grid, 256, 0, stream>>>(c, k, v, k_stride, v_stride, table, width, seqs, seq,
                                                            pos, per_row, total);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Eviction: which tokens stay, then their rows' copies.  One launch for
// sequences of up to 32768 tokens: the selection is short next to the copies,
// but one workgroup per (sequence, head) would leave most of the chip idle,
// so `parts` workgroups each make the whole selection (from L2) and write and
// copy their share of the kept tokens.  Longer sequences, whose selection
// reads the weights several times, take a launch for it and one for the
// copies.  (Two launches for all took 14.7 + 4.7 us for 16 heads of 1100 tokens,
// one takes 12.5 us.)  Bound by the copies and, in short sequences, by the
// selection's passes one after the other: 16 x 8 heads of 32768 tokens cut to
// 4096 MXFP8 take 81 us, about 22 of them before the copies begin, which then
// run at 5.6 TB/s.
//
// Which: with R = min(recent, budget) tokens kept for being last, the others'
// weights become 32-bit keys in the weights' order, and a radix selection
// finds the key T of the (budget - R)-th largest and how many equal to T still
// belong.  Its first digit is the top 11 bits of the keys' actual range
// (smallest to largest), so that the LDS histogram's counts spread however
// narrow the weights lie.  The bin then in question mostly holds few keys,
// which are ranked directly; else more digits narrow it (three in all at
// most).  32768 keys stay in LDS from pass to pass; longer sequences are read
// again.  For the output every thread takes a run of tokens, so one scan over
// the threads gives all places.  (Keys in registers were slower: every pass
// is then code unrolled 32 times, run once, and fetching it took longer than
// running it: a selection of 1100 tokens took 14.8 us against 7.7 us.)
// ---------------------------------------------------------------------------
constexpr uint32_t kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr uint32_t kChunk = 32768;  // keys held at a time
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit;
constexpr uint32_t kFew = 256;  // keys ranked directly
static_assert(kBins == 2 * kSelThreads, "two bins a thread");
static_assert(kChunk / kSelThreads == 32, "a thread's run fits a 32-bit mask");

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));  // weights' rows have any stride

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = f2u(w + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The weight of a key (-0 as +0).
__device__ __forceinline__ float key_weight(uint32_t k) {
  return k == 0xFFFFFFFFu ? NAN : u2f((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Smallest and largest over the wavefront, in every lane.
template <bool MAX>
__device__ __forceinline__ uint32_t wave_extreme(uint32_t v) {
  const auto pick = [](uint32_t x, uint32_t y) { return MAX ? max(x, y) : min(x, y); };
  v = pick(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x121, 0xF, 0xF, false));
  v = pick(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x122, 0xF, 0xF, false));
  v = pick(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, false));
  v = pick(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false));
  return pick(pick((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
              pick((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// Sum of v over the threads before this one; `all`: over all of them.
// wave_sum is not in use by an earlier scan (a barrier lies between).
__device__ __forceinline__ uint32_t scan_before(uint32_t v, uint32_t* wave_sum, uint32_t& all) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= (uint32_t)d) s += o;
  }
  if (lane == 63u) wave_sum[wave] = s;
  __syncthreads();
  uint32_t before = 0u;
  all = 0u;
#pragma unroll
  for (uint32_t i = 0; i < kSelWaves; ++i) {
    const uint32_t x = wave_sum[i];
    before += i < wave ? x : 0u;
    all += x;
  }
  return before + s - v;
}

struct EvictArgs {
  KvPool src;
  const int32_t* src_table;
  int64_t src_width;
  const int32_t* lens;
  const float* weights;
  int64_t weights_stride;
  KvPool dst;
  const int32_t* dst_table;
  int64_t dst_width;
  int32_t* out_lens;
  float* out_weights;
  int64_t out_stride;
  int32_t* kept;
  int64_t max_len, budget, recent;
  uint32_t row_bytes;
};

// Copies the rows of kept tokens [from, to) of sequence b, head h to their
// places: 16 bytes a thread, K and V of kRows tokens at a time in flight,
// loads and stores marked as used once (16 x 8 heads of 4096 MXFP8 tokens: 97
// us without, 81 us with).
template <uint32_t THREADS>
__device__ __forceinline__ void copy_rows(const EvictArgs& a, uint32_t b, uint32_t h, uint32_t from, uint32_t to) {
  constexpr uint32_t kRows = 4;
  const uint32_t pieces = a.row_bytes / 16u, step = THREADS / pieces;  // threads of a row; rows of a step
  const uint32_t r = threadIdx.x / pieces, piece = threadIdx.x % pieces;
  if (r >= step) return;
  const int32_t* kept = a.kept + ((size_t)b * a.src.kv_heads + h) * (size_t)a.budget;
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)a.src.page_size), in_page = (uint32_t)a.src.page_size - 1u;
  const uint32_t pairs = (uint32_t)a.src.head_dim / 64u;  // scale bytes two by two
  for (uint32_t at0 = from + r; at0 < to; at0 += kRows * step) {
    uint64_t s[kRows], d[kRows];
    bool ok[kRows];
#pragma unroll
    for (uint32_t k = 0; k < kRows; ++k) {
      const uint32_t at = min(at0 + k * step, to - 1u);
      const int32_t t = kept[at];
      const int32_t sp = a.src_table[(size_t)b * a.src_width + ((uint32_t)max(t, 0) >> shift)];
      const int32_t dp = a.dst_table[(size_t)b * a.dst_width + (at >> shift)];
      ok[k] = at0 + k * step < to && t >= 0 && sp >= 0 && sp < a.src.pages && dp >= 0 && dp < a.dst.pages;
      s[k] = ok[k] ? (((uint64_t)(uint32_t)sp * a.src.kv_heads + h) << shift) + ((uint32_t)t & in_page) : 0u;
      d[k] = ok[k] ? (((uint64_t)(uint32_t)dp * a.dst.kv_heads + h) << shift) + (at & in_page) : 0u;
    }
    u32x4 x[kRows], y[kRows];
#pragma unroll
    for (uint32_t k = 0; k < kRows; ++k) {
      // (Row 0 stands in for one that is not copied; a pool without pages has none to copy.)
      const uint64_t at = s[k] * a.row_bytes + piece * 16u;
      if (a.src.pages > 0) {
        x[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.src.k) + at));
        y[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.src.v) + at));
      }
    }
#pragma unroll
    for (uint32_t k = 0; k < kRows; ++k) {
      if (!ok[k]) continue;
      const uint64_t at = d[k] * a.row_bytes + piece * 16u;
      __builtin_nontemporal_store(x[k], reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.dst.k) + at));
      __builtin_nontemporal_store(y[k], reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.dst.v) + at));
      if (a.src.fmt != kKvBf16) {
        for (uint32_t i = piece; i < pairs; i += pieces) {
          reinterpret_cast<uint16_t*>(a.dst.ks)[d[k] * pairs + i] =
              reinterpret_cast<const uint16_t*>(a.src.ks)[s[k] * pairs + i];
          reinterpret_cast<uint16_t*>(a.dst.vs)[d[k] * pairs + i] =
              reinterpret_cast<const uint16_t*>(a.src.vs)[s[k] * pairs + i];
        }
      }
    }
  }
}

// Workgroup (part, head, sequence); `copy`: also the rows of its share.
__global__ __launch_bounds__(kSelThreads) __attribute__((amdgpu_waves_per_eu(4, 4))) void evict_kernel(EvictArgs a,
                                                                                                      bool copy) {
  extern __shared__ __attribute__((aligned(16))) uint32_t keys[];  // min(max_len, kChunk) of them, to a multiple of 4
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wave_sum[2][kSelWaves];
  __shared__ uint32_t pick[3], few;
  const uint32_t part = blockIdx.x, parts = gridDim.x, h = blockIdx.y, b = blockIdx.z;
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const size_t bh = (size_t)b * a.src.kv_heads + h;
  const float* __restrict__ w = a.weights + bh * (size_t)a.weights_stride;
  float* ow = a.out_weights + bh * (size_t)a.out_stride;
  int32_t* kp = a.kept + bh * (size_t)a.budget;
  const int64_t l = a.lens[b], len64 = l < 0 ? 0 : (l < a.max_len ? l : a.max_len);
  const uint32_t n = (uint32_t)len64, keep = (uint32_t)(len64 < a.budget ? len64 : a.budget);
  // This workgroup's share of the kept tokens.
  const uint32_t share = (keep + parts - 1u) / parts, from = min(part * share, keep), to = min(from + share, keep);
  if (part == 0u) {
    if (h == 0u && tid == 0u) a.out_lens[b] = (int32_t)keep;
    for (uint32_t t = keep + tid; t < (uint32_t)a.budget; t += kSelThreads) kp[t] = -1;
    for (uint32_t t = keep + tid; t < (uint32_t)a.out_stride; t += kSelThreads) ow[t] = 0.0f;
  }
  if (from >= to) return;
  if (n <= keep) {
    for (uint32_t t = from + tid; t < to; t += kSelThreads) {
      kp[t] = (int32_t)t;
      ow[t] = key_weight(weight_key(w[t]));
    }
    __syncthreads();
    if (copy) copy_rows<kSelThreads>(a, b, h, from, to);
    return;
  }
  const uint32_t last = (uint32_t)(a.recent < (int64_t)keep ? a.recent : (int64_t)keep);
  const uint32_t cand = n - last;  // >= 1: n > keep >= last
  uint32_t rem = keep - last;      // of the candidates
  const uint32_t chunks = (n + kChunk - 1u) / kChunk;

  // The keys of tokens c kChunk .., and their smallest and largest among the candidates.
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  const auto load = [&](uint32_t c) __attribute__((always_inline)) {
    const uint32_t t0 = c * kChunk, here = min(n - t0, kChunk), here4 = here / 4u;
    // 16 bytes a load and eight loads a thread: a whole chunk is on its way at once.
    for (uint32_t i0 = tid; i0 < here4; i0 += 8u * kSelThreads) {
      f32x4_any x[8];
#pragma unroll
      for (uint32_t k = 0; k < 8u; ++k)
        x[k] = *reinterpret_cast<const f32x4_any*>(w + t0 + 4u * min(i0 + k * kSelThreads, here4 - 1u));
#pragma unroll
      for (uint32_t k = 0; k < 8u; ++k) {
        const uint32_t i = i0 + k * kSelThreads;
        if (i < here4) {
          u32x4 q;
#pragma unroll
          for (uint32_t j = 0; j < 4u; ++j) {
            q[j] = weight_key(x[k][j]);
            const bool is = t0 + 4u * i + j < cand;
            lo = min(lo, is ? q[j] : 0xFFFFFFFFu);
            hi = max(hi, is ? q[j] : 0u);
          }
          reinterpret_cast<u32x4*>(keys)[i] = q;
        }
      }
    }
    if (tid < (here & 3u)) {
      const uint32_t i = 4u * here4 + tid, key = weight_key(w[t0 + i]);
      keys[i] = key;
      lo = min(lo, t0 + i < cand ? key : 0xFFFFFFFFu);
      hi = max(hi, t0 + i < cand ? key : 0u);
    }
  };
  // f of every candidate's key in chunk c.
  const auto each = [&](uint32_t c, auto f) __attribute__((always_inline)) {
    const uint32_t here = c * kChunk < cand ? min(cand - c * kChunk, kChunk) : 0u;
#pragma unroll 2
    for (uint32_t i = 4u * tid; i < here; i += 4u * kSelThreads) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(keys + i);  // (the array is a multiple of four long)
#pragma unroll
      for (uint32_t j = 0; j < 4u; ++j)
        if (i + j < here) f(q[j]);
    }
  };
  for (uint32_t c = 0; c < chunks; ++c) {
    if (c > 0u) __syncthreads();
    load(c);
  }
  uint32_t held = chunks - 1u;
  // Chunk c in LDS, for every thread.
  const auto hold = [&](uint32_t c) __attribute__((always_inline)) {
    if (held == c) return;
    __syncthreads();
    load(c);
    held = c;
    __syncthreads();
  };
  hist[tid] = 0u;
  hist[kSelThreads + tid] = 0u;
  if (tid == 0u) few = 0u;
  lo = wave_extreme<false>(lo);
  hi = wave_extreme<true>(hi);
  if (lane == 0u) {
    wave_sum[0][wave] = lo;
    wave_sum[1][wave] = hi;
  }
  __syncthreads();

  uint32_t T = 0xFFFFFFFFu, equal = 0u;  // rem == 0: no key is above T, and none equal is taken
  if (rem > 0u) {
    lo = wave_extreme<false>(wave_sum[0][lane & (kSelWaves - 1u)]);
    hi = wave_extreme<true>(wave_sum[1][lane & (kSelWaves - 1u)]);
    T = lo;
    equal = cand;
    uint32_t bits = hi == lo ? 0u : 32u - (uint32_t)__builtin_clz(hi - lo);  // keys of interest: T .. T + 2^bits - 1
    while (bits > 0u) {
      const uint32_t shift = bits > kDigit ? bits - kDigit : 0u, bins = 1u << (bits - shift);
      for (uint32_t c = 0; c < chunks; ++c) {
        hold(c);
        each(c, [&](uint32_t key) __attribute__((always_inline)) {
          const uint32_t bin = (key - T) >> shift;
          if (key >= T && bin < bins) atomicAdd(&hist[bin], 1u);
        });
      }
      __syncthreads();
      // Two bins a thread, the highest first: where the count from the top passes rem.
      const uint32_t d1 = kBins - 1u - 2u * tid, d0 = d1 - 1u, n1 = hist[d1], n0 = hist[d0];
      uint32_t all;
      const uint32_t above = scan_before(n1 + n0, wave_sum[0], all);
      if (above < rem && rem <= above + n1 + n0) {
        const bool first = rem <= above + n1;
        pick[0] = first ? d1 : d0;
        pick[1] = first ? rem - above : rem - above - n1;
        pick[2] = first ? n1 : n0;
      }
      __syncthreads();
      T += pick[0] << shift;
      rem = pick[1];
      equal = pick[2];
      bits = shift;
      if (bits == 0u) break;
      if (equal > kFew) {
        hist[tid] = 0u;
        hist[kSelThreads + tid] = 0u;
        __syncthreads();
        continue;
      }
      // Few keys left: collected, and each counts those above it.
      for (uint32_t c = 0; c < chunks; ++c) {
        hold(c);
        each(c, [&](uint32_t key) __attribute__((always_inline)) {
          if (key >= T && (key - T) >> bits == 0u) hist[atomicAdd(&few, 1u)] = key;
        });
      }
      __syncthreads();
      if (tid < equal) {
        const uint32_t mine = hist[tid];
        uint32_t above_it = 0u, same = 0u;
#pragma unroll 8
        for (uint32_t i = 0; i < equal; ++i) {
          const uint32_t o = hist[i];
          above_it += o > mine ? 1u : 0u;
          same += o == mine ? 1u : 0u;
        }
        if (above_it < rem && rem <= above_it + same) {  // every key equal to the one wanted writes the same
          pick[0] = mine;
          pick[1] = rem - above_it;
          pick[2] = same;
        }
      }
      __syncthreads();
      T = pick[0];
      rem = pick[1];
      equal = pick[2];
      bits = 0u;
    }
  }

  __syncthreads();  // wave_sum is free

  // Tokens in order: key > T, or one of the first `rem` equal to T, or last.
  // A thread's run has an odd length, or 32 read from another place by each
  // lane, so that the threads' reads of one step fall into different banks.
  uint32_t base = 0u, eq_base = 0u;
  for (uint32_t c = 0; c < chunks; ++c) {
    hold(c);
    const uint32_t t0 = c * kChunk, here = min(n - t0, kChunk), per = (here + kSelThreads - 1u) / kSelThreads;
    const uint32_t run = per == 32u ? 32u : per | 1u, turn = per == 32u ? lane : 0u;
    const uint32_t i0 = min(tid * run, here), i1 = min(i0 + run, here);
    uint32_t stay = 0u, eq = 0u;  // bit i - i0
#pragma unroll 8
    for (uint32_t s = 0; s < run; ++s) {
      const uint32_t i = (s + turn) & 31u, key = keys[min(i0 + i, here - 1u)];
      stay |= (key > T ? 1u : 0u) << i;
      eq |= (key == T ? 1u : 0u) << i;
    }
    // Only what is in the run; the last tokens, no candidates, all stay.
    const auto first = [](uint32_t k) { return k >= 32u ? 0xFFFFFFFFu : (1u << k) - 1u; };
    const uint32_t in = first(i1 - i0), cands = first(t0 + i0 < cand ? cand - (t0 + i0) : 0u);
    stay = in & (stay | ~cands);
    eq &= in & cands;
    uint32_t all, eq_all;
    uint32_t at = base + scan_before((uint32_t)__popc(stay), wave_sum[0], all);
    const uint32_t eq_at = eq_base + scan_before((uint32_t)__popc(eq), wave_sum[1], eq_all);
    // Of the equal ones before this run, the first rem stayed; of its own, as many as are left.
    at += min(eq_at, rem) - min(eq_base, rem);
    for (uint32_t left = rem - min(eq_at, rem); left > 0u && eq != 0u; --left) {
      stay |= eq & -eq;
      eq &= eq - 1u;
    }
    for (; stay != 0u && at < to; stay &= stay - 1u, ++at) {
      const uint32_t i = i0 + (uint32_t)__builtin_ctz(stay);
      if (at < from) continue;
      kp[at] = (int32_t)(t0 + i);
      ow[at] = key_weight(keys[i]);
    }
    base += all + min(eq_base + eq_all, rem) - min(eq_base, rem);
    eq_base += eq_all;
    __syncthreads();  // wave_sum is free again; the share's tokens are written
  }
  if (copy) copy_rows<kSelThreads>(a, b, h, from, to);
}

constexpr uint32_t kCopyThreads = 256, kCopyRows = 64;  // of a workgroup of the copies' own launch
__global__ __launch_bounds__(kCopyThreads) void evict_copy_kernel(EvictArgs a) {
  const int64_t l = a.lens[blockIdx.z], len = l < 0 ? 0 : (l < a.max_len ? l : a.max_len);
  const uint32_t keep = (uint32_t)(len < a.budget ? len : a.budget), from = blockIdx.x * kCopyRows;
  if (from < keep) copy_rows<kCopyThreads>(a, blockIdx.z, blockIdx.y, from, min(from + kCopyRows, keep));
}

}  // namespace

hipError_t launch_kv_append(const KvPool& c, const void* k, const void* v, int in_dtype, int64_t k_stride,
                            int64_t v_stride, const int32_t* table, int64_t width, int64_t seqs, const int32_t* seq,
                            const int32_t* pos, int64_t rows, hipStream_t stream) {
  switch (c.fmt) {
    case kKvBf16:
      return append_fmt<kKvBf16>(c, k, v, in_dtype, k_stride, v_stride, table, width, seqs, seq, pos, rows, stream);
    case kKvMx8:
      return append_fmt<kKvMx8>(c, k, v, in_dtype, k_stride, v_stride, table, width, seqs, seq, pos, rows, stream);
    default:
      return append_fmt<kKvMx4>(c, k, v, in_dtype, k_stride, v_stride, table, width, seqs, seq, pos, rows, stream);
  }
}

size_t kv_evict_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_kv_evict(const KvPool& src, const int32_t* src_table, int64_t src_width, const int32_t* lens,
                           const float* weights, int64_t weights_stride, const KvPool& dst, const int32_t* dst_table,
                           int64_t dst_width, int32_t* out_lens, float* out_weights, int64_t out_stride,
                           int32_t* kept, int64_t B, int64_t max_len, int64_t budget, int64_t recent, void*,
                           hipStream_t stream) {
  const EvictArgs a{src, src_table, src_width, lens, weights, weights_stride, dst, dst_table, dst_width, out_lens,
                    out_weights, out_stride, kept, max_len, budget, recent,
                    kv_row_bytes(src.fmt, (uint32_t)src.head_dim)};
  const uint32_t lds = (uint32_t)(max_len < (int64_t)kChunk ? (max_len + 3) / 4 * 4 : (int64_t)kChunk) * 4u;
  const int64_t heads = B * src.kv_heads, most = budget < max_len ? budget : max_len;
  const bool one = max_len <= (int64_t)kChunk;
  // One launch: parts that bring the workgroups to about one a CU, of at least 16 tokens each.
  int64_t parts = one ? 256 / heads : 1;
  if (parts > (most + 15) / 16) parts = (most + 15) / 16;
  if (parts < 1) parts = 1;
  evict_kernel<<<dim3((uint32_t)parts, (uint32_t)src.kv_heads, (uint32_t)B), kSelThreads, lds, stream>>>(a, one);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || one || most == 0) return e;
  evict_copy_kernel<<<dim3((uint32_t)((most + kCopyRows - 1) / kCopyRows), (uint32_t)src.kv_heads, (uint32_t)B),
                      kCopyThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp4
