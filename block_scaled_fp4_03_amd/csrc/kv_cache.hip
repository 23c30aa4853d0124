// kv_cache.hip -- the paged key-value cache: writing new keys and values into
// it in its row format, and evicting tokens by accumulated attention weight.
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"

namespace fp4 {
namespace {

// ---------------------------------------------------------------------------
// Append.  One thread per 8 values of a new key row and the same 8 of the
// value row; in the MX formats the four threads of a 32-value block share its
// maximum by DPP (blocks never straddle a wave: a row is a multiple of 64
// values).
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void load8(const void* x, size_t i, float (&v)[8]) {
  if (DT == kDtF32) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + i);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = u2f(a[k]);
      v[4 + k] = u2f(b[k]);
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = u2f(a[k] << 16);
      v[2 * k + 1] = u2f(a[k] & 0xFFFF0000u);
    }
  }
}

// The 8 values of `v` as elements d0 .. d0 + 7 of cache row `row`.  Every
// lane of the wavefront takes part (the block maximum); `valid` writes.
template <int FMT>
__device__ __forceinline__ void store8(void* pool, uint8_t* scales, uint64_t row, uint32_t D, uint32_t d0,
                                       const float (&v)[8], bool valid) {
  if (FMT == kKvBf16) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
    if (valid) *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(pool) + (row * D + d0) * 2u) = w;
    return;
  }
  float am = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) am = fmaxf(am, fabsf(v[k]));
  am = fmaxf(am, lane_xor1(am));
  am = fmaxf(am, lane_xor2(am));
  const uint32_t byte = FMT == kKvMx8 ? mx8_scale_byte<kFmtMX8>(am) : mx_scale_byte<kFmtMX>(am);
  const float inv = u2f((254u - byte) << 23);  // 2^(127 - byte), exact
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = v[k] * inv;
  if (!valid) return;
  if (FMT == kKvMx8) {
    u32x2 w;
    w[0] = e4m3x4_sat(y[0], y[1], y[2], y[3]);
    w[1] = e4m3x4_sat(y[4], y[5], y[6], y[7]);
    *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(pool) + row * D + d0) = w;
  } else {
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pool) + (row * D + d0) / 2u) = pack8(y);
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
  const uint32_t i = (in ? at : 0u) / per_row, e = ((in ? at : 0u) % per_row) * 8u;
  const uint32_t D = (uint32_t)c.head_dim, h = e / D, d0 = e % D;
  float a[8], b[8];
  load8<DT>(k, (size_t)i * (size_t)k_stride + e, a);
  load8<DT>(v, (size_t)i * (size_t)v_stride + e, b);
  const int32_t s = seq[i], t = pos[i];
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)c.page_size);
  bool ok = in && s >= 0 && s < seqs && t >= 0 && (int64_t)(t >> shift) < width;
  const int32_t page = ok ? table[(size_t)s * (size_t)width + (uint32_t)(t >> shift)] : -1;
  ok = ok && page >= 0 && page < c.pages;
  const uint64_t row =
      ok ? (((uint64_t)(uint32_t)page * (uint32_t)c.kv_heads + h) << shift) + ((uint32_t)t & (c.page_size - 1u)) : 0u;
  store8<FMT>(c.k, c.ks, row, D, d0, a, ok);
  store8<FMT>(c.v, c.vs, row, D, d0, b, ok);
}

template <int FMT>
hipError_t append_fmt(const KvPool& c, const void* k, const void* v, int in_dtype, int64_t k_stride, int64_t v_stride,
                      const int32_t* table, int64_t width, int64_t seqs, const int32_t* seq, const int32_t* pos,
                      int64_t rows, hipStream_t stream) {
  const uint32_t per_row = (uint32_t)(c.kv_heads * c.head_dim / 8);
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
// Eviction, in two launches: which tokens stay (one workgroup per sequence
// and head), then their rows' copies (spread over the chip).
//
// Which: with R = min(recent, budget) tokens kept for being last, the others'
// weights become 32-bit keys in the weights' order, and a radix selection
// finds the key T of the (budget - R)-th largest and how many equal to T still
// belong.  Its first digit is the top 11 bits of the keys' actual range
// (smallest to largest), so that the LDS histogram's counts spread however
// narrow the weights lie.  The bin then in question mostly holds few keys,
// which are ranked directly; else more digits narrow it (three in all at
// most).  32768 keys (32 a thread) stay in registers from digit to digit;
// longer sequences are read again.  Then the kept tokens are counted per 64
// (ballots), the counts scanned once, and numbers and weights written in
// order.
// ---------------------------------------------------------------------------
constexpr uint32_t kSelThreads = 1024, kSelWaves = kSelThreads / 64, kPer = 32, kChunk = kSelThreads * kPer;
constexpr uint32_t kDigit = 11, kBins = 1u << kDigit;
constexpr uint32_t kFew = 256;  // keys ranked directly
static_assert(kBins == 2 * kSelThreads, "two bins a thread");

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = f2u(w + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The weight of a key (-0 as +0).
__device__ __forceinline__ float key_weight(uint32_t k) {
  return k == 0xFFFFFFFFu ? NAN : u2f((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Sum of v over the threads before this one; `all`: over all of them.
__device__ __forceinline__ uint32_t scan_before(uint32_t v, uint32_t* wave_sum, uint32_t& all) {
  const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= (uint32_t)d) s += o;
  }
  __syncthreads();  // wave_sum may still be read from the last scan
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

// (One workgroup of 16 waves fills a CU: four waves a SIMD may use 128 registers each.)
__global__ __launch_bounds__(kSelThreads) __attribute__((amdgpu_waves_per_eu(4, 4))) void evict_select_kernel(
    const int32_t* __restrict__ lens, const float* __restrict__ weights, int64_t weights_stride,
    int32_t* __restrict__ out_lens, float* __restrict__ out_weights, int64_t out_stride, int32_t* __restrict__ kept,
    uint32_t heads, int64_t max_len, int64_t budget, int64_t recent) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wave_sum[kSelWaves];
  __shared__ uint32_t pick[3], few;
  __shared__ uint32_t count[kPer * kSelWaves];
  const uint32_t h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const size_t bh = (size_t)b * heads + h;
  const float* w = weights + bh * (size_t)weights_stride;
  float* ow = out_weights + bh * (size_t)out_stride;
  int32_t* kp = kept + bh * (size_t)budget;
  const int64_t len64 = lens[b] < 0 ? 0 : (lens[b] < max_len ? lens[b] : max_len);
  const uint32_t n = (uint32_t)len64, keep = (uint32_t)(len64 < budget ? len64 : budget);
  if (h == 0u && tid == 0u) out_lens[b] = (int32_t)keep;
  for (uint32_t t = keep + tid; t < (uint32_t)budget; t += kSelThreads) kp[t] = -1;
  for (uint32_t t = keep + tid; t < (uint32_t)out_stride; t += kSelThreads) ow[t] = 0.0f;
  if (n <= keep) {
    for (uint32_t t = tid; t < n; t += kSelThreads) {
      kp[t] = (int32_t)t;
      ow[t] = w[t];
    }
    return;
  }
  const uint32_t last = (uint32_t)(recent < (int64_t)keep ? recent : (int64_t)keep);
  const uint32_t cand = n - last;  // >= 1: n > keep >= last
  uint32_t rem = keep - last;      // of the candidates
  const uint32_t chunks = (n + kChunk - 1u) / kChunk;

  uint32_t key[kPer];
  // Key i of chunk c: token c kChunk + i kSelThreads + tid (past the end: the last one's).
  const auto load = [&](uint32_t c) {
    // Eight loads at a time without a branch between them, so that they are
    // all on their way together.
    float x[kPer] = {};
#pragma unroll
    for (uint32_t i0 = 0; i0 < kPer; i0 += 8u)
      if (c * kChunk + i0 * kSelThreads < n) {
#pragma unroll
        for (uint32_t i = i0; i < i0 + 8u; ++i) x[i] = w[min(c * kChunk + i * kSelThreads + tid, n - 1u)];
      }
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i)
      if (c * kChunk + i * kSelThreads < n) key[i] = weight_key(x[i]);
  };
  load(0u);

  uint32_t T = 0xFFFFFFFFu, equal = 0u;  // rem == 0: no key is above T, and none equal is taken
  if (rem > 0u) {
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    for (uint32_t c = 0; c < chunks; ++c) {
      if (chunks > 1u) load(c);
#pragma unroll
      for (uint32_t i = 0; i < kPer; ++i)
        if (c * kChunk + i * kSelThreads < cand) {
          const bool is = c * kChunk + i * kSelThreads + tid < cand;
          lo = min(lo, is ? key[i] : 0xFFFFFFFFu);
          hi = max(hi, is ? key[i] : 0u);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      lo = min(lo, (uint32_t)__shfl_xor(lo, d));
      hi = max(hi, (uint32_t)__shfl_xor(hi, d));
    }
    if (lane == 0u) {
      hist[wave] = lo;
      hist[kSelWaves + wave] = hi;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kSelWaves; ++i) {
      lo = min(lo, hist[i]);
      hi = max(hi, hist[kSelWaves + i]);
    }
    __syncthreads();
    T = lo;
    equal = cand;
    uint32_t bits = hi == lo ? 0u : 32u - (uint32_t)__builtin_clz(hi - lo);  // keys of interest: T .. T + 2^bits - 1
    while (bits > 0u) {
      const uint32_t shift = bits > kDigit ? bits - kDigit : 0u, bins = 1u << (bits - shift);
      hist[tid] = 0u;
      hist[kSelThreads + tid] = 0u;
      if (tid == 0u) few = 0u;
      __syncthreads();
      for (uint32_t c = 0; c < chunks; ++c) {
        if (chunks > 1u) load(c);
#pragma unroll
        for (uint32_t i = 0; i < kPer; ++i) {
          if (c * kChunk + i * kSelThreads >= cand) continue;  // (uniform: short sequences skip what they lack)
          const uint32_t t = c * kChunk + i * kSelThreads + tid;
          const uint32_t bin = (key[i] - T) >> shift;
          if (t < cand && key[i] >= T && bin < bins) atomicAdd(&hist[bin], 1u);
        }
      }
      __syncthreads();
      // Two bins a thread, the highest first: where the count from the top passes rem.
      const uint32_t d1 = kBins - 1u - 2u * tid, d0 = d1 - 1u, n1 = hist[d1], n0 = hist[d0];
      uint32_t all;
      const uint32_t above = scan_before(n1 + n0, wave_sum, all);
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
      if (bits == 0u || equal > kFew) continue;
      // Few keys left: collected, and each counts those above it.
      for (uint32_t c = 0; c < chunks; ++c) {
        if (chunks > 1u) load(c);
#pragma unroll
        for (uint32_t i = 0; i < kPer; ++i) {
          if (c * kChunk + i * kSelThreads >= cand) continue;
          const uint32_t t = c * kChunk + i * kSelThreads + tid;
          if (t < cand && key[i] >= T && (key[i] - T) >> bits == 0u) hist[atomicAdd(&few, 1u)] = key[i];
        }
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

  // Tokens in order: key > T, or one of the first `rem` equal to T, or last.
  const bool all_equal = rem == equal;  // no tie to break (and rem == 0 takes none)
  uint32_t base = 0u, eq_base = 0u;
  for (uint32_t c = 0; c < chunks; ++c) {
    if (chunks > 1u) load(c);
    const uint32_t counts = min((n - c * kChunk + kSelThreads - 1u) / kSelThreads, kPer) * kSelWaves;
    uint32_t flags = 0u;  // bit i: token i stays
    uint32_t eq = 0u;     // bit i: equal to T
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) {
      if (c * kChunk + i * kSelThreads >= n) continue;
      const uint32_t t = c * kChunk + i * kSelThreads + tid;
      if (t < n && (t >= cand || key[i] > T)) flags |= 1u << i;
      if (t < cand && key[i] == T) eq |= 1u << i;
    }
    const uint64_t below = (1ull << lane) - 1ull;
    uint32_t all;
    if (all_equal) {
      if (rem > 0u) flags |= eq;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < kPer; ++i) {
        if (c * kChunk + i * kSelThreads >= n) continue;
        const uint64_t m = __ballot((eq >> i) & 1u);
        if (lane == 0u) count[i * kSelWaves + wave] = (uint32_t)__popcll(m);
      }
      __syncthreads();
      const uint32_t mine = tid < counts ? count[tid] : 0u;
      const uint32_t at = scan_before(mine, wave_sum, all);
      if (tid < counts) count[tid] = eq_base + at;
      __syncthreads();
#pragma unroll
      for (uint32_t i = 0; i < kPer; ++i) {
        if (c * kChunk + i * kSelThreads >= n) continue;
        const uint64_t m = __ballot((eq >> i) & 1u);
        if (((eq >> i) & 1u) && count[i * kSelWaves + wave] + (uint32_t)__popcll(m & below) < rem) flags |= 1u << i;
      }
      eq_base += all;
      __syncthreads();
    }
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) {
      if (c * kChunk + i * kSelThreads >= n) continue;
      const uint64_t m = __ballot((flags >> i) & 1u);
      if (lane == 0u) count[i * kSelWaves + wave] = (uint32_t)__popcll(m);
    }
    __syncthreads();
    const uint32_t mine = tid < counts ? count[tid] : 0u;
    const uint32_t at0 = scan_before(mine, wave_sum, all);
    if (tid < counts) count[tid] = base + at0;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) {
      if (c * kChunk + i * kSelThreads >= n) continue;
      const uint64_t m = __ballot((flags >> i) & 1u);
      const uint32_t at = count[i * kSelWaves + wave] + (uint32_t)__popcll(m & below);
      if (((flags >> i) & 1u) && at < keep) {
        const uint32_t t = c * kChunk + i * kSelThreads + tid;
        kp[at] = (int32_t)t;
        ow[at] = key_weight(key[i]);
      }
    }
    base += all;
    __syncthreads();
  }
}

// Rows of the kept tokens to their new places: 16 bytes a thread, the K row
// and the V row of one token; the scale bytes by the row's first threads.
__global__ __launch_bounds__(256) void evict_copy_kernel(KvPool src, const int32_t* __restrict__ src_table,
                                                         int64_t src_width, KvPool dst,
                                                         const int32_t* __restrict__ dst_table, int64_t dst_width,
                                                         const int32_t* __restrict__ kept, int64_t budget,
                                                         uint32_t pieces, uint32_t row_bytes) {
  const uint32_t h = blockIdx.y, b = blockIdx.z;
  const uint32_t at = blockIdx.x * (256u / pieces) + threadIdx.x / pieces, piece = threadIdx.x % pieces;
  if (at >= (uint32_t)budget || threadIdx.x >= 256u / pieces * pieces) return;
  const int32_t t = kept[((size_t)b * src.kv_heads + h) * (size_t)budget + at];
  if (t < 0) return;
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)src.page_size), in_page = (uint32_t)src.page_size - 1u;
  const int32_t sp = src_table[(size_t)b * src_width + ((uint32_t)t >> shift)];
  const int32_t dp = dst_table[(size_t)b * dst_width + (at >> shift)];
  if (sp < 0 || sp >= src.pages || dp < 0 || dp >= dst.pages) return;
  const uint64_t from = (((uint64_t)(uint32_t)sp * src.kv_heads + h) << shift) + ((uint32_t)t & in_page);
  const uint64_t to = (((uint64_t)(uint32_t)dp * dst.kv_heads + h) << shift) + (at & in_page);
  const u32x4 k = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(src.k) + from * row_bytes + piece * 16u);
  const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(src.v) + from * row_bytes + piece * 16u);
  *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(dst.k) + to * row_bytes + piece * 16u) = k;
  *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(dst.v) + to * row_bytes + piece * 16u) = v;
  if (src.fmt != kKvBf16) {
    const uint32_t pairs = (uint32_t)src.head_dim / 64u;  // scale bytes two by two
    for (uint32_t i = piece; i < pairs; i += pieces) {
      reinterpret_cast<uint16_t*>(dst.ks)[to * pairs + i] = reinterpret_cast<const uint16_t*>(src.ks)[from * pairs + i];
      reinterpret_cast<uint16_t*>(dst.vs)[to * pairs + i] = reinterpret_cast<const uint16_t*>(src.vs)[from * pairs + i];
    }
  }
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
  evict_select_kernel<<<dim3((uint32_t)src.kv_heads, (uint32_t)B), kSelThreads, 0, stream>>>(
      lens, weights, weights_stride, out_lens, out_weights, out_stride, kept, (uint32_t)src.kv_heads, max_len, budget,
      recent);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || budget == 0 || max_len == 0) return e;
  const uint32_t row_bytes = kv_row_bytes(src.fmt, (uint32_t)src.head_dim), pieces = row_bytes / 16u;
  const uint32_t rows = 256u / pieces;
  evict_copy_kernel<<<dim3((uint32_t)((budget + rows - 1) / rows), (uint32_t)src.kv_heads, (uint32_t)B), 256, 0,
                      stream>>>(src, src_table, src_width, dst, dst_table, dst_width, kept, budget, pieces, row_bytes);
  return hipGetLastError();
}

}  // namespace fp4
