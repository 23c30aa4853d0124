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
// (four 8-bit digits, high to low, LDS histograms) finds the key T of the
// (budget - R)-th largest and how many equal to T still belong.  One more
// pass in token order writes the kept tokens' numbers and weights.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;

__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = f2u(w + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ __launch_bounds__(kSelThreads) void evict_select_kernel(
    const int32_t* __restrict__ lens, const float* __restrict__ weights, int64_t weights_stride,
    int32_t* __restrict__ out_lens, float* __restrict__ out_weights, int64_t out_stride, int32_t* __restrict__ kept,
    uint32_t heads, int64_t max_len, int64_t budget, int64_t recent) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];
  __shared__ uint32_t count[2][kSelWaves];
  const uint32_t h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  const size_t bh = (size_t)b * heads + h;
  const float* w = weights + bh * (size_t)weights_stride;
  float* ow = out_weights + bh * (size_t)out_stride;
  int32_t* kp = kept + bh * (size_t)budget;
  const int64_t len64 = lens[b] < 0 ? 0 : (lens[b] < max_len ? lens[b] : max_len);
  const uint32_t n = (uint32_t)len64, keep = (uint32_t)(len64 < budget ? len64 : budget);
  if (h == 0u && tid == 0u) out_lens[b] = (int32_t)keep;
  if (n <= keep) {
    for (uint32_t t = tid; t < n; t += kSelThreads) {
      kp[t] = (int32_t)t;
      ow[t] = w[t];
    }
  } else {
    const uint32_t last = (uint32_t)(recent < (int64_t)keep ? recent : (int64_t)keep);
    const uint32_t cand = n - last;
    uint32_t rem = keep - last, prefix = 0u, mask = 0u;
    if (rem == 0u) prefix = 0xFFFFFFFFu;  // nothing beyond the last tokens
    for (int shift = 24; shift >= 0 && rem > 0u; shift -= 8) {
      if (tid < 256u) hist[tid] = 0u;
      __syncthreads();
      for (uint32_t t = tid; t < cand; t += kSelThreads) {
        const uint32_t key = weight_key(w[t]);
        if (((key ^ prefix) & mask) == 0u) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid < 256u) {
        uint32_t above = 0u;
        for (uint32_t d = tid + 1u; d < 256u; ++d) above += hist[d];
        if (above < rem && rem <= above + hist[tid]) {
          pick[0] = tid;
          pick[1] = rem - above;
        }
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= 255u << shift;
      rem = pick[1];
      __syncthreads();
    }
    // Tokens in order: key > T, or one of the first `rem` equal to T, or last.
    uint32_t base = 0u, eq_base = 0u;
    for (uint32_t t0 = 0u; t0 < n; t0 += kSelThreads) {
      const uint32_t t = t0 + tid;
      const uint32_t key = t < cand ? weight_key(w[t]) : 0u;
      const bool eq = t < cand && key == prefix;
      const uint64_t eqs = __ballot(eq), below = (1ull << lane) - 1ull;
      if (lane == 0u) count[0][wave] = (uint32_t)__popcll(eqs);
      __syncthreads();
      uint32_t eq_before = eq_base, eq_all = 0u;
      for (uint32_t i = 0u; i < kSelWaves; ++i) {
        if (i < wave) eq_before += count[0][i];
        eq_all += count[0][i];
      }
      const bool stays =
          t < n && (t >= cand || key > prefix || (eq && eq_before + (uint32_t)__popcll(eqs & below) < rem));
      const uint64_t st = __ballot(stays);
      if (lane == 0u) count[1][wave] = (uint32_t)__popcll(st);
      __syncthreads();
      uint32_t at = base, all = 0u;
      for (uint32_t i = 0u; i < kSelWaves; ++i) {
        if (i < wave) at += count[1][i];
        all += count[1][i];
      }
      at += (uint32_t)__popcll(st & below);
      if (stays && at < keep) {
        kp[at] = (int32_t)t;
        ow[at] = w[t];
      }
      base += all;
      eq_base += eq_all;
      __syncthreads();
    }
  }
  for (uint32_t t = keep + tid; t < (uint32_t)budget; t += kSelThreads) kp[t] = -1;
  for (uint32_t t = keep + tid; t < (uint32_t)out_stride; t += kSelThreads) ow[t] = 0.0f;
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
    const uint32_t blocks = (uint32_t)src.head_dim / 32u;
    for (uint32_t i = piece; i < blocks; i += pieces) {
      dst.ks[to * blocks + i] = src.ks[from * blocks + i];
      dst.vs[to * blocks + i] = src.vs[from * blocks + i];
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
