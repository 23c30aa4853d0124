// attn_decode.hip -- attention of one new token per sequence over the paged
// key-value cache, split over the cache's length and joined.
//
// For the G query heads of a kv head, s = scale q.K^T, p = softmax(s), o = p V.
// Each K and V row is read once and serves all G heads, so the work is bound
// by the cache's bytes (G FLOP a byte in BF16, 4 G in MXFP4, far below the
// matrix core's rate) as long as decoding, softmax and moving stay cheap:
//
//   - A wave takes 32 tokens at a time.  S^T = K Q^T on the 16x16x32 BF16
//     matrix instruction puts a head in each lane column and tokens in the
//     lanes' registers: a lane (c = lane & 15, g = lane >> 4) gets head c,
//     tokens 4g..4g+3 of each 16-token half.  Those eight probabilities are,
//     as they lie, the B operand of O^T += V^T P^T when the contraction
//     index 8g + j stands for token 4g + j (j < 4) or 16 + 4g + j - 4: no
//     move across lanes between the two products.
//   - V^T's A operand wants eight tokens of one element d per lane.  Lane
//     (c, g) loads, of its eight tokens, elements c D/16 .. of the row (all
//     16 lanes together: whole rows), and pairs of tokens are interleaved by
//     v_perm: one VALU operation per two elements, no LDS.  Output row c of
//     product e then stands for d = c D/16 + e.  (BF16: the chunks its loads
//     bring, as for K.)
//   - K's elements may be contracted in any order too: lane (c, g) holds a
//     quarter of token c's, in the chunks that its loads bring.
//   - MXFP8 / MXFP4 rows are converted to BF16 by the scaling converters
//     (exact: at most 4 significant bits).
//   - The tiles of all (sequence, kv head) units laid end to end are cut into
//     equal shares, one for each of two workgroups a CU, whatever the lengths:
//     a workgroup walks its share, which may end one unit, hold several and
//     begin another.  The units that are cut are joined from the workgroups'
//     partial results by the last of them to arrive.  (A fixed number of
//     splits per sequence leaves the chip waiting for the longest.)
//   - Whole long caches run at what the memory gives: 4 x 131071 MXFP8 tokens
//     (1.1 GB) 183 us, 6.0 TB/s; 8 x 16000 BF16 tokens, 8 kv heads of 128, 92
//     us, 5.7 TB/s; 32 ragged MXFP4 sequences (293 MB) 59 us, 5.0 TB/s.  What a
//     call adds is 8 to 10 us of waits one after the other: lengths, page
//     table, first rows, the waves' sums, results to the coherence point, the
//     join.
//   - Softmax statistics are FP32 and running.  The reference maximum of a
//     head moves only when a score passes it by 2^kLazy, so most tiles need
//     no reduction across lanes and no rescaling.
#include "attn_split.h"
#include "fp4_device.h"
#include "fp4_launch.h"
#include "kv_device.h"
#include "workspace.h"

namespace fp4 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kWaves = 4;             // waves of a workgroup, taking every fourth tile
// Scores may pass the reference maximum by this much (in powers of two)
// before it moves: probabilities up to 2^8, no loss in FP32 or BF16.
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct AttnArgs {
  KvPool c;
  const void* q;
  int64_t q_stride;
  const int32_t* table;
  int64_t width;
  const int32_t* lens;
  int32_t q_heads;
  int32_t group;       // query heads of a kv head
  int32_t head_tiles;  // ceil(group / 16)
  int64_t max_len;
  int64_t window;
  float scale_log2;    // scale * log2 e
  void* out;
  float* lse;
  int32_t q_f32, out_f32;
  int32_t batch;
  bool join;           // the workspace has room for the pieces of cut units
  uint32_t* done;      // arrival counters, one for each workgroup that begins a unit
  float* part;         // partial sums: workgroups x 2 x 16 heads x D
  float* stats;        // (maximum, sum): workgroups x 2 x 16 heads x 2
  float* final_stats;  // B x q_heads x (maximum, 1 / sum), for the weights
  float* scores;       // B x q_heads x score_stride, or null
  int64_t score_stride;
  const float* w_in;
  float* w_out;
  int64_t w_stride;
};

// ---- loads ----
// BYTES bytes of a cache row from p (aligned to their largest power of two,
// at most 16) as dwords.  Rows are read once: without the hint that says so 4
// x 131071 MXFP8 tokens take 199 us, with it 183 us.
template <int BYTES, int STEP = 0>
__device__ __forceinline__ void load_bytes(const uint8_t* __restrict__ p, uint32_t (&w)[(BYTES + 3) / 4]) {
  constexpr int kAlign = BYTES & -BYTES, kStep = STEP ? STEP : kAlign >= 16 ? 16 : kAlign;
  if constexpr (kAlign >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + i * kStep));
#pragma unroll
      for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
    }
  } else if constexpr (kAlign == 8) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i) {
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + i * kStep));
      w[2 * i] = v[0];
      w[2 * i + 1] = v[1];
    }
  } else if constexpr (kAlign == 4) {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p) + i);
  } else {
    static_assert(kAlign == 2, "rows are whole multiples of 32 bytes");
#pragma unroll
    for (int i = 0; i < (BYTES + 3) / 4; ++i) {
      w[i] = reinterpret_cast<const uint16_t*>(p)[2 * i];
      if (4 * i + 2 < BYTES) w[i] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
    }
  }
}

// BYTES (a multiple of 8) of scales from p, 8-byte aligned.
typedef uint32_t u32x4_by8 __attribute__((ext_vector_type(4), aligned(8)));
template <int BYTES>
__device__ __forceinline__ void load_scales(const uint8_t* __restrict__ p, uint32_t (&w)[BYTES / 4]) {
  constexpr int kQuads = BYTES / 16;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const u32x4 v = reinterpret_cast<const u32x4_by8*>(p)[i];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
  }
  if constexpr (BYTES % 16 != 0) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p + 16 * kQuads);
    w[4 * kQuads] = v[0];
    w[4 * kQuads + 1] = v[1];
  }
}

// Byte blk of token i's BLOCKS scale bytes in the dwords of four tokens.
template <int BLOCKS>
__device__ __forceinline__ uint32_t scale_byte(const uint32_t (&w)[BLOCKS], int i, uint32_t blk) {
  const int at = i * BLOCKS;  // the token's first byte
  if constexpr (BLOCKS <= 4) return (w[at / 4] >> (8u * (at % 4) + 8u * blk)) & 0xFFu;
  const uint64_t both = (uint64_t)w[at / 4] | (uint64_t)w[at / 4 + 1] << 32;
  return (uint32_t)(both >> (8u * (at % 4) + 8u * blk)) & 0xFFu;
}

__device__ __forceinline__ float e8m0(uint32_t byte) { return u2f(byte << 23); }

// Elements 2i, 2i + 1 of a lane's piece of a row (its dwords w) times s, as a BF16 pair.
template <int FMT, int N>
__device__ __forceinline__ uint32_t pair_of(const uint32_t (&w)[N], int i, float s) {
  if constexpr (FMT == kKvBf16) {
    return w[i];
  } else if constexpr (FMT == kKvMx8) {
    return (i & 1) ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], s, true))
                   : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i >> 1], s, false));
  } else {
    switch (i & 3) {
      case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i >> 2], s, 0));
      case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i >> 2], s, 1));
      case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i >> 2], s, 2));
      default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i >> 2], s, 3));
    }
  }
}

__device__ __forceinline__ v8bf frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(v8bf, u32x4{a, b, c, d});
}

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// v as TERMS BF16 terms (each the remainder's nearest BF16): TERMS = 3 is
// exact for normal FP32, 2 leaves at most 2^-17 relative.
template <int TERMS, int N>
__device__ __forceinline__ void split_terms(const float (&v)[N], uint32_t (&t)[TERMS][N / 2]) {
  float r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = v[i];
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      t[k][i] = bf16_pair(r[2 * i], r[2 * i + 1]);
      if (k + 1 < TERMS) {
        r[2 * i] -= u2f(t[k][i] << 16);
        r[2 * i + 1] -= u2f(t[k][i] & 0xFFFF0000u);
      }
    }
  }
}

// Two floats through the device's coherence point (other XCDs' workgroups
// read them; a plain store could stay in this XCD's L2).
__device__ __forceinline__ void store2_agent(float* p, float a, float b) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)f2u(a) | ((uint64_t)f2u(b) << 32), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ v2f load2_agent(const float* p) {
  const uint64_t u = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  return v2f{u2f((uint32_t)u), u2f((uint32_t)(u >> 32))};
}

__device__ __forceinline__ void store_out2(const AttnArgs& a, size_t i, float x, float y) {
  if (a.out_f32)
    *reinterpret_cast<v2f*>(static_cast<float*>(a.out) + i) = v2f{x, y};
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + i) = bf16_pair(x, y);
}

// p[i] for an index that is the same in the whole wavefront, by a scalar load
// (page tables and lengths do not change while the kernel runs, which the
// constant address space says).  A vector load here would be the youngest in
// flight, and waiting for it would wait for all of K and V (a fifth of the
// rate over an MXFP4 cache).
__device__ __forceinline__ int32_t load_uniform(const int32_t* p, size_t i) {
  typedef const __attribute__((address_space(4))) int32_t* constant_ptr;
  return ((constant_ptr)(uintptr_t)p)[i];
}

// The tokens of a sequence that the call attends to, in tiles of 32 aligned
// to the pages (a page is at least 16 tokens).
struct Range {
  uint32_t first, len;    // tokens [first, len)
  uint32_t tile0, tiles;  // tiles of the sequence from tile0 on
  __device__ __forceinline__ uint32_t counted(uint32_t more) const { return counted_tiles(tiles, more); }
};
__device__ __forceinline__ Range range_at(const AttnArgs& a, int64_t l) {
  Range r;
  r.len = (uint32_t)(l < 0 ? 0 : l < a.max_len ? l : a.max_len);
  r.first = a.window > 0 && a.window < (int64_t)r.len ? r.len - (uint32_t)a.window : 0u;
  r.tile0 = r.first / kTile;
  r.tiles = a.c.pages > 0 ? (r.len + kTile - 1) / kTile - r.tile0 : 0u;  // an empty pool has nothing to read
  return r;
}

__device__ __forceinline__ Range range_of(const AttnArgs& a, uint32_t b) { return range_at(a, a.lens[b]); }

// Inclusive sum over the lanes up to this one (DPP: within rows of 16, then
// each row's last lane to the next row, then lane 31 to the upper half).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
  return v;
}

// A workgroup's share [pos, end) of the tiles laid end to end, sequence b
// beginning at `base` (in tiles of one unit; a sequence has `units` of them).
// All counts fit 32 bits: the host bounds them.
struct Share {
  uint32_t pos, end, base, share, b, more;
};
__device__ __forceinline__ Share share_of(const AttnArgs& a, uint32_t units, uint32_t change) {
  const uint32_t lane = threadIdx.x & 63u, B = (uint32_t)a.batch;
  const uint32_t each = (B + 63u) / 64u, b0 = lane * each;  // sequences of a lane
  uint32_t mine = 0u;
  for (uint32_t i = 0u; i < each; ++i)
    if (b0 + i < B) mine += range_of(a, b0 + i).counted(0u);
  uint32_t upto = wave_scan(mine);
  Share s;
  uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63) * units;
  s.share = share_tiles(total, gridDim.x);
  s.more = counted_change(s.share, change, a.join);
  if (s.more > 0u) {
    mine += s.more * (b0 < B ? min(each, B - b0) : 0u);
    upto = wave_scan(mine);
    total = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63) * units;
    s.share = share_tiles(total, gridDim.x);
  }
  s.pos = min(blockIdx.x * s.share, total);
  s.end = s.pos + min(s.share, total - s.pos);
  const uint64_t past = __ballot(upto * units > s.pos);
  const int at = past == 0u ? 0 : (int)__builtin_ctzll(past);
  s.base = (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), at);
  s.b = (uint32_t)at * each;
  while (s.pos < s.end) {
    const uint32_t v = range_at(a, load_uniform(a.lens, s.b)).counted(s.more);
    if ((s.base + v) * units > s.pos) break;
    s.base += v;
    ++s.b;
  }
  return s;
}

// A workgroup's shared memory.
template <int D>
struct Shared {
  float red[2][kHeadTile][D + 4];  // sums of two waves (rows padded against bank conflicts); in a join, factors
  float wave_m[kWaves][kHeadTile], wave_l[kWaves][kHeadTile];
  uint32_t last_arrival;
};

// A workgroup's piece of a unit (tiles past the sequence's last only count) for
// the query heads head0 .. head0 + heads - 1, which read kv head h of sequence b.
struct Piece : Cut {
  Range r;
  uint32_t b, h, head0, heads;
};

// Element pairs of a piece's results, 256 at a time: f(head, d).
template <int D, typename F>
__device__ __forceinline__ void each_pair(uint32_t heads, F f) {
  for (uint32_t i = threadIdx.x; i < heads * (D / 2); i += 256u) f(i / (D / 2), 2u * (i % (D / 2)));
}

// Head hd's output elements d, d + 1.
template <int D>
__device__ __forceinline__ void write_out(const AttnArgs& a, const Piece& pc, uint32_t hd, uint32_t d, float x,
                                          float y) {
  store_out2(a, ((size_t)pc.b * (uint32_t)a.q_heads + pc.head0 + hd) * D + d, x, y);
}

// Head hd's maximum and sum to where they are wanted (one thread a head).
__device__ __forceinline__ void write_stats(const AttnArgs& a, const Piece& pc, uint32_t hd, float mx, float s) {
  const size_t at = (size_t)pc.b * (uint32_t)a.q_heads + pc.head0 + hd;
  if (a.lse) a.lse[at] = s == 0.0f ? -INFINITY : (mx + __builtin_log2f(s)) * kLn2;
  if (a.final_stats) *reinterpret_cast<v2f*>(a.final_stats + 2 * at) = v2f{mx, s == 0.0f ? 0.0f : 1.0f / s};
}

// The results of n <= 16 pieces, first, first + step, .., joined by one
// workgroup: every head's maximum and sum into sh.wave_m[0], sh.wave_l[0], its
// sums of V to result(head, d, x, y), ITEMS pairs of elements a thread, BATCH
// pieces at a time.  A load
// from the coherence point takes about a microsecond, so they are asked for
// many at a time, the first of them before the factors 2^(m_p - M) are known.
template <int D, int ITEMS, int BATCH, typename F>
__device__ __forceinline__ void join_items(const AttnArgs& a, const Piece& pc, Shared<D>& sh, uint32_t first,
                                           uint32_t step, uint32_t n, F result) {
  const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
  float* factor = &sh.red[0][0][0];  // 16 heads x 16 pieces
  static_assert(kHeadTile * kDirect * sizeof(float) <= sizeof(sh.red), "factors fit in the array they reuse");
  v2f ms[kHeadTile / kWaves];
#pragma unroll
  for (int k = 0; k < kHeadTile / kWaves; ++k) {
    const uint32_t hd = k * kWaves + wave;
    ms[k] = v2f{-INFINITY, 0.0f};
    if (hd < pc.heads && lane < n) ms[k] = load2_agent(a.stats + 2u * (place_of(pc.wg0, first + lane * step) + hd));
  }
  v2f v[(uint32_t)BATCH][ITEMS];
  const auto ask = [&](uint32_t q0) __attribute__((always_inline)) {
#pragma unroll
    for (uint32_t j = 0; j < (uint32_t)BATCH; ++j) {
      if (q0 + j >= n) continue;
      const float* from = a.part + (size_t)place_of(pc.wg0, first + (q0 + j) * step) * D;
#pragma unroll
      for (uint32_t k = 0; k < ITEMS; ++k)
        if ((k * 256u + tid) / (D / 2) < pc.heads) v[j][k] = load2_agent(from + 2u * (k * 256u + tid));
    }
  };
  ask(0u);
#pragma unroll
  for (int k = 0; k < kHeadTile / kWaves; ++k) {
    const uint32_t hd = k * kWaves + wave;
    const float to = wave_fmax(ms[k][0]);
    const float f = ms[k][0] == -INFINITY ? 0.0f : exp2_fast(ms[k][0] - to);
    const float s = wave_fsum(ms[k][1] * f);
    if (lane < kDirect) factor[hd * kDirect + lane] = f;
    if (lane == 0u) {
      sh.wave_m[0][hd] = to;
      sh.wave_l[0][hd] = s;
    }
  }
  __syncthreads();
  float x[ITEMS], y[ITEMS];
#pragma unroll
  for (uint32_t k = 0; k < ITEMS; ++k) x[k] = y[k] = 0.0f;
  for (uint32_t q0 = 0u; q0 < n; q0 += (uint32_t)BATCH) {
    if (q0 > 0u) ask(q0);
#pragma unroll
    for (uint32_t j = 0; j < (uint32_t)BATCH; ++j) {
      if (q0 + j >= n) continue;
#pragma unroll
      for (uint32_t k = 0; k < ITEMS; ++k) {
        const uint32_t hd = (k * 256u + tid) / (D / 2);
        if (hd >= pc.heads) continue;
        const float f = factor[hd * kDirect + q0 + j];
        x[k] = __builtin_fmaf(f, v[j][k][0], x[k]);
        y[k] = __builtin_fmaf(f, v[j][k][1], y[k]);
      }
    }
  }
#pragma unroll
  for (uint32_t k = 0; k < ITEMS; ++k) {
    const uint32_t i = k * 256u + tid, hd = i / (D / 2);
    if (hd < pc.heads) result(hd, 2u * (i % (D / 2)), x[k], y[k]);
  }
}

template <int D, typename F>
__device__ __forceinline__ void join_pieces(const AttnArgs& a, const Piece& pc, Shared<D>& sh, uint32_t first,
                                            uint32_t step, uint32_t n, F result) {
  constexpr int kItems = kHeadTile * (D / 2) / 256;
  const uint32_t items = (pc.heads * (D / 2) + 255u) / 256u;
  if (items <= 1u)
    join_items<D, 1, 8>(a, pc, sh, first, step, n, result);
  else if (kItems > 2 && items <= kItems / 2u)
    join_items<D, kItems / 2, 8>(a, pc, sh, first, step, n, result);
  else
    join_items<D, kItems, kItems <= 4 ? 8 : 4>(a, pc, sh, first, step, n, result);
}

// One piece: the attention to its tokens, and the unit's result if it is the
// only one, else its part of it.
template <int FMT, int D, bool EX>
__device__ __forceinline__ void attend_piece(const AttnArgs& a, const Piece& pc, Shared<D>& sh) {
  constexpr int kRow = (int)kv_row_bytes(FMT, D);
  constexpr int kSteps = D / 32;               // matrix instructions along D for 16 tokens
  constexpr int EV = D / 16;                   // elements of V per lane and token
  constexpr int kKB = kRow / 4, kVB = kRow / 16;
  constexpr int kKW = kKB / 4, kVW = (kVB + 3) / 4;
  constexpr bool MX = FMT != kKvBf16;
  constexpr int kBlocks = D / 32;
  // A lane's share of a K row lies in chunks of up to 16 bytes, four lanes'
  // side by side, so that a load takes whole 64 bytes (a quarter of the row
  // for each lane costs a load of every line for each of its 16 bytes: 8
  // sequences of 16000 tokens, 8 kv heads of 128 BF16, 116 us against 92).
  constexpr int kChunk = (kKB & -kKB) < 16 ? (kKB & -kKB) : 16, kChunks = kKB / kChunk;
  constexpr int kChunkElems = D / 4 / kChunks;
  // Element of step s that a lane begins with.
  const auto k_elem = [](uint32_t g, int s) __attribute__((always_inline)) {
    return ((uint32_t)(8 * s / kChunkElems) * 4u + g) * kChunkElems + (uint32_t)(8 * s % kChunkElems);
  };
  // BF16 V the same way: elements that a lane has side by side.
  constexpr int kPart = MX ? EV : EV % 8 == 0 ? 8 : 4;
  // Element that row `row` of product e stands for.
  const auto v_elem = [](uint32_t row, int e) __attribute__((always_inline)) {
    return (uint32_t)(e / kPart) * 16u * kPart + row * kPart + (uint32_t)(e % kPart);
  };
  // BF16 terms of a query and of a probability: three hold FP32's 24 bits.  With
  // BF16 q and out over an MX cache, whose values have 4 significant bits at
  // most, probabilities take two (2^-17): the third costs 32 ragged MXFP4
  // sequences 6% (59.4 to 63.1 us) and 8 x 16000 MXFP8 tokens 0.4% to 3% (heads
  // of 128: 54.9 to 55.1 us, of 64: 29.6 to 30.6).  Over a BF16 cache it costs
  // nothing (88.4 and 88.5 us, heads of 256 169.8 and 169.7).
  constexpr int kQTerms = EX ? 3 : 1, kPTerms = EX || !MX ? 3 : 2;

  const uint32_t lane = threadIdx.x & 63u, c = lane & 15u, g = lane >> 4;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t shift = (uint32_t)__builtin_ctz((uint32_t)a.c.page_size), in_page = (uint32_t)a.c.page_size - 1u;
  const Range r = pc.r;
  const uint32_t b = pc.b, h = pc.h, head0 = pc.head0, heads = pc.heads, t_end = min(pc.t_end, r.tiles);

  // Q: head c's elements k_elem(g, s) .. + 7 in step s; zero for heads past
  // the group.  Asked for here, looked at once K and V are asked for too.
  const size_t q_at = (size_t)b * (size_t)a.q_stride + (size_t)(head0 + (c < heads ? c : 0u)) * D;
  u32x4 q_raw[kSteps];
  if constexpr (!EX) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      q_raw[s] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.q) + q_at + k_elem(g, s));
  }

  v4f o[EV];
#pragma unroll
  for (int e = 0; e < EV; ++e) o[e] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;  // of head c; l of this lane's tokens alone

  const uint32_t pages_used = (r.len + in_page) >> shift;
  const int32_t* table = a.table + (size_t)b * (size_t)a.width;

  // Row number of a half tile's first token, or ~0 where its page is not in the pool.
  const auto half_row = [&](uint32_t tile, uint32_t j) -> uint64_t {
    const uint32_t t = (r.tile0 + tile) * kTile + 16u * j, p = t >> shift;
    const int32_t page = tile < t_end && p < pages_used ? load_uniform(table, p) : -1;
    if (page < 0 || page >= a.c.pages) return ~0ull;
    return (((uint64_t)(uint32_t)page * (uint32_t)a.c.kv_heads + h) << shift) + (t & in_page);
  };

  uint32_t kw[2][kKW], vw[8][kVW];
  // MX: K's scale bytes (all of a token's, or one for each chunk, which lies in
  // one block), and all of V's of the lane's four consecutive tokens of each
  // half: few wide loads, since every load is a request to the caches however
  // narrow.
  constexpr bool kAllScales = kBlocks == 4 || kBlocks == 8;
  uint32_t kb[2][kAllScales ? kBlocks / 4 : kChunks], vb[2][kBlocks];
  const uint32_t k_off = c * kRow + g * kChunk, v_off = 4u * g * kRow + c * (MX ? kVB : 2 * kPart);
  constexpr int kVScales = 32 % EV == 0 ? 1 : 2;
  const uint32_t k_blk = g * kChunkElems / 32u, v_blk = c * EV / 32u;

  const auto load_k = [&](const uint64_t (&row)[2]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint64_t at = row[j] == ~0ull ? 0u : row[j];
      load_bytes<kKB, 4 * kChunk>(static_cast<const uint8_t*>(a.c.k) + at * kRow + k_off, kw[j]);
      if constexpr (MX) {
        const uint8_t* from = a.c.ks + at * kBlocks + c * kBlocks;
        if constexpr (kBlocks == 8) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(from);
          kb[j][0] = w[0];
          kb[j][1] = w[1];
        } else if constexpr (kBlocks == 4) {
          kb[j][0] = *reinterpret_cast<const uint32_t*>(from);
        } else {
#pragma unroll
          for (int i = 0; i < kChunks; ++i) kb[j][i] = from[k_blk + i * kChunkElems / 8];
        }
      }
    }
  };
  const auto load_v = [&](const uint64_t (&row)[2]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t at = row[j >> 2] == ~0ull ? 0u : row[j >> 2];
      const uint8_t* from = static_cast<const uint8_t*>(a.c.v) + at * kRow + v_off + (j & 3) * kRow;
      load_bytes<kVB, MX ? 0 : 32 * kPart>(from, vw[j]);
    }
    if constexpr (MX) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint64_t at = row[j] == ~0ull ? 0u : row[j];
        load_scales<4 * kBlocks>(a.c.vs + at * kBlocks + 4u * g * kBlocks, vb[j]);
      }
    }
  };

  uint32_t tile = pc.t_begin + wave;
  uint64_t row[2] = {~0ull, ~0ull}, next[2] = {~0ull, ~0ull};
  if (tile < t_end) {
    row[0] = half_row(tile, 0);
    row[1] = half_row(tile, 1);
    next[0] = half_row(tile + kWaves, 0);
    next[1] = half_row(tile + kWaves, 1);
    load_k(row);
    load_v(row);
  }
  v8bf q[kQTerms][kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if constexpr (EX) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const size_t at = q_at + k_elem(g, s) + i;
        v[i] = a.q_f32 ? static_cast<const float*>(a.q)[at]
                       : u2f((uint32_t) static_cast<const uint16_t*>(a.q)[at] << 16);
        v[i] = c < heads ? v[i] : 0.0f;
      }
      uint32_t t[3][4];
      split_terms<3>(v, t);
#pragma unroll
      for (int k = 0; k < 3; ++k) q[k][s] = frag(t[k][0], t[k][1], t[k][2], t[k][3]);
    } else {
      if (c >= heads) q_raw[s] = u32x4{0u, 0u, 0u, 0u};
      q[0][s] = __builtin_bit_cast(v8bf, q_raw[s]);
    }
  }
  for (; tile < t_end; tile += kWaves) {
    const bool more = tile + kWaves < t_end;
    // S^T: rows tokens, columns heads.
    v4f st[2] = {v4f{0.0f, 0.0f, 0.0f, 0.0f}, v4f{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float ks[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int blk = i * kChunkElems / 8;  // of the chunk, counted from k_blk
        ks[i] = 1.0f;
        if constexpr (MX && kAllScales) ks[i] = e8m0((kb[j][blk / 4] >> (8u * (blk % 4) + 8u * k_blk)) & 0xFFu);
        if constexpr (MX && !kAllScales) ks[i] = e8m0(kb[j][i]);
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const float sc = ks[8 * s / kChunkElems];
        const v8bf kf = frag(pair_of<FMT>(kw[j], 4 * s, sc), pair_of<FMT>(kw[j], 4 * s + 1, sc),
                             pair_of<FMT>(kw[j], 4 * s + 2, sc), pair_of<FMT>(kw[j], 4 * s + 3, sc));
#pragma unroll
        for (int k = 0; k < kQTerms; ++k) st[j] = mfma(kf, q[k][s], st[j]);
      }
    }
    const bool in0 = row[0] != ~0ull, in1 = row[1] != ~0ull;
    if (more) load_k(next);

    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = st[i >> 2][i & 3] * a.scale_log2;
    const uint32_t t0 = (r.tile0 + tile) * kTile;
    const bool full = t0 >= r.first && t0 + kTile <= r.len && in0 && in1;
    if (!full) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t t = t0 + 16u * (i >> 2) + 4u * g + (i & 3);
        const bool ok = t >= r.first && t < r.len && ((i >> 2) ? in1 : in0);
        x[i] = ok ? x[i] : -INFINITY;
      }
    }
    if (a.scores && c < heads) {
      float* at = a.scores + ((size_t)b * (uint32_t)a.q_heads + head0 + c) * (size_t)a.score_stride + t0 + 4u * g;
      *reinterpret_cast<v4f*>(at) = v4f{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<v4f*>(at + 16) = v4f{x[4], x[5], x[6], x[7]};
    }
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__any(top > m + kLazy)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float to = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.0f : exp2_fast(m - to);
      l *= f;
#pragma unroll
      for (int e = 0; e < EV; ++e) o[e] *= f;
      m = to;
    }
    const float ref = m == -INFINITY ? 0.0f : m;  // nothing but masked tokens so far: all p are 0
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = exp2_fast(x[i] - ref);
      l += p[i];
    }
    uint32_t pt[kPTerms][4];
    split_terms<kPTerms>(p, pt);

    // V: tokens paired two by two per element.
    uint32_t vp[8][EV / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float vs[2] = {1.0f, 1.0f};
      if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < kVScales; ++i)
          vs[i] = e8m0(scale_byte<kBlocks>(vb[j >> 2], j & 3, min(v_blk + i, (uint32_t)kBlocks - 1u)));
      }
#pragma unroll
      for (int i = 0; i < EV / 2; ++i) {
        float sc = vs[0];
        if constexpr (kVScales == 2) sc = c * EV + 2 * i >= 32u * (v_blk + 1u) ? vs[1] : vs[0];
        vp[j][i] = pair_of<FMT>(vw[j], i, sc);
      }
    }
    if (!full) {
      // Whatever lies in a masked slot (NaN too) must not meet p = 0.
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t t = t0 + 16u * (j >> 2) + 4u * g + (j & 3);
        const bool ok = t >= r.first && t < r.len && ((j >> 2) ? in1 : in0);
#pragma unroll
        for (int i = 0; i < EV / 2; ++i) vp[j][i] = ok ? vp[j][i] : 0u;
      }
    }
    if constexpr (MX) {  // the raw registers are free once converted
      if (more) load_v(next);
    }
#pragma unroll
    for (int e = 0; e < EV; ++e) {
      constexpr uint32_t kLo = 0x05040100u, kHi = 0x07060302u;
      const uint32_t sel = (e & 1) ? kHi : kLo;
      const int i = e >> 1;
      const auto two = [&](int j) { return __builtin_amdgcn_perm(vp[j + 1][i], vp[j][i], sel); };
      const v8bf vf = frag(two(0), two(2), two(4), two(6));
#pragma unroll
      for (int k = 0; k < kPTerms; ++k) o[e] = mfma(vf, frag(pt[k][0], pt[k][1], pt[k][2], pt[k][3]), o[e]);
    }
    if constexpr (!MX) {
      if (more) load_v(next);
    }
    row[0] = next[0];
    row[1] = next[1];
    if (more) {
      next[0] = half_row(tile + 2 * kWaves, 0);
      next[1] = half_row(tile + 2 * kWaves, 1);
    }
  }

  // ---- the four waves' results: a common maximum, then sums in fixed order ----
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lane < 16u) {
    sh.wave_m[wave][c] = m;
    sh.wave_l[wave][c] = l;
  }
  __syncthreads();
  float M = sh.wave_m[0][c];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) M = fmaxf(M, sh.wave_m[w][c]);
  const float f = m == -INFINITY ? 0.0f : exp2_fast(m - M);
  // Lane (c, g) holds head c, d = (4g + i) EV + e of o[e][i].
  if (wave < 2u && c < heads) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < EV; ++e) sh.red[wave][c][v_elem(4 * g + i, e)] = o[e][i] * f;
  }
  __syncthreads();
  if (wave >= 2u && c < heads) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < EV; ++e) sh.red[wave - 2u][c][v_elem(4 * g + i, e)] += o[e][i] * f;
  }
  __syncthreads();

  // Head hd's sum over the waves, for the workgroup's maximum mx.  (A wave whose
  // scores are all NaN has the maximum of one without tokens, but a NaN sum,
  // which has to stay: 0 times it.)
  const auto head_sum = [&](uint32_t hd, float& mx) {
    mx = sh.wave_m[0][hd];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, sh.wave_m[w][hd]);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      s += sh.wave_l[w][hd] * (sh.wave_m[w][hd] == -INFINITY ? 0.0f : exp2_fast(sh.wave_m[w][hd] - mx));
    return s;
  };
  float mx;
  if (pc.pieces == 1u) {
    each_pair<D>(heads, [&](uint32_t hd, uint32_t d) {
      const float s = head_sum(hd, mx), inv = s == 0.0f ? 0.0f : 1.0f / s;
      write_out<D>(a, pc, hd, d, (sh.red[0][hd][d] + sh.red[1][hd][d]) * inv,
                   (sh.red[0][hd][d + 1] + sh.red[1][hd][d + 1]) * inv);
    });
    if (threadIdx.x < heads) {
      const float s = head_sum(threadIdx.x, mx);
      write_stats(a, pc, threadIdx.x, mx, s);
    }
    return;
  }

  // ---- a part of the unit: written through, and the last to arrive joins them ----
  const uint32_t mine = place_of(pc.wg0, blockIdx.x - pc.wg0);
  each_pair<D>(heads, [&](uint32_t hd, uint32_t d) {
    store2_agent(a.part + (size_t)(mine + hd) * D + d, sh.red[0][hd][d] + sh.red[1][hd][d],
                 sh.red[0][hd][d + 1] + sh.red[1][hd][d + 1]);
  });
  if (threadIdx.x < heads) {
    const float s = head_sum(threadIdx.x, mx);
    store2_agent(a.stats + 2u * (mine + threadIdx.x), mx, s);
  }
  uint32_t step = 1u, left = pc.pieces, level = 0u;
  for (;;) {
    const Join j = join_of(pc.wg0, blockIdx.x - pc.wg0, step, left, ++level);
    uint32_t* done = a.done + j.done;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's results have reached the coherence point
    __syncthreads();
    if (threadIdx.x == 0u) {
      const uint32_t before = __hip_atomic_fetch_add(done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh.last_arrival = before == j.n - 1u;
      if (sh.last_arrival) __hip_atomic_store(done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!sh.last_arrival) return;
    const auto result = [&](uint32_t hd, uint32_t d, float x, float y) __attribute__((always_inline)) {
      if (!j.whole) {
        store2_agent(a.part + (size_t)(place_of(pc.wg0, j.first) + hd) * D + d, x, y);
      } else {
        const float s = sh.wave_l[0][hd], inv = s == 0.0f ? 0.0f : 1.0f / s;
        write_out<D>(a, pc, hd, d, x * inv, y * inv);
      }
    };
    join_pieces<D>(a, pc, sh, j.first, step, j.n, result);
    if (threadIdx.x < heads) {
      const float mx = sh.wave_m[0][threadIdx.x], s = sh.wave_l[0][threadIdx.x];
      if (!j.whole)
        store2_agent(a.stats + 2u * (place_of(pc.wg0, j.first) + threadIdx.x), mx, s);
      else
        write_stats(a, pc, threadIdx.x, mx, s);
    }
    if (j.whole) return;
    step *= 8u;
    left = (left + 7u) / 8u;
  }
}

template <int FMT, int D, bool EX>
__global__ __launch_bounds__(256, groups_of(D, EX) / 256u) void attn_decode_kernel(AttnArgs a) {
  __shared__ Shared<D> sh;
  const uint32_t units = (uint32_t)a.c.kv_heads * (uint32_t)a.head_tiles;
  constexpr uint32_t kChange = change_tiles(kv_row_bytes(FMT, D));
  Share w = share_of(a, units, kChange);
  while (w.pos < w.end) {
    // The share's next piece, of unit `unit` of sequence w.b.
    Piece pc;
    pc.b = w.b;
    pc.r = range_at(a, load_uniform(a.lens, w.b));
    const uint32_t counted = pc.r.counted(w.more), unit = (w.pos - w.base * units) / counted;
    const uint32_t unit0 = w.base * units + unit * counted;
    static_cast<Cut&>(pc) = cut_at(w.pos, w.end, unit0, counted, w.share);
    const uint32_t ht = unit % (uint32_t)a.head_tiles;
    pc.h = unit / (uint32_t)a.head_tiles;
    pc.heads = min((uint32_t)a.group - ht * kHeadTile, (uint32_t)kHeadTile);
    pc.head0 = pc.h * (uint32_t)a.group + ht * kHeadTile;
    attend_piece<FMT, D, EX>(a, pc, sh);
    w.pos += pc.t_end - pc.t_begin;
    if (pc.t_end == counted && unit + 1u == units) {
      w.base += counted;
      ++w.b;
    }
    __syncthreads();  // the shared memory is free for the next piece
  }
}

// weights_out = weights_in + sum over the kv head's query heads of p, from the
// stored scores: p = 2^(x - M) / L, and 0 for a masked token (x = -inf) also
// where a NaN among the others makes L one.  Four tokens a thread.  The scores
// cross memory once more (FP32, a fifth of the rows' bytes for 64 BF16 elements
// and 8 heads), since M and L are known only at the end: 48 ragged sequences of
// up to 4099 tokens, 64 heads, 7.7 us after the attention's 56.
__global__ __launch_bounds__(256) void attn_weights_kernel(AttnArgs a) {
  const uint32_t h = blockIdx.y, b = blockIdx.z, t = (blockIdx.x * 256u + threadIdx.x) * 4u;
  const Range r = range_of(a, b);
  if (t >= r.len) return;
  const size_t at = ((size_t)b * gridDim.y + h) * (size_t)a.w_stride + t;
  const uint32_t n = min(r.len - t, 4u);
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (r.tiles > 0u && t >= r.tile0 * kTile) {  // earlier tiles were not scored: all before the window
    const size_t head0 = (size_t)b * (uint32_t)a.q_heads + (size_t)h * (uint32_t)a.group;
    for (uint32_t k = 0u; k < (uint32_t)a.group; ++k) {
      const v4f x = *reinterpret_cast<const v4f*>(a.scores + (head0 + k) * (size_t)a.score_stride + t);
      const v2f ms = *reinterpret_cast<const v2f*>(a.final_stats + 2 * (head0 + k));
      const float ref = ms[0] == -INFINITY ? 0.0f : ms[0];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] += x[i] == -INFINITY ? 0.0f : exp2_fast(x[i] - ref) * ms[1];
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < 4u; ++i)
    if (i < n) a.w_out[at + i] = (a.w_in ? a.w_in[at + i] : 0.0f) + w[i];
}

template <int FMT, int D>
void launch_d(const AttnArgs& a, uint32_t grid, bool exact, hipStream_t stream) {
  if (exact)
    attn_decode_kernel<FMT, D, true><<<grid, 256, 0, stream>>>(a);
  else
    attn_decode_kernel<FMT, D, false><<<grid, 256, 0, stream>>>(a);
}

template <int FMT>
void launch_fmt(const AttnArgs& a, uint32_t grid, bool exact, hipStream_t stream) {
  switch (a.c.head_dim) {
    case 64: return launch_d<FMT, 64>(a, grid, exact, stream);
    case 128: return launch_d<FMT, 128>(a, grid, exact, stream);
    case 192: return launch_d<FMT, 192>(a, grid, exact, stream);
    default: return launch_d<FMT, 256>(a, grid, exact, stream);
  }
}

}  // namespace

static_assert(kGroups * 4u == kControlBytes);
size_t attn_decode_workspace(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_len,
                             bool weights) {
  if (B == 0 || q_heads == 0) return 0;
  return layout_of(B, q_heads, kv_heads, head_dim, max_len, weights).total;
}

hipError_t launch_attn_decode(const KvPool& c, const void* q, int q_dtype, int64_t q_stride, const int32_t* table,
                              int64_t width, const int32_t* lens, int64_t B, int64_t q_heads, int64_t max_len,
                              int64_t window, float scale, void* out, int out_dtype, float* lse,
                              const float* weights_in, float* weights_out, int64_t weights_stride, void* workspace,
                              hipStream_t stream) {
  const Layout w = layout_of(B, q_heads, c.kv_heads, c.head_dim, max_len, weights_out != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnArgs a{};
  a.c = c;
  a.q = q;
  a.q_stride = q_stride;
  a.table = table;
  a.width = width;
  a.lens = lens;
  a.q_heads = (int32_t)q_heads;
  a.group = (int32_t)(q_heads / c.kv_heads);
  a.head_tiles = (int32_t)w.head_tiles;
  a.batch = (int32_t)B;
  a.join = w.join;
  a.max_len = max_len;
  a.window = window;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.lse = lse;
  a.q_f32 = q_dtype == kDtF32;
  a.out_f32 = out_dtype == kDtF32;
  a.done = reinterpret_cast<uint32_t*>(ws + w.done);
  a.stats = reinterpret_cast<float*>(ws + w.stats);
  a.part = reinterpret_cast<float*>(ws + w.part);
  if (weights_out) {
    a.final_stats = reinterpret_cast<float*>(ws + w.final_stats);
    a.scores = reinterpret_cast<float*>(ws + w.scores);
    a.score_stride = w.score_stride;
    a.w_in = weights_in;
    a.w_out = weights_out;
    a.w_stride = weights_stride;
  }
  const bool exact = q_dtype == kDtF32 || out_dtype == kDtF32;
  const uint32_t most = groups_of(c.head_dim, exact), grid = w.groups < most ? w.groups : most;
  switch (c.fmt) {
    case kKvBf16: launch_fmt<kKvBf16>(a, grid, exact, stream); break;
    case kKvMx8: launch_fmt<kKvMx8>(a, grid, exact, stream); break;
    default: launch_fmt<kKvMx4>(a, grid, exact, stream); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !weights_out || max_len == 0) return e;
  attn_weights_kernel<<<dim3((uint32_t)((max_len + 1023) / 1024), (uint32_t)c.kv_heads, (uint32_t)B), 256, 0,
                        stream>>>(a);
  return hipGetLastError();
}

}  // namespace fp4
