// attn_split.h -- how fp4_attn_decode cuts its work into workgroups' shares,
// and where the pieces of a cut unit keep their results.  The kernel, the host
// that sizes the workspace and the CPU test of both (tests/test_attn_split.py)
// compile this one source.  Internal header, of whole numbers only.
#pragma once

#include "host_device.h"

namespace fp4 {

constexpr int kTile = 32;         // tokens of a wave's step
constexpr uint32_t kGrain = 4;    // shares and units are whole multiples of this many tiles
constexpr int kHeadTile = 16;     // query heads of a workgroup
constexpr uint32_t kDirect = 16;  // pieces of a unit that are joined at once
// Workgroups: as many as fit at once, two a CU, or one where a row's
// accumulators, or three terms of a query, fill the registers.
//   32 ragged MXFP4 sequences of 128-element rows: 61 us in 512, 89, 80 and 72
//   in 256, 768 and 1024; 4 x 131071 MXFP8 tokens 190 us, 190, 227, 200.
//   8 x 16000 MXFP4 tokens of 256-element rows: 48 us in 256, 65 in 512 of
//   which 256 fit, 66 in 512 with the registers cut so that they fit.
constexpr uint32_t kGroups = 512;
FP4_HOST_DEVICE constexpr uint32_t groups_of(int64_t D, bool exact) {
  return D > 128 || (exact && D > 64) ? kGroups / 2u : kGroups;
}

// Tiles that a unit (the tokens of a sequence that one kv head's 16 query
// heads attend to) counts: whole grains, and one at least (an empty sequence's
// result has to be written too), and `more` for the time that changing from
// one unit to the next takes.
FP4_HOST_DEVICE uint32_t counted_tiles(uint32_t tiles, uint32_t more) {
  const uint32_t grains = tiles / kGrain + (tiles % kGrain != 0u ? 1u : 0u);
  return (grains > 1u ? grains : 1u) * kGrain + more;
}

// Changing units (the end of one, the first loads of the next) takes about as
// long as 48 KB of rows: in tiles, to whole grains.  With none counted 32
// ragged MXFP4 sequences take 66 us, with it 60 us.
FP4_HOST_DEVICE constexpr uint32_t change_tiles(uint32_t row_bytes) {
  return (49152u / (2u * kTile * row_bytes) + kGrain - 1u) / kGrain * kGrain;
}

// What of `change` is counted, for shares of `share` tiles: all where shares
// are long enough not to be cut because of it, and none where the call has no
// room for the pieces of a cut unit (`join` false: no sequence has more than a
// grain).  Units of one grain with nothing more lie on whole shares' grains
// and are never cut; with a change of units counted they would be, which is
// slower too (193 sequences of 128 BF16 tokens, 8 kv heads of 128: 29.7 us whole,
// 32.4 cut and joined; 1500 of MXFP8 134 and 139).
FP4_HOST_DEVICE uint32_t counted_change(uint32_t share, uint32_t change, bool join) {
  return join && share >= 4u * change ? change : 0u;
}

// A workgroup's share of `total` tiles (whole grains) among `groups`.
FP4_HOST_DEVICE uint32_t share_tiles(uint32_t total, uint32_t groups) {
  const uint32_t n = total / kGrain;
  return (n / groups + (n % groups != 0u ? 1u : 0u)) * kGrain;
}

// The piece of a unit that a share holds from `pos` on: tiles [t_begin, t_end)
// of it, the unit's `counted` tiles beginning at unit0; `pieces` workgroups
// from wg0 on have one.
struct Cut {
  uint32_t t_begin, t_end, wg0, pieces;
};
FP4_HOST_DEVICE Cut cut_at(uint32_t pos, uint32_t end, uint32_t unit0, uint32_t counted, uint32_t share) {
  Cut c;
  c.t_begin = pos - unit0;
  c.t_end = c.t_begin + (end - pos) < counted ? c.t_begin + (end - pos) : counted;
  c.wg0 = unit0 / share;
  c.pieces = (unit0 + counted - 1u) / share - c.wg0 + 1u;
  return c;
}

// Where piece p of a unit begun by workgroup wg0 keeps its results, in heads'
// rows: a workgroup has a place for a unit it begins and one for a unit begun
// before.
FP4_HOST_DEVICE uint32_t place_of(uint32_t wg0, uint32_t p) {
  return (2u * (wg0 + p) + (p == 0u ? 1u : 0u)) * kHeadTile;
}

// Up to kDirect pieces are joined at once.  More are joined eight by eight
// first, and eight of those, each by the last to arrive of its own, into the
// place of its first piece.  The unit's counter is that of the workgroup that
// begins it; the others are those of workgroups wholly inside the unit, which
// begin none.  (One workgroup for all: 131000 tokens of one kv head of 256
// BF16, in 512 pieces, 479 us; so, 94 us, and in today's 256 pieces 52.)
// Piece p at a level (the first is 1) where `left` results, every step-th
// piece's, are left to join: `n` of them from piece `first` on are joined
// together, and arrive at counter `done`.
struct Join {
  bool whole;  // what is left of the unit
  uint32_t first, n, done;
};
FP4_HOST_DEVICE Join join_of(uint32_t wg0, uint32_t p, uint32_t step, uint32_t left, uint32_t level) {
  Join j;
  j.whole = left <= kDirect;
  const uint32_t at = p / (8u * step);
  j.first = j.whole ? 0u : 8u * step * at;
  j.n = j.whole ? left : left - 8u * at < 8u ? left - 8u * at : 8u;
  j.done = wg0 + (j.whole ? 0u : at == 0u ? level : j.first - level);
  return j;
}

// The workspace: arrival counters (zero between calls), then statistics, partial sums, scores.
struct Layout {
  uint32_t groups;
  bool join;  // room for the pieces of cut units
  int64_t head_tiles, score_stride;
  size_t done, stats, final_stats, part, scores, total;
};
inline Layout layout_of(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t max_len, bool weights) {
  Layout w{};
  w.head_tiles = (q_heads / kv_heads + kHeadTile - 1) / kHeadTile;
  w.score_stride = (max_len + kTile - 1) / kTile * kTile;
  const int64_t units = B * kv_heads * w.head_tiles;
  const int64_t grains = max_len == 0 ? 1 : (max_len + kTile * kGrain - 1) / (kTile * kGrain);
  const uint32_t most = groups_of(D, false);
  w.groups = units > most || units * grains > most ? most : (uint32_t)(units * grains);
  w.join = grains > 1;  // (counted_change keeps units of one grain whole)
  // The counters take the same place whatever the sizes, so that no other
  // call's data ever lies where a call expects zeros.
  w.done = 0;
  w.stats = w.join || weights ? (size_t)kGroups * 4 : 0;
  w.final_stats = w.stats + (w.join ? (size_t)w.groups * 2 * kHeadTile * 8 : 0);
  w.part = w.final_stats + (weights ? ((size_t)(B * q_heads) * 8 + 15) / 16 * 16 : 0);
  w.scores = w.part + (w.join ? (size_t)w.groups * 2 * kHeadTile * (size_t)D * 4 : 0);
  w.total = w.scores + (weights ? (size_t)(B * q_heads) * (size_t)w.score_stride * 4 : 0);
  return w;
}

}  // namespace fp4
