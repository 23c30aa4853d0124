// Replays on the host how fp4_attn_decode cuts a call into shares (the
// arithmetic of csrc/attn_split.h, which the kernel and the host compile too)
// and checks what the kernel relies on.  For tests/test_attn_split.py.
#include "attn_split.h"

#include <algorithm>
#include <cstdio>
#include <vector>

namespace {
struct Unit {
  uint64_t begin;  // where its counted tiles begin
  uint32_t counted;
};
}  // namespace

// 0, or -1 with the fault in `msg`.  seen: {change counted, cut units, most pieces of a unit, share}.
extern "C" int attn_split_check(int64_t B, int64_t kv_heads, int64_t group, int64_t D, int64_t row_bytes, int exact,
                                int64_t max_len, int64_t window, const int32_t* lens, int weights, uint32_t* seen,
                                size_t* total_bytes, char* msg, size_t msg_bytes) {
  using namespace fp4;
#define FAULT(...) return std::snprintf(msg, msg_bytes, __VA_ARGS__), -1
  const int64_t q_heads = kv_heads * group;
  const Layout w = layout_of(B, q_heads, kv_heads, D, max_len, weights != 0);
  *total_bytes = w.total;
  const uint32_t grid = std::min(w.groups, groups_of(D, exact != 0));
  const uint64_t heads = (uint64_t)kv_heads * (uint64_t)w.head_tiles;

  // Every array of the workspace lies behind the one before it, wherever one is needed.
  const size_t places = (size_t)w.groups * 2 * kHeadTile;
  const size_t join_stats = w.join ? places * 8 : 0, join_part = w.join ? places * (size_t)D * 4 : 0;
  const size_t final_stats = weights ? (size_t)(B * q_heads) * 8 : 0;
  if ((w.join || weights) && w.stats < w.done + kGroups * 4) FAULT("statistics on the counters");
  if (w.final_stats < w.stats + join_stats || w.part < w.final_stats + final_stats || w.scores < w.part + join_part ||
      w.total < w.scores + (weights ? (size_t)(B * q_heads) * (size_t)w.score_stride * 4 : 0))
    FAULT("overlapping arrays");
  if ((w.stats | w.final_stats | w.part | w.scores) % 16 != 0) FAULT("an array that is not aligned");
  if (weights && w.score_stride < max_len) FAULT("scores shorter than max_len");

  // The sequences' tiles and the shares, as share_of finds them.
  std::vector<uint32_t> tiles((size_t)B);
  uint64_t sum = 0;
  for (int64_t b = 0; b < B; ++b) {
    const int64_t len = std::clamp<int64_t>(lens[b], 0, max_len);
    const int64_t first = window > 0 && window < len ? len - window : 0;
    tiles[(size_t)b] = (uint32_t)((len + kTile - 1) / kTile - first / kTile);
    sum += counted_tiles(tiles[(size_t)b], 0u);
  }
  if (sum * heads > 0xFFFFFFFFull) FAULT("tiles past 32 bits");
  uint32_t share = share_tiles((uint32_t)(sum * heads), grid);
  const uint32_t more = counted_change(share, change_tiles((uint32_t)row_bytes), w.join);
  if (more > 0u) {
    sum += (uint64_t)more * (uint64_t)B;
    if (sum * heads > 0xFFFFFFFFull) FAULT("counted tiles past 32 bits");
    share = share_tiles((uint32_t)(sum * heads), grid);
  }
  const uint64_t total = sum * heads;
  seen[0] = more;
  seen[1] = seen[2] = 0;
  seen[3] = share;
  if ((uint64_t)share * grid < total) FAULT("shares that do not hold all tiles");

  std::vector<Unit> units;
  units.reserve((size_t)((uint64_t)B * heads));
  uint64_t at = 0;
  for (int64_t b = 0; b < B; ++b)
    for (uint64_t h = 0; h < heads; ++h) {
      units.push_back({at, counted_tiles(tiles[(size_t)b], more)});
      at += units.back().counted;
    }

  // The workgroups' pieces in turn: together they are every unit once.
  std::vector<uint8_t> place_used(places / kHeadTile, 0), counter_used(kGroups, 0);
  size_t u = 0;
  uint32_t met = 0, done_tiles = 0;  // of unit u
  for (uint32_t wg = 0; wg < grid; ++wg) {
    uint64_t pos = std::min<uint64_t>((uint64_t)wg * share, total);
    const uint64_t end = pos + std::min<uint64_t>(share, total - pos);
    while (pos < end) {
      if (u >= units.size()) FAULT("workgroup %u goes past the last unit", wg);
      const Unit& x = units[u];
      const Cut c = cut_at((uint32_t)pos, (uint32_t)end, (uint32_t)x.begin, x.counted, share);
      if (c.t_begin != done_tiles || c.t_end <= c.t_begin || c.t_end > x.counted)
        FAULT("unit %zu: tiles %u to %u after %u", u, c.t_begin, c.t_end, done_tiles);
      if (c.wg0 + met != wg || met >= c.pieces)
        FAULT("unit %zu: piece %u of %u in workgroup %u, the first in %u", u, met, c.pieces, wg, c.wg0);
      if ((c.t_begin == 0u) != (met == 0u)) FAULT("unit %zu: which piece is its first", u);
      if (c.pieces > 1u) {
        if (!w.join) FAULT("unit %zu is cut, the workspace has no room for its pieces", u);
        const uint32_t place = place_of(c.wg0, met);
        if (place % kHeadTile != 0u || place / kHeadTile >= place_used.size())
          FAULT("unit %zu: place %u of %zu", u, place, places);
        if (place_used[place / kHeadTile]++) FAULT("unit %zu: place %u taken twice", u, place);
      }
      pos += c.t_end - c.t_begin;
      done_tiles = c.t_end;
      ++met;
      if (done_tiles != x.counted) continue;
      if (met != c.pieces) FAULT("unit %zu: %u pieces, %u counted", u, met, c.pieces);
      seen[2] = std::max(seen[2], c.pieces);
      if (c.pieces > 1u) {
        ++seen[1];
        // The joins, level by level: each its own counter, and in the end one of all.
        uint32_t step = 1u, left = c.pieces;
        for (uint32_t level = 1u;; ++level, step *= 8u, left = (left + 7u) / 8u) {
          const bool last = join_of(c.wg0, 0u, step, left, level).whole;
          uint32_t arrivals = 0u;
          for (uint32_t p = 0u; p < c.pieces;) {
            const Join j = join_of(c.wg0, p, step, left, level);
            if (j.whole != last || j.n == 0u || j.n > (last ? kDirect : 8u) || j.first != p)
              FAULT("unit %zu: level %u joins %u from %u", u, level, j.n, j.first);
            if (j.first + (uint64_t)(j.n - 1u) * step >= c.pieces) FAULT("unit %zu: a join past its pieces", u);
            for (uint32_t i = 0u; i < j.n; ++i) {
              const Join o = join_of(c.wg0, j.first + i * step, step, left, level);
              if (o.first != j.first || o.n != j.n || o.done != j.done) FAULT("unit %zu: pieces disagree", u);
            }
            if (j.done >= grid || j.done >= kGroups) FAULT("unit %zu: counter %u", u, j.done);
            if (counter_used[j.done]++) FAULT("unit %zu: counter %u taken twice", u, j.done);
            arrivals += j.n;
            p = last ? c.pieces : j.first + 8u * step;
          }
          if (arrivals != left) FAULT("unit %zu: level %u joins %u of %u", u, level, arrivals, left);
          if (last) break;
        }
      }
      ++u;
      met = done_tiles = 0u;
    }
  }
  if (u != units.size()) FAULT("%zu of %zu units", u, units.size());
  return 0;
}
