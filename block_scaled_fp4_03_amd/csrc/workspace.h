// workspace.h -- what lies where in a workspace (host arithmetic, for the launches, the
// size functions and the CPU test, tests/test_workspaces.py).
//
// Control words (arrival counters and the like, zero between calls) take the first
// kControlBytes, whichever operator has them, and nothing else lies there: so one
// zero-filled workspace serves calls of any operators and sizes in turn.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace fp4 {

constexpr size_t kControlBytes = 2048;

// ---- verification of drafts ----
constexpr int64_t kVerifyBatch = 256;     // sequences that a launch takes
constexpr int64_t kVerifyRowWaves = 4;    // waves, and parts, of a workgroup of the rows'
constexpr int64_t kVerifyMaxSplits = 32;  // workgroups of a row
constexpr int64_t kVerifyChunk = 512;     // tokens of a chunk
// Workgroups for the rows of a launch (64 x 15 rows of 100003 BF16: 3000 +6%, 960 +10%).
constexpr int64_t kVerifyWantedGroups = 2048;
constexpr size_t kVerifyPartBytes = 16, kVerifyChosenBytes = 32, kLineBytes = 128;

struct VerifyLayout {
  uint32_t splits, chunks;
  // Words between two sequences' row counters: as far apart as all of them go.  Adds to
  // one 128-byte line are made one after the other, 8 ns each.
  uint32_t counter_words;
  size_t drawn, chosen, sums, parts, total;  // bytes; the row counters come first
};
// n sequences (kVerifyBatch at most) of `rows` rows of V logits.
inline VerifyLayout verify_layout(int64_t n, int64_t rows, int64_t V) {
  VerifyLayout w{};
  // Enough workgroups for the chip, each with 4096 logits or more.
  const int64_t all = n * rows, wanted = (kVerifyWantedGroups + all - 1) / all;
  w.splits = (uint32_t)std::min({wanted, std::max<int64_t>(V / 4096, 1), kVerifyMaxSplits});
  w.chunks = (uint32_t)((V + kVerifyChunk - 1) / kVerifyChunk);
  w.counter_words = (uint32_t)(kControlBytes / 4);
  while ((size_t)n * w.counter_words > kControlBytes / 4) w.counter_words /= 2u;
  // A line of each sequence's counter of the draw; cleared by the first launch.
  w.drawn = kControlBytes;
  w.chosen = w.drawn + (size_t)n * kLineBytes;
  w.sums = w.chosen + (size_t)n * kVerifyChosenBytes;
  w.parts = w.sums + ((size_t)n * w.chunks * 8u + 15u) / 16u * 16u;
  w.total = w.parts + (size_t)(all * w.splits * kVerifyRowWaves) * kVerifyPartBytes;
  return w;
}
static_assert(kControlBytes / 4 >= kVerifyBatch, "a row counter of each sequence");
// What calls of up to n sequences, rows and logits take at most.  (The number of splits falls
// as rows are added, and with it all rows' parts, by less than what one split of each is.)
inline size_t verify_bytes(int64_t n, int64_t rows, int64_t V) {
  const int64_t all = n * rows, most = std::min(std::max<int64_t>(V / 4096, 1), kVerifyMaxSplits);
  const int64_t groups = std::min(all * most, all + kVerifyWantedGroups - 1);
  return verify_layout(n, rows, V).parts + (size_t)(groups * kVerifyRowWaves) * kVerifyPartBytes;
}

}  // namespace fp4
