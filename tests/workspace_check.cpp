// Checks on the host what csrc/workspace.h says of fp4_verify_drafts' workspace (the launch
// and its kernels use the same arithmetic).  For tests/test_workspaces.py.
#include "workspace.h"

#include <cstdio>
#include <vector>

extern "C" size_t control_bytes() { return fp4::kControlBytes; }

// 0, or -1 with the fault in `msg`; the bytes that n sequences of `rows` rows of V logits take in *total.
extern "C" int verify_layout_check(int64_t n, int64_t rows, int64_t V, size_t* total, char* msg, size_t msg_bytes) {
  using namespace fp4;
#define FAULT(...) return std::snprintf(msg, msg_bytes, __VA_ARGS__), -1
  const VerifyLayout w = verify_layout(n, rows, V);
  *total = w.total;
  if (w.counter_words < 1 || (size_t)(n - 1) * w.counter_words * 4 + 4 > kControlBytes)
    FAULT("row counters beyond the control words");
  if (w.drawn < kControlBytes) FAULT("the draw's counters on the control words");
  if (w.chosen < w.drawn + (size_t)n * kLineBytes || w.sums < w.chosen + (size_t)n * kVerifyChosenBytes ||
      w.parts < w.sums + (size_t)n * w.chunks * 8 ||
      w.total < w.parts + (size_t)(n * rows) * w.splits * kVerifyRowWaves * kVerifyPartBytes)
    FAULT("overlapping arrays");
  if (w.drawn % 4 != 0 || (w.chosen | w.sums) % 8 != 0 || w.parts % 16 != 0) FAULT("an array that is not aligned");
  if (w.splits < 1 || w.splits > kVerifyMaxSplits) FAULT("%u splits", w.splits);
  if ((int64_t)w.chunks * kVerifyChunk < V) FAULT("tokens of no chunk");
  return 0;
}
