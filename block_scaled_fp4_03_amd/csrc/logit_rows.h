// logit_rows.h -- a row of logits as 16-byte blocks, and which of them can be
// loaded whole.  The kernels of logprobs.hip and a CPU test
// (tests/test_logit_rows.py) compile this one source.  Internal header.
#pragma once

#include "host_device.h"

namespace fp4 {

// A row as 16-byte blocks from its first 128-byte line on: block j holds
// elements j E - head .. (the first blocks and the last may be partly or
// wholly outside the row).  Blocks are loaded whole, also those that reach into
// the rows beside, as long as they lie within the matrix; the first of its
// first rows and the last of its last may not.  (A wavefront's 1 KB is then
// eight whole lines.)
struct RowBlocks {
  uint32_t head, blocks;
  uint32_t lo, hi;  // blocks [lo, hi) can be loaded whole
};

// Row n of `rows`, its first element at address `at`, V elements of SIZE bytes.
template <uint32_t SIZE>
FP4_HOST_DEVICE RowBlocks row_blocks(uint64_t at, uint32_t n, uint32_t rows, uint32_t stride, uint32_t V) {
  constexpr uint32_t E = 16u / SIZE, kLine = 128u / SIZE;
  RowBlocks r;
  r.head = (uint32_t)(at & 127u) / SIZE;
  r.blocks = (V + r.head + E - 1u) / E;
  // Elements of the rows before this one, and of those behind it, as far as a
  // block can reach (each factor cut there first, so that products are small).
  const auto upto = [](uint32_t rows_, uint32_t stride_, uint32_t most) {
    const uint32_t x = (rows_ < most ? rows_ : most) * (stride_ < most ? stride_ : most);
    return x < most ? x : most;
  };
  const uint32_t before = upto(n, stride, kLine), after = upto(rows - 1u - n, stride, E);
  r.lo = r.head > before ? (r.head - before + E - 1u) / E : 0u;
  r.hi = r.blocks - (r.blocks * E - r.head - V > after ? 1u : 0u);  // what the last block has past the row
  return r;
}

}  // namespace fp4
