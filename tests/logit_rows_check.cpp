// csrc/logit_rows.h on the host, for tests/test_logit_rows.py.
#include "logit_rows.h"

// {head, blocks, lo, hi} of row n whose first element lies at byte `at`.
extern "C" void logit_row_blocks(uint32_t size, uint64_t at, uint32_t n, uint32_t rows, uint32_t stride, uint32_t V,
                                 uint32_t* out) {
  const fp4::RowBlocks r = size == 4u ? fp4::row_blocks<4>(at, n, rows, stride, V)
                                      : fp4::row_blocks<2>(at, n, rows, stride, V);
  out[0] = r.head;
  out[1] = r.blocks;
  out[2] = r.lo;
  out[3] = r.hi;
}
