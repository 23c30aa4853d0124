"""Calls of fp4_attn_decode that reach what few or short sequences do not: the
CPU replay (test_attn_split.py) shows that they do, the GPU tests
(test_gpu_attn_shares.py) compare their results."""
import numpy as np

# (format, FP32 query and output, sequences, kv heads, query heads of one, head size, most tokens).
# Sequences of up to 128 tokens by the hundred: several units a workgroup, none
# cut, and a workspace without room for pieces (none at all without weights).
SHORT = [("bf16", False, 49, 32, 2, 128, 128), ("bf16", False, 97, 8, 4, 256, 128), ("bf16", False, 264, 8, 4, 128, 128),
         ("mxfp8", False, 449, 8, 2, 128, 100), ("mxfp4", False, 705, 8, 2, 128, 128), ("bf16", True, 193, 8, 3, 128, 97),
         ("mxfp8", True, 200, 16, 1, 64, 128)]
# Shares long enough that the change of units is counted, units that they cut.
COUNTED = [("bf16", False, 136, 8, 4, 64, 1024), ("bf16", False, 96, 8, 2, 128, 1000), ("mxfp8", False, 200, 8, 2, 128, 1300),
           ("mxfp4", False, 80, 8, 4, 256, 1100), ("mxfp8", False, 80, 8, 3, 192, 900), ("bf16", True, 72, 8, 2, 128, 700),
           ("mxfp4", True, 72, 8, 1, 256, 1100)]


def lens_of(case):
    """Ragged lengths: the longest among them, every eighth sequence empty."""
    B, most = case[2], case[6]
    lens = np.random.default_rng(B + most).integers(1, most + 1, B).astype(np.int32)
    lens[::8] = 0
    lens[B // 2] = most
    return lens
