"""fp4_logprobs and its gradient on matrices of a few bytes: rows shorter than
a 16-byte block at every alignment, dense and with gaps, forward and backward,
with the tolerances of test_gpu_logprobs.py."""
import numpy as np
import pytest

import test_gpu_logprobs as lp
from gpu_helpers import say, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("V", (1, 2, 3, 5, 6, 7, 9, 17, 40))
def test_small_matrices(dtype, V):
    import torch
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(V)
    for N in (1, 2, 3, 4, 13):
        for skip in (0, 1, 3):                       # elements before the matrix: its alignment
            for pad in (0, 1, 5):
                x = rng.standard_normal((N, V)).astype(np.float32)
                d, vals = lp._dev(x, dtype)
                flat = torch.full((skip + N * (V + pad),), float("nan"), dtype=d.dtype, device="cuda")
                xd = flat[skip:].view(N, V + pad)[:, :V]
                xd.copy_(d)
                tokens = rng.integers(0, V, (N, 2)).astype(np.int32)
                what = "small %s N %d V %d skip %d pad %d" % (dtype, N, V, skip, pad)
                say(what)
                res = fp4.logprobs(xd, to_dev(tokens), top_k=3)
                lp.check_forward(vals, 1.0, tokens, res, 3, what)
                g, ge = rng.standard_normal((N, 2)).astype(np.float32), rng.standard_normal(N).astype(np.float32)
                dx = fp4.logprobs_backward(xd, to_dev(tokens), res.lse, to_dev(g), res.entropy, to_dev(ge))
                lp.check_grad(vals, 1.0, tokens, g, ge, dx.double().cpu().numpy(), dtype, what)
