"""fp4_attn_decode where the values cancel: the output is near zero, so that its
own rounding to BF16 hides nothing of the probabilities' precision.

Five tokens; scores that are exact (queries with one element, keys and scale
powers of two apart from them); the last two values, as BF16, make the sum of
p_t V_t small twice over.  Error of an output, in u = 2^-24 times sum p |V|: a
score times log2 e (|x| < 3) 6, the exponential 2, the sum of probabilities and
its reciprocal 7 (of the output alone), five products of up to three terms each
in FP32, every addition rounding or truncating, 16: 31 in all, with the
output's own rounding 2^-8 |out|.  A BF16 cache takes the probabilities whole
(three BF16 terms hold FP32's 24 bits); in the MX formats two terms leave 2^-17
of each."""
import numpy as np
import pytest

import decode_reference as ref
import synth
from gpu_helpers import say, to_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bf16(x):
    return (synth.to_bf16_bits(np.asarray(x, np.float32)).astype(np.uint32) << 16).view(np.float32)


@pytest.mark.parametrize("D", (64, 128, 192, 256))
@pytest.mark.parametrize("f32", (False, True))
def test_cancelling_values(D, f32):
    import torch
    import block_scaled_fp4_03_amd as fp4
    B, H, T, page = 4, 64, 5, 16
    rng = np.random.default_rng(D)
    s = -rng.integers(0, 17, (B, H, T)) / 8.0                      # scores
    p = ref.softmax(s)
    V = np.zeros((B, H, T, D))
    V[:, :, :3] = _bf16(rng.uniform(0.5, 1.0, (B, H, 3, D)))
    for t in (3, 4):
        V[:, :, t] = _bf16(-(p[..., None] * V).sum(axis=2) / p[:, :, t, None])
    k = np.zeros((B, H, page, D), np.float32)
    k[:, :, :T, 5] = 8.0 * s
    v = np.zeros((B, H, page, D), np.float32)
    v[:, :, :T] = V
    q = np.zeros((B, H, D), np.float32)
    q[:, :, 5] = 1.0
    dt = torch.float32 if f32 else torch.bfloat16
    say("attention of cancelling values, D %d, f32 %d" % (D, f32))
    cache = fp4.KVCache(to_dev(synth.to_bf16_bits(k)), to_dev(synth.to_bf16_bits(v)))
    out = fp4.decode_attention(torch.from_numpy(q).cuda().to(dt), cache, to_dev(np.arange(B, dtype=np.int32)[:, None]),
                               to_dev(np.full(B, T, np.int32)), scale=0.125).double().cpu().numpy()
    want, size = (p[..., None] * V).sum(axis=2), (p[..., None] * np.abs(V)).sum(axis=2)
    assert np.abs(want).max() < 1e-3 * size.max()
    tol = 31 * U * size + (2 * U if f32 else 2.0 ** -8) * np.abs(want)
    off = np.abs(out - want) / tol
    worst = float(off.max())
    assert worst <= 1, "%d of %d outputs, up to %.3g of the tolerance" % ((off > 1).sum(), off.size, worst)
