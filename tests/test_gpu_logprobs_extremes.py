"""fp4_logprobs on rows that hold a NaN at any place, and on logits far from
zero, against the definition."""
import numpy as np
import pytest

import test_gpu_logprobs as lp
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu


def _order(x, k):
    """The top k indices of each row: NaN above all, then the values, ties to the lowest index; -1 past the row."""
    N, V = x.shape
    out = np.full((N, k), -1)
    for n in range(N):
        v = np.where(np.isnan(x[n]), 0.0, x[n])
        out[n, :min(k, V)] = np.lexsort((np.arange(V), -v, ~np.isnan(x[n])))[:k]
    return out


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("N,V,k", [(5, 9001, 4), (5, 3, 4), (5, 1, 2), (5, 40, 32), (600, 513, 8), (2, 60000, 32)])
def test_top_of_rows_with_nan(dtype, N, V, k):
    """A NaN in the first place, in all places, in the first and the last; one
    beside +inf; and an ordinary row."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    x = torch.randn((N, V), generator=torch.Generator().manual_seed(V)).numpy()
    kinds = [lambda r: r.__setitem__(0, np.nan), lambda r: r.fill(np.nan),
             lambda r: r.__setitem__([0, V - 1], np.nan), lambda r: r.__setitem__([0, V // 2], [np.inf, np.nan]),
             lambda r: None]
    for n in range(N):
        kinds[n % 5](x[n])
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    xd = torch.from_numpy(x).cuda().to(dt)
    vals = xd.float().cpu().numpy()
    say("logprobs of rows with NaN, %s N %d V %d k %d" % (dtype, N, V, k))
    r = fp4.logprobs(xd, to_dev(np.zeros((N, 1), np.int32)), top_k=k)
    np.testing.assert_array_equal(to_host(r.top_index), _order(vals, k))
    special = np.isnan(vals).any(axis=1) | np.isposinf(vals).any(axis=1)
    assert np.isnan(to_host(r.lse)[special]).all() and np.isfinite(to_host(r.lse)[~special]).all()
    top = to_host(r.top_logp)
    assert np.isnan(top[special][:, :min(k, V)]).all() and np.isneginf(top[:, V:]).all()
    assert np.isfinite(top[~special][:, :min(k, V)]).all()


@pytest.mark.parametrize("N,V", [(64, 50), (64, 1000), (9, 30011), (3, 200003), (600, 4100)])
@pytest.mark.parametrize("offset", (0.0, 100.0, -3000.0, 20000.0, -40000.0, 60000.0, 1e7))
def test_logits_with_a_common_offset(N, V, offset):
    """softmax does not change when all logits move by the same amount.  With
    scale 1 the differences of FP32 logits to their maximum lose nothing, so
    the entropy's tolerance is test_gpu_logprobs.py's without the terms of y's
    own size, and that of log-sum-exp has its last place's alone (u = 2^-24):
    r = (V / 256 + 72 + 2 E|t|) 2u; |dH| <= r (1 + 2 E|t|) + 4u (E t^2 + |H|);
    |d lse| <= r + 4u |lse|."""
    import block_scaled_fp4_03_amd as fp4
    U = 2.0 ** -24
    rng = np.random.default_rng(V)
    x = (3.0 * rng.standard_normal((N, V)) + offset).astype(np.float32)
    say("logprobs at %g, N %d V %d" % (offset, N, V))
    r = fp4.logprobs(to_dev(x), to_dev(np.zeros((N, 1), np.int32)))
    y = x.astype(np.float64)
    m = y.max(axis=1, keepdims=True)
    t = y - m
    e = np.exp(t)
    s = e.sum(axis=1)
    p = e / s[:, None]
    lse, et, et2 = m[:, 0] + np.log(s), (p * -t).sum(axis=1), (p * t * t).sum(axis=1)
    H = np.log(s) + et
    rel = (V / 256 + 72 + 2 * et) * 2 * U
    off = np.abs(to_host(r.lse) - lse) / (rel + 4 * U * np.abs(lse))
    offH = np.abs(to_host(r.entropy) - H) / (rel * (1 + 2 * et) + 4 * U * (et2 + np.abs(H)))
    assert off.max() <= 1 and offH.max() <= 1, "lse %.3g, entropy %.3g of the tolerance" % (off.max(), offH.max())


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_largest_and_smallest_scale(dtype):
    """2^127 on logits of 2^-126 and 2^-100 on logits of 2^100: the same softmax."""
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(3)
    for at, scale in ((-126, 2.0 ** 127), (101, 2.0 ** -100)):
        x = np.ldexp(rng.integers(-8, 9, (4, 3001)), at).astype(np.float32)
        xd, vals = lp._dev(x, dtype)
        tokens = rng.integers(0, 3001, (4, 2)).astype(np.int32)
        say("logprobs at scale %g, %s" % (scale, dtype))
        res = fp4.logprobs(xd, to_dev(tokens), top_k=5, scale=scale)
        lp.check_forward(vals, scale, tokens, res, 5, "scale %g" % scale)
