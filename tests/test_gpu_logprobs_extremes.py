"""fp4_logprobs on rows that hold a NaN at any place, against the definition."""
import numpy as np
import pytest

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
