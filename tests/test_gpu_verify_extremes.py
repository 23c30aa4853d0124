"""Verification of drafted tokens where the running sums' reference is at its limits,
against FP64 as in test_gpu_verify.py: tokens and counts equal, chances within 2^-23."""
import pytest

from gpu_helpers import say
from test_gpu_verify import _case, _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_logit_at_high_temperatures(dtype):
    """Temperatures whose steps of the reference are beyond FP32: a +inf logit behind a
    wave's first step, or at a row's edges, leaves no distribution all the same."""
    import torch
    inf, V = float("inf"), 8191
    s = _case(torch, 15, 3, V, dtype, 31)
    s["temperature"] = torch.tensor([1e36, 3e38, inf] * 5, device="cuda")
    for b in range(3):
        s["target"][b, 1, 8000] = inf
        s["draft"][3 + b, 1, 8000] = inf
        s["target"][6 + b, 3, 6000] = inf
        s["target"][9 + b, 2, 0] = inf
        s["draft"][9 + b, 0, V - 1] = inf
        s["target"][12 + b, b, V - 1] = inf
    say("verify, +inf at high temperatures %s" % dtype)
    kept = _check(s)
    assert kept.max() <= 3 and (kept[:6] <= 1).all()
