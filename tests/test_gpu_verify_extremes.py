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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_terms_before_and_behind_a_move_of_the_reference(dtype):
    """Logits about 0, then some just short of 2^500 above, then some just past it: the
    last move the reference when the sum already holds terms as large as theirs."""
    import torch
    # (Rows in one piece: one step of a wave's is 4096 BF16 or 2048 FP32 logits.)
    B, G, V, step = (256, 7, 12300, 4096) if dtype == "bf16" else (5, 6, 8191, 2048)
    s = _case(torch, B, G, V, dtype, 32, draft=False)
    g = torch.Generator(device="cuda").manual_seed(33)
    s["target"] = -torch.rand((B, G + 1, V), generator=g, device="cuda")
    rest = s["target"].shape[:2] + (V - step - 8,)
    past = torch.arange(V - step - 8, device="cuda") >= step
    # 500 log 2 is 346.57; BF16 has the even numbers there.
    low, high = (346.0, 348.0) if dtype == "bf16" else (345.5, 346.8)
    s["target"][..., step + 8:] = torch.where(past, high, low) + 0.6 * torch.rand(rest, generator=g, device="cuda")
    s["target"] = s["target"].to(torch.float32 if dtype == "f32" else torch.bfloat16)
    s["temperature"] = None
    s["tokens"] = torch.randint(step + 8, V, (B, G), generator=g, device="cuda").to(torch.int32)
    say("verify, moves of the reference %s" % dtype)
    _check(s)


def test_lowest_logits_beside_masked_ones():
    """Rows, or their beginnings, of FP32's lowest value and -inf at a temperature that
    makes a step of the reference reach below that value."""
    import torch
    lowest, inf, V = torch.finfo(torch.float32).min, float("inf"), 8191
    s = _case(torch, 6, 3, V, "f32", 34, draft=False)
    for b, until in enumerate((V, V, 5000, 5000, 300, 5)):
        s["target"][b, :, :until] = lowest
        s["target"][b, :, :until:3] = -inf
    s["temperature"] = torch.tensor([1e30, 2e30] * 3, device="cuda")
    s["tokens"][:] = torch.tensor([1, 301, 8000], dtype=torch.int32, device="cuda")
    s["u"][:, :3] *= 2.0 ** -14
    say("verify, the lowest value beside -inf")
    kept = _check(s)
    assert (kept[:2] > 0).any()


def test_empty_batch():
    """No sequences: empty results (with a workspace allocated here, and without one)."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    say("verify, an empty batch")
    for draft in (True, False):
        s = _case(torch, 2, 3, 50, "bf16", 35, draft=draft)
        s = {n: None if t is None else t[:0] for n, t in s.items()}
        out, kept, chance = fp4.verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["temperature"])
        assert out.shape == (0, 4) and kept.shape == (0,) and chance.shape == (0, 3)
