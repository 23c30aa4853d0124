"""Verification of drafted tokens against FP64: tokens and counts equal, the
chances within 2^-23 relative (one rounding to FP32, and FP64 sums).  The seeds'
borders are 1e-9 apart at least with probability 1 - 1e-4 a draw; both sides sum
in FP64 (1e-13)."""
import numpy as np
import pytest

import layer_reference as ref
from gpu_helpers import say, to_host

pytestmark = pytest.mark.gpu


def _case(torch, B, G, V, dtype, seed=0, noise=0.4, draft=True, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    s = {"target": (scale * torch.randn((B, G + 1, V), generator=g, device="cuda")).to(dt)}
    y = s["target"][:, :G].float()
    s["draft"] = (y + noise * torch.randn(y.shape, generator=g, device="cuda")).to(dt) if draft else None
    s["temperature"] = 0.5 + torch.rand(B, generator=g, device="cuda")
    logits = (s["draft"] if draft else s["target"][:, :G]).float() / s["temperature"][:, None, None]
    race = torch.empty((B, G, V), device="cuda").exponential_(generator=g)
    s["tokens"] = (logits - torch.log(race)).argmax(2).to(torch.int32) if G else torch.zeros((B, 0), dtype=torch.int32,
                                                                                           device="cuda")
    s["u"] = torch.rand((B, G + 1), generator=g, device="cuda")
    return s


def _check(s, what=""):
    import block_scaled_fp4_03_amd as fp4
    out, kept, chance = fp4.verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["temperature"])
    out, kept, chance = to_host(out), to_host(kept), to_host(chance)
    host = {n: None if s[n] is None else to_host(s[n].float() if s[n].is_floating_point() else s[n]).astype(
        np.float64 if s[n].is_floating_point() else np.int64) for n in s}
    if host["temperature"] is None:
        host["temperature"] = np.ones(len(out))
    for b in range(len(out)):
        want = ref.verify(host["target"][b], None if s["draft"] is None else host["draft"][b], host["tokens"][b],
                          host["u"][b], host["temperature"][b])
        assert (out[b].tolist(), kept[b]) == (want[0], want[1]), "%s sequence %d" % (what, b)
        np.testing.assert_allclose(chance[b], want[2], rtol=2.0 ** -23, atol=1e-37, err_msg=what)
    return kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,G,V", [(1, 1, 1), (3, 2, 2), (5, 4, 17), (4, 3, 1000), (2, 4, 4096), (3, 5, 4097), (7, 7, 8191),
                                   (2, 1, 32768), (1, 4, 100003), (3, 8, 50021), (40, 3, 999), (1, 32, 513), (2, 0, 3001),
                                   (1, 3, 300001)])
def test_shapes(B, G, V, dtype):
    import torch
    kept = 0
    for seed in range(3):
        say("verify %d x %d of %d %s seed %d" % (B, G, V, dtype, seed))
        kept += int(_check(_case(torch, B, G, V, dtype, seed)).sum())
        _check(_case(torch, B, G, V, dtype, seed + 10, draft=False), "without draft logits")
    assert kept > 0 or G == 0


def test_more_sequences_than_a_launch_takes():
    import torch
    say("verify, 2300 sequences")
    for draft in (True, False):
        kept = _check(_case(torch, 2300, 1, 37, "bf16", 21, draft=draft))
        assert 0 < kept.sum() < 2300
    s = _case(torch, 1025, 2, 5003, "f32", 22, draft=False)
    s["temperature"] = None
    _check(s)


def test_every_outcome():
    """Over many sequences: none kept, some, all, and greedy ones of each."""
    import torch
    say("verify, outcomes")
    s = _case(torch, 200, 3, 50, "f32", 4, noise=1.0, scale=1.0)
    s["temperature"][::4] = 0.0
    best = s["target"][:, :3].argmax(2).to(torch.int32)
    s["tokens"][::8] = best[::8]
    s["tokens"][4::16, :2] = best[4::16, :2]
    kept = _check(s)
    assert set(kept.tolist()) == {0, 1, 2, 3} and set(kept[::4].tolist()) >= {0, 2, 3}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_temperatures(dtype):
    """0, negative and NaN: greedy; tiny, huge and infinite ones; none given."""
    import torch
    say("verify, temperatures %s" % dtype)
    s = _case(torch, 12, 3, 1003, dtype, 2)
    s["temperature"] = torch.tensor([0.0, -1.0, float("nan"), 1e-45, 1e-30, 1e-3, 0.05, 1.0, 40.0, 1e30, 3e38,
                                     float("inf")], device="cuda")
    s["target"][:, :, 5:9] = -float("inf")
    s["draft"][:, :, 7:12] = -float("inf")
    _check(s)
    s["temperature"] = None
    _check(s)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_without_a_distribution(dtype, draft):
    """NaN, +inf, and rows masked whole, of the target and the draft, sampled and
    greedy; tokens that are none."""
    import torch
    say("verify, rows without a distribution %s %d" % (dtype, draft))
    inf, nan = float("inf"), float("nan")
    s = _case(torch, 24, 3, 4099, dtype, 3, draft=draft, noise=0.0)
    s["u"] *= 0.5
    s["temperature"][12:] = 0.0
    s["tokens"][12:] = s["target"][12:, :3].float().argmax(2).to(torch.int32)
    for b in (0, 12):
        s["target"][b, 0, 4098] = nan
        s["target"][b + 1, 1, 0] = inf
        s["target"][b + 2, 3] = -inf
        s["target"][b + 3, 0] = -inf
        s["target"][b + 4, 2, :4000] = -inf
        s["target"][b + 5, 3, 4000:] = nan
        if draft:
            s["draft"][b + 6, 0, 17] = nan
            s["draft"][b + 7, 1] = -inf
            s["draft"][b + 8, 2, 4095] = inf
            s["draft"][b + 9, 0, 100:] = -inf
    s["tokens"][10, 1] = -1
    s["tokens"][11, 0] = 4099
    s["tokens"][22, 2] = 2 ** 31 - 1
    s["tokens"][23, 0] = -2 ** 31
    _check(s)


def test_masked_tokens_are_never_drawn():
    """u = 0 and u just below 1 with masked tokens at both ends, all but one masked, and
    the type's lowest value as a mask."""
    import torch
    say("verify, masked tokens")
    for mask in (-float("inf"), torch.finfo(torch.float32).min):
        s = _case(torch, 6, 2, 9001, "f32", 6)
        for t in (s["target"], s["draft"]):
            t[:, :, :300] = mask
            t[:, :, -300:] = mask
            t[4:, :, :-301] = mask
        s["tokens"][0] = 5          # q = p = 0: never kept
        s["tokens"][4:] = 9001 - 301
        s["u"][:, 2] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.0, 1.0 - 2.0 ** -24, 0.0, 1.0 - 2.0 ** -24])
        s["temperature"] = None
        _check(s)


def test_a_draft_like_the_target_is_kept():
    """p equal to q: kept at every u below 1; a draft's certain token that the target
    excludes: never."""
    import torch
    say("verify, equal distributions")
    s = _case(torch, 4, 5, 20011, "bf16", 7, noise=0.0)
    s["u"][:, :5] = 1.0 - 2.0 ** -24
    assert _check(s).tolist() == [5] * 4
    s = _case(torch, 3, 2, 301, "f32", 8, draft=False)
    for b in range(3):
        s["target"][b, 0, int(s["tokens"][b, 0])] = -float("inf")
    s["u"][:, 0] = 0.0
    assert _check(s).tolist() == [0] * 3


def test_far_logits():
    """Logits far from zero and from each other (the running reference moves)."""
    import torch
    say("verify, far logits")
    s = _case(torch, 4, 3, 30011, "f32", 9)
    ramp = torch.arange(30011, device="cuda") / 30011
    s["target"] += (1e4 * ramp) * torch.tensor([1.0, -1.0, 0.0, 0.0], device="cuda").view(4, 1, 1) + 1e5
    s["draft"] += (1e4 * ramp) * torch.tensor([1.0, -1.0, 0.0, 0.0], device="cuda").view(4, 1, 1) - 1e5
    s["target"][2] *= 1e30
    s["draft"][2] *= 1e30
    _check(s)


def test_strides():
    """Padded vocabularies, rows at odd offsets, draft logits stacked step by step, one
    draft row shared by all sequences."""
    import torch
    say("verify, strides")
    for dtype in ("bf16", "f32"):
        s = _case(torch, 5, 3, 2003, dtype, 11)
        want = {n: s[n] for n in s}
        pad = torch.zeros((5, 4, 2010), dtype=s["target"].dtype, device="cuda")
        pad[:, :, 3:2006] = s["target"]
        steps = s["draft"].transpose(0, 1).contiguous()
        t = dict(want, target=pad[:, :, 3:2006], draft=steps.transpose(0, 1))
        _check(t)
        t["draft"] = s["draft"][:1].expand(5, 3, 2003)
        _check(t)


def test_refusals():
    import torch
    import block_scaled_fp4_03_amd as fp4
    s = _case(torch, 2, 3, 100, "f32")
    ok = [s["target"], s["draft"], s["tokens"], s["u"], s["temperature"]]

    def bad(error, at, value):
        a = list(ok)
        a[at] = value
        with pytest.raises(error):
            fp4.verify_drafts(*a)

    bad(ValueError, 0, s["target"][:, :3])
    bad(ValueError, 0, s["target"][:1])
    bad(ValueError, 0, s["target"].transpose(1, 2).contiguous().transpose(1, 2))
    bad(TypeError, 1, s["draft"].to(torch.bfloat16))
    bad(ValueError, 1, s["draft"][:, :, :99])
    bad(TypeError, 2, s["tokens"].long())
    bad(ValueError, 3, s["u"][:, :3].contiguous())
    bad(TypeError, 3, s["u"].double())
    bad(ValueError, 4, s["temperature"][:1])
    with pytest.raises(fp4.Fp4Error):
        fp4.verify_drafts(*ok, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fp4.Fp4Error):
        fp4.verify_drafts(torch.zeros((1, 34, 8), device="cuda"), None,
                          torch.zeros((1, 33), dtype=torch.int32, device="cuda"), torch.zeros((1, 34), device="cuda"))
