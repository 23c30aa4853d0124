"""Norms of queries and keys with rotary positions, and their gradient, against
FP64.

Forward, FP32: the sum of squares (chains of at most 16 FMAs and 5 levels) is
off by 21 steps of 2^-24 relative, its root by half of that, the reciprocal
root by 2^-23; two products, the rotation's product and FMA: 4 steps.  cos and
sin: the turn is rounded to FP32 (pi 2^-24 in the angle), the functions give 2
steps.  Together less than 11 + 2 + 4 + 4 + 4 = 25 steps of 2^-24 of |a| + |b|,
the pair's normed values: 1.5e-6; 2e-6 is taken.  At positions up to 2^31 the
FP64 angle, of up to 2^31 radians, is off by 2 roundings of 2^-53: 5e-7 more.
BF16 outputs add half a step, 2^-8 of the value.

Gradient, FP32: the same for the rotation and the factors, twice (the value and
the mean term): 4e-6 of the magnitudes' formula.  The weights' sums: chains of
at most 200 additions, 200 * 2^-24 = 1.2e-5, and the terms' 4e-6: 1.6e-5 of the
sum of magnitudes."""
import numpy as np
import pytest

import layer_reference as ref
from gpu_helpers import say, to_host

pytestmark = pytest.mark.gpu
FWD, BWD, SUMS = 2.5e-6, 4.5e-6, 1.6e-5


def _case(torch, n, hq, hk, D, dtype, R=None, sections=None, interleaved=False, cyclic=False, weights="qk", far=5000,
          seed=0, pad=0, freq=None):
    import block_scaled_fp4_03_amd as fp4
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    qkv = torch.randn((n, hq + 2 * hk + pad, D), generator=g, device="cuda").to(dt)
    s = {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "R": D if R is None else R}
    s["gq"] = torch.randn((n, hq, D), generator=g, device="cuda").to(dt)
    s["gk"] = torch.randn((n, hk, D), generator=g, device="cuda").to(dt)
    s["wq"], s["wk"] = (1.0 + 0.3 * torch.randn(D, generator=g, device="cuda") if c in weights else None for c in "qk")
    pairs = s["R"] // 2
    s["sections"] = sections or [pairs]
    if freq is None:
        freq = torch.pow(10000.0, -torch.arange(pairs, device="cuda") / max(pairs, 1)).float()
    s["freq"] = freq
    s["pos"] = torch.randint(-far, far, (len(s["sections"]), n), generator=g, device="cuda").to(torch.int32)
    s["rope"] = fp4.Rope(s["freq"], sections=sections, interleaved=interleaved, cyclic=cyclic) if pairs else None
    s["cs"] = ref.cos_sin(to_host(s["pos"]), to_host(s["freq"]), ref.axis_of_pairs(s["sections"], cyclic))
    s["interleaved"] = interleaved
    return s


def _f64(t):
    return None if t is None else to_host(t.float()).astype(np.float64)


def _check(got, want, mag, tol, dtype, what):
    bound = tol * mag + (0.0 if dtype == "f32" else 2.0 ** -8 * np.abs(want))
    bad = ~(np.abs(_f64(got) - want) <= bound)
    assert not bad.any(), "%s: %d of %d off, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[:3].tolist())


def _run(s, dtype, eps=1e-6):
    import block_scaled_fp4_03_amd as fp4
    q, k = fp4.qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"], eps=eps)
    back = fp4.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"], eps=eps)
    for i, (name, got) in enumerate((("q", q), ("k", k))):
        x, w, g = _f64(s[name]), _f64(s["w" + name]), _f64(s["g" + name])
        args = (eps, *s["cs"], s["R"], s["interleaved"])
        want = ref.norm_rope(x, w, *args)
        normed = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
        _check(got, want, ref.rotate_magnitude(normed, s["R"], s["interleaved"]), FWD, dtype, name)
        dx, dw, dmag, wmag = ref.norm_rope_grad(x, w, *args, g)
        _check(back[i], dx, dmag, BWD, dtype, "d" + name)
        if w is None:
            assert back[2 + i] is None
        else:
            _check(back[2 + i], dw, wmag, SUMS, "f32", "dw" + name)
    return (q, k) + back


SHAPES = [
    # rows, query heads, key heads, head_dim
    (1, 1, 1, 64), (1, 32, 8, 128), (3, 5, 1, 80), (7, 4, 4, 256), (33, 7, 2, 192), (2, 3, 2, 32), (5, 2, 1, 40),
    (600, 16, 2, 64), (131, 3, 3, 96), (4, 1, 0, 64), (4, 0, 3, 128), (9, 20, 4, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    import torch
    n, hq, hk, D = shape
    say("norm and rope %s %s" % (shape, dtype))
    for interleaved in (False, True):
        _run(_case(torch, n, hq, hk, D, dtype, interleaved=interleaved, seed=n + D), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(64, 32), (128, 16), (128, 8), (128, 120), (80, 40), (256, 64), (96, 0), (192, 176)])
def test_part_of_a_head(D, R, dtype):
    import torch
    say("norm and rope %d of %d %s" % (R, D, dtype))
    for interleaved in (False, True):
        _run(_case(torch, 17, 4, 2, D, dtype, R=R, interleaved=interleaved, seed=R), dtype)


@pytest.mark.parametrize("cyclic", [False, True])
@pytest.mark.parametrize("sections", [(16, 24, 24), (32, 32), (64, 0), (0, 0, 64), (1, 62, 1), (10, 20, 30, 4),
                                      (24, 20, 20)])
def test_axes(sections, cyclic):
    import torch
    say("norm and rope, sections %s cyclic %d" % (sections, cyclic))
    for interleaved in (False, True):
        for dtype in ("bf16", "f32"):
            _run(_case(torch, 21, 3, 1, 128, dtype, sections=sections, cyclic=cyclic, interleaved=interleaved), dtype)


@pytest.mark.parametrize("weights", ["q", "k", ""])
def test_without_weights(weights):
    import torch
    say("norm and rope, weights of %r" % weights)
    for dtype in ("bf16", "f32"):
        _run(_case(torch, 19, 6, 2, 128, dtype, weights=weights), dtype)


def test_far_positions():
    """Angles of positions up to 2^31: FP32 products would be off by whole turns."""
    import torch
    say("norm and rope, far positions")
    _run(_case(torch, 64, 2, 1, 128, "f32", far=2 ** 31 - 1), "f32")
    s = _case(torch, 2, 2, 1, 64, "f32")
    s["pos"] = torch.tensor([[2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    s["cs"] = ref.cos_sin(to_host(s["pos"]), to_host(s["freq"]), [0] * 32)
    _run(s, "f32")


def test_large_and_small_values():
    """Rows of zeros (eps alone), of tiny and of large values."""
    import torch
    say("norm and rope, scales of rows")
    s = _case(torch, 6, 2, 1, 64, "f32", pad=1)
    scale = torch.tensor([0.0, 1e-12, 1e-3, 1.0, 1e6, 1e17], device="cuda").view(6, 1, 1)
    s["q"], s["k"] = s["q"] * scale, s["k"] * scale
    _run(s, "f32", eps=1e-5)


def test_strides_and_in_place():
    """Rows of a wider matrix, outputs in place, in given strided tensors."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    say("norm and rope, in place and strided")
    for dtype in ("bf16", "f32"):
        s = _case(torch, 37, 5, 2, 128, dtype, pad=3)
        want = fp4.qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
        grads = fp4.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
        wide = torch.zeros((37, 11, 128), dtype=s["q"].dtype, device="cuda")
        got = fp4.qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"][0], s["wq"], s["wk"], q_out=wide[:, 1:6],
                               k_out=wide[:, 8:10])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not wide[:, [0, 6, 7, 10]].any()
        for target in ("g", ""):   # the gradient over the output's gradient, and over the input
            copy = {n: s[n].clone() for n in ("gq", "gk", "q", "k")}
            back = fp4.qk_norm_rope_backward(copy["gq"], copy["gk"], copy["q"], copy["k"], s["rope"], s["pos"],
                                             s["wq"], s["wk"], dq=copy[target + "q"], dk=copy[target + "k"])
            for a, b in zip(back, grads):
                assert torch.equal(a, b)
        rest = torch.ones_like(wide)
        rest[:, :5], rest[:, 5:7] = s["q"], s["k"]
        q, k = rest[:, :5], rest[:, 5:7]
        fp4.qk_norm_rope(q, k, s["rope"], s["pos"], s["wq"], s["wk"], q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and (rest[:, 7:] == 1).all()


def test_one_row_of_any_stride():
    """A single row's stride is no more than a number: an odd one is no obstacle."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    s = _case(torch, 1, 4, 2, 64, "bf16")
    want = fp4.qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
    q, k = (s[n].as_strided(s[n].shape, (777, 64, 1), s[n].storage_offset()) for n in "qk")
    got = fp4.qk_norm_rope(q, k, s["rope"], s["pos"], s["wq"], s["wk"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows():
    """No rows: empty outputs, and gradients of the weights that are 0."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    s = _case(torch, 0, 4, 2, 64, "bf16")
    q, k = fp4.qk_norm_rope(s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    junk = torch.full((64,), 7.0, device="cuda")
    del junk
    out = fp4.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
    assert not out[2].any() and not out[3].any()
    s = _case(torch, 3, 2, 0, 64, "bf16")
    out = fp4.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])
    assert out[2].any() and not out[3].any()


def test_refusals():
    import torch
    import block_scaled_fp4_03_amd as fp4
    s = _case(torch, 4, 2, 1, 64, "bf16")
    ok = (s["q"], s["k"], s["rope"], s["pos"], s["wq"], s["wk"])

    def bad(error, at, value):
        a = list(ok)
        a[at] = value
        with pytest.raises(error):
            fp4.qk_norm_rope(*a)

    bad(ValueError, 1, s["k"][:3])
    bad(TypeError, 1, s["k"].float())
    bad(ValueError, 0, s["q"].transpose(1, 2))
    bad(TypeError, 2, "rope")
    bad(TypeError, 3, s["pos"].long())
    bad(ValueError, 3, s["pos"][:, :3])
    bad(ValueError, 4, s["wq"][:32])
    bad(ValueError, 5, torch.ones(65, device="cuda"))
    bad(TypeError, 5, s["wk"].to(torch.bfloat16))
    with pytest.raises(ValueError):
        fp4.Rope(s["freq"][:30])
    with pytest.raises(ValueError):
        fp4.Rope(s["freq"], sections=(16, 15))
    with pytest.raises(fp4.Fp4Error):   # the rotated part is larger than the head
        fp4.qk_norm_rope(s["q"][..., :32].contiguous(), s["k"][..., :32].contiguous(), s["rope"], s["pos"])
    with pytest.raises(ValueError):
        fp4.qk_norm_rope_backward(s["gq"][:, :1], s["gk"], *ok)
