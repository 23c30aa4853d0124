"""Routing to experts, the order by expert, rows there and back, and the
gradients, against FP64.

Weights: the exponent's difference is off by half a step of its size and the
exponential by one, sums of up to 512 positive terms by 512 / 16 + 4 steps, the
quotient by one: (|x| + 40) 2^-24 relative.  The gradient adds a mean of up to
512 terms: twice that, of the sum of magnitudes.
Joined rows: top_k FMAs, each off by 2^-24 of the sum of magnitudes.  Their
weights' gradients: a dot of H terms in chains of at most H / 64 + 16 FMAs."""
import numpy as np
import pytest

import layer_reference as ref
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


def _dt(torch, dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def _f64(t):
    return to_host(t.float()).astype(np.float64)


def _close(got, want, bound, dtype, what):
    bound = bound + (0.0 if dtype == "f32" else 2.0 ** -8 * np.abs(want))
    err = np.abs(_f64(got) - want)
    bad = ~((err <= bound) | (np.isnan(want) & np.isnan(_f64(got))))
    assert not bad.any(), "%s: %d of %d off, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[:3].tolist())


def _route(x, k, renormalise, dtype, what):
    import block_scaled_fp4_03_amd as fp4
    import torch
    ids, w = fp4.moe_route(x, k, renormalise=renormalise)
    xh = _f64(x)
    want_ids, want_w = ref.route(xh, k, renormalise)
    np.testing.assert_array_equal(to_host(ids), want_ids, err_msg=what)
    finite = np.where(np.isfinite(xh), np.abs(xh), 0.0).max(initial=0.0)
    tol = (2.0 * finite + 40.0) * STEP
    _close(w, want_w, tol * np.abs(want_w) + 1e-37, "f32", what)
    g = torch.randn(ids.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    dx = fp4.moe_route_backward(x, ids, g, renormalise=renormalise)
    if np.isnan(xh).any() or (xh == np.inf).any():
        return
    want, p, full = ref.route_grad(xh, want_ids, _f64(g), renormalise)
    mag = p * (np.abs(full) + (p * np.abs(full)).sum(1, keepdims=True))
    _close(dx, want, 2.0 * tol * mag + 1e-37, dtype, what + " gradient")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (1, 1, 1), (3, 4, 4), (16, 32, 4), (17, 60, 6), (33, 128, 8), (5, 160, 16),
                                   (257, 256, 8), (7, 512, 10), (64, 5, 1), (15, 16, 16), (2, 33, 3)])
def test_route(T, E, k, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + E)
    for renormalise in (True, False):
        say("route %d x %d top %d %s %d" % (T, E, k, dtype, renormalise))
        x = (2.0 * torch.randn((T, E), generator=g, device="cuda")).to(_dt(torch, dtype))
        _route(x, k, renormalise, dtype, "plain")
        # Many ties: the lowest expert first.
        _route(torch.round(x), k, renormalise, dtype, "ties")
        # Columns of a wider matrix, at an odd offset.
        wide = torch.randn((T, E + 7), generator=g, device="cuda").to(_dt(torch, dtype))
        _route(wide[:, 3:3 + E], k, renormalise, dtype, "strided")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_extremes(dtype):
    """Masked experts (-inf and the type's lowest value), rows of nothing else,
    infinities, NaN, zeros of both signs, large values."""
    import torch
    dt = _dt(torch, dtype)
    inf, low = float("inf"), torch.finfo(dt).min
    rows = [[1.0, -inf, 2.0, -inf, 0.5], [-inf] * 5, [-inf, 3.0, -inf, -inf, -inf], [low] * 5, [low, 1.0, low, 2.0, low],
            [0.0, -0.0, 0.0, -0.0, -1.0], [3e38, -3e38, 1e38, 3e38, 0.0], [1.0, inf, 0.0, -inf, 2.0],
            [1.0, float("nan"), 5.0, 2.0, 0.0], [float("nan")] * 5]
    for renormalise in (True, False):
        for k in (1, 3, 5):
            say("route extremes top %d %s %d" % (k, dtype, renormalise))
            for i, row in enumerate(rows):
                _route(torch.tensor([row], device="cuda").to(dt), k, renormalise, dtype, "row %d" % i)


def test_route_backward_ids():
    """Ids outside the experts count for nothing, one given twice counts twice."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    x = torch.randn((3, 6), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    ids = torch.tensor([[0, -1, 6], [2, 2, 5], [-7, 99, -1]], dtype=torch.int32, device="cuda")
    g = torch.randn((3, 3), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    for renormalise in (True, False):
        got = fp4.moe_route_backward(x, ids, g, renormalise=renormalise)
        want, p, full = ref.route_grad(_f64(x), to_host(ids), _f64(g), renormalise)
        _close(got, want, 60 * STEP * p * (np.abs(full) + (p * np.abs(full)).sum(1, keepdims=True)), "f32", "ids")


def _ids(T, k, E, seed, kind):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E // 2, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "holes":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.05] = E
        ids[rng.random((T, k)) < 0.05] = 2 ** 31 - 1
    return ids


@pytest.mark.parametrize("kind", ["random", "holes", "one", "none"])
@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (1, 4, 32), (16, 4, 32), (63, 1, 3), (65, 2, 512), (1000, 8, 128),
                                   (2048, 4, 60), (2049, 4, 60), (5000, 8, 256), (40000, 3, 512), (16384, 8, 128),
                                   (32769, 4, 37), (70001, 8, 512), (300007, 2, 3)])
def test_sort(T, k, E, kind):
    import block_scaled_fp4_03_amd as fp4
    say("sort %d x %d of %d, %s" % (T, k, E, kind))
    ids = _ids(T, k, E, T + E, kind)
    off, rows, pos = fp4.moe_sort(to_dev(ids), E)
    want = ref.sort(ids, E)
    for got, w, name in zip((off, rows, pos), want, ("group_off", "row_idx", "pos")):
        np.testing.assert_array_equal(to_host(got), w, err_msg=name)


ROWS = [(1, 1, 8), (1, 4, 2880), (3, 2, 64), (16, 4, 2880), (65, 8, 520), (200, 3, 1032), (37, 6, 4096), (2, 16, 16), (5, 64, 128),
        (300, 1, 72)]


@pytest.mark.parametrize("kind", ["random", "holes", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", ROWS)
def test_rows_there_and_back(T, k, H, dtype, kind):
    import block_scaled_fp4_03_amd as fp4
    import torch
    say("rows %d x %d of %d %s %s" % (T, k, H, dtype, kind))
    dt, E = _dt(torch, dtype), 9
    g = torch.Generator(device="cuda").manual_seed(T + H)
    pos = fp4.moe_sort(to_dev(_ids(T, k, E, T, kind)), E)[2]
    p = to_host(pos)
    r = np.where(p < 0, -1 - p, p)
    x = torch.randn((T, H + 16), generator=g, device="cuda").to(dt)[:, 8:8 + H]   # columns of a wider matrix
    rows = fp4.moe_gather(x, pos)
    want = np.zeros((T * k, H))
    want[r.reshape(-1)] = np.repeat(_f64(x), k, axis=0)
    np.testing.assert_array_equal(_f64(rows), want)

    y = torch.randn((T * k, H), generator=g, device="cuda").to(dt)
    w = torch.randn((T, k), generator=g, device="cuda")
    live = (p >= 0)[..., None]
    yh, wh = np.where(live, _f64(y)[r], 0.0), _f64(w)[..., None]
    for weights, wt in ((w, wh), (None, np.ones_like(wh))):
        out = torch.full((T, H + 8), 7.0, device="cuda").to(dt)
        got = fp4.moe_combine(y, pos, weights, out=out[:, :H])
        assert (out[:, H:] == 7.0).all()
        _close(got, (wt * yh).sum(1), (k + 1) * STEP * (np.abs(wt * yh)).sum(1), dtype, "combine")
        assert torch.equal(fp4.moe_combine(y, pos, weights), got)

    go = torch.randn((T, H + 8), generator=g, device="cuda").to(dt)[:, :H]
    dy, dw = fp4.moe_combine_backward(go, y, pos, w)
    gh = _f64(go)[:, None]
    want = np.zeros((T * k, H))
    want[r.reshape(-1)] = np.where(live, wh * gh, 0.0).reshape(T * k, H)
    _close(dy, want, STEP * np.abs(want), dtype, "dy")
    _close(dw, (gh * yh).sum(-1), (H / 64 + 32) * STEP * np.abs(gh * yh).sum(-1), "f32", "dw")


def test_rows_that_are_none():
    """Entries past the rows of y are skipped in every direction, and rows that
    no entry names stay as they were."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    pos = torch.tensor([[0, 5], [-6, 2147483647], [1, -2147483648]], dtype=torch.int32, device="cuda")
    x = torch.arange(3 * 8, device="cuda").view(3, 8).float()
    out = torch.full((3, 8), -1.0, device="cuda")
    fp4.moe_gather(x, pos, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[2]) and (out[2] == -1.0).all()
    w = torch.ones((3, 2), device="cuda")
    got = fp4.moe_combine(x, pos, w)
    assert torch.equal(got[0], x[0]) and not got[1].any() and torch.equal(got[2], x[1])
    dy = torch.full((3, 8), -1.0, device="cuda")
    fp4.moe_combine_backward(x, x, pos, w, dy=dy)
    assert torch.equal(dy[0], x[0]) and torch.equal(dy[1], x[2]) and (dy[2] == -1.0).all()


def test_no_tokens_no_rows():
    import block_scaled_fp4_03_amd as fp4
    import torch
    i32 = torch.int32
    x = torch.zeros((0, 64), device="cuda")
    assert fp4.moe_gather(x, torch.zeros((0, 4), dtype=i32, device="cuda")).shape == (0, 64)
    ids, w = fp4.moe_route(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    # Tokens without an entry, and without a row to read: zeros.
    assert not fp4.moe_combine(x, torch.zeros((5, 0), dtype=i32, device="cuda")).any()
    assert not fp4.moe_combine(x, torch.zeros((5, 2), dtype=i32, device="cuda")).any()
    off = fp4.moe_sort(torch.zeros((5, 0), dtype=i32, device="cuda"), 3)[0]
    assert off.tolist() == [0, 0, 0, 0]


def test_masked_values_stay_out():
    """NaN in rows that no entry names, and behind entries of no expert, reach nothing."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    ids = np.array([[0, -1], [-1, 1], [1, 0]], np.int32)
    pos = fp4.moe_sort(to_dev(ids), 2)[2]
    y = torch.ones((6, 16), device="cuda")
    y[4:] = float("nan")
    w = torch.full((3, 2), 2.0, device="cuda")
    w[0, 1] = w[1, 0] = float("nan")
    assert fp4.moe_combine(y, pos, w).tolist() == [[2.0] * 16] * 2 + [[4.0] * 16]
    dy, dw = fp4.moe_combine_backward(torch.ones((3, 16), device="cuda"), y, pos, w)
    assert dw.tolist() == [[16.0, 0.0], [0.0, 16.0], [16.0, 16.0]] and not dy[4:].any()


def test_refusals():
    import block_scaled_fp4_03_amd as fp4
    import torch
    i32 = torch.int32
    x = torch.zeros((4, 64), device="cuda")
    pos = torch.zeros((4, 2), dtype=i32, device="cuda")
    for k in (0, 17, -1):
        with pytest.raises(fp4.Fp4Error):
            fp4.moe_route(x, k)
    with pytest.raises(fp4.Fp4Error):
        fp4.moe_route(torch.zeros((4, 513), device="cuda"), 2)
    with pytest.raises(ValueError):
        fp4.moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        fp4.moe_route_backward(x, pos, torch.zeros((4, 3), device="cuda"))
    for e in (0, 513, -5):
        with pytest.raises(fp4.Fp4Error):
            fp4.moe_sort(pos, e)
    with pytest.raises(TypeError):
        fp4.moe_sort(pos.long(), 4)
    with pytest.raises(ValueError):
        fp4.moe_gather(x, pos[:3].contiguous())
    with pytest.raises(fp4.Fp4Error):
        fp4.moe_gather(torch.zeros((4, 60), device="cuda", dtype=torch.bfloat16), pos)
    with pytest.raises(ValueError):
        fp4.moe_gather(x, pos, out=torch.zeros((8, 32), device="cuda"))
    with pytest.raises(ValueError):
        fp4.moe_combine(x, pos, torch.zeros((4, 3), device="cuda"))
    with pytest.raises(TypeError):
        fp4.moe_combine(x, pos, torch.zeros((4, 2), device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fp4.moe_combine_backward(x[:3], x, pos, torch.zeros((4, 2), device="cuda"))
