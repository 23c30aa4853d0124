"""fp4_logprobs and fp4_logprobs_backward on the GPU against FP64.

Tolerances (u = 2^-24, t_i = y_i - max y, E the mean under p).  y itself is
rounded (u |y|); e^t has relative error (|t| + |y| + 4) 2u; sums run in chains
of at most V / 256 + 64 additions, each u relative.  So with
  r = (V / 256 + 72 + 2 E|t| + 2 max|y|) 2u
lse is off by at most r + 4u |lse|, a log probability by that plus 4u (|y| +
|lse|), the entropy by r (1 + 2 E|t|) + 2u (E t^2 + |H|) 2.  The gradient's
p_i = e^(y_i - lse) has relative error (|y| + |lse| + |y - lse| + 6) 2u and
lse itself is FP32; g sums are of M terms; BF16 rounds the result (2^-8)."""
import numpy as np
import pytest

import decode_reference as ref
import synth
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _dev(x, dtype):
    """x (float32) on the device as f32 or bf16, and the values it then has."""
    if dtype == "f32":
        return to_dev(x), x
    b = synth.to_bf16_bits(x) if np.isfinite(x).all() else None
    import torch
    t = torch.from_numpy(x).cuda().to(torch.bfloat16) if b is None else to_dev(b)
    return t, t.float().cpu().numpy()


def _rows(x, dtype, stride):
    """The matrix with a row stride of its own, the gap filled with NaN."""
    import torch
    d, vals = _dev(x, dtype)
    if stride > x.shape[1]:
        wide = torch.full((x.shape[0], stride), float("nan"), dtype=d.dtype, device="cuda")
        wide[:, :x.shape[1]] = d
        d = wide[:, :x.shape[1]]
    return d, vals


def _bounds(y):
    """Per row: max, lse, p, entropy and the bound r."""
    V = y.shape[1]
    m = y.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        t = np.where(np.isneginf(y), -np.inf, y - m)
    e = np.exp(t)
    s = e.sum(axis=1, keepdims=True)
    p = e / s
    lse = (m + np.log(s))[:, 0]
    tf = np.where(p > 0, t, 0.0)
    Et, Et2 = (p * -tf).sum(axis=1), (p * tf * tf).sum(axis=1)
    H = np.log(s[:, 0]) + Et
    ymax = np.abs(np.where(p > 0, y, 0.0)).max(axis=1)
    r = (V / 256 + 72 + 2 * Et + 2 * ymax) * 2 * U
    return lse, H, r, Et, Et2


def check_forward(vals, scale, tokens, res, top_k, what):
    y = vals.astype(np.float64) * np.float64(np.float32(scale))
    N, V = y.shape
    lse, H, r, Et, Et2 = _bounds(y)
    got = to_host(res.lse)
    assert np.all(np.abs(got - lse) <= r + 4 * U * np.abs(lse)), what + " lse"
    tolH = r * (1 + 2 * Et) + 4 * U * (Et2 + np.abs(H))
    assert np.all(np.abs(to_host(res.entropy) - H) <= tolH), what + " entropy"
    lp = to_host(res.logp)
    for j in range(tokens.shape[1]):
        t = tokens[:, j]
        ok = (t >= 0) & (t < V)
        assert not lp[~ok, j].any()
        yt = y[np.arange(N), np.where(ok, t, 0)]
        with np.errstate(invalid="ignore"):
            bad = ok & ~np.where(np.isneginf(yt), np.isneginf(lp[:, j]),
                                 np.abs(lp[:, j] - (yt - lse)) <= r + 4 * U * (np.abs(yt) + np.abs(lse)))
        assert not bad.any(), what + " logp"
    if top_k:
        idx, tv = to_host(res.top_index), to_host(res.top_logp)
        k = min(top_k, V)
        want = np.argsort(-vals.astype(np.float64), axis=1, kind="stable")[:, :k]
        np.testing.assert_array_equal(idx[:, :k], want, err_msg=what + " top")
        assert np.all(idx[:, k:] == -1) and np.all(np.isneginf(tv[:, k:]))
        yt = np.take_along_axis(y, want, 1)
        with np.errstate(invalid="ignore"):
            bad = ~np.where(np.isneginf(yt), np.isneginf(tv[:, :k]),
                            np.abs(tv[:, :k] - (yt - lse[:, None])) <=
                            (r + 4 * U * np.abs(lse))[:, None] + 4 * U * np.abs(yt))
        assert not bad.any(), what + " top values"


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("N,V,M,k,pad,scale", [
    (1, 1, 1, 1, 0, 1.0), (1, 2, 1, 5, 1, 1.0), (3, 31, 2, 32, 0, 0.5), (2, 64, 0, 1, 3, 1.0), (5, 1000, 3, 20, 1, 1.0),
    (1, 4096, 1, 0, 0, 1.3), (7, 8193, 1, 32, 0, 1.0), (64, 513, 5, 8, 7, 2.0), (3, 50001, 1, 20, 0, 1.0),
    (1, 131072, 1, 20, 0, 1.0), (2, 200003, 4, 32, 5, 0.7), (300, 2049, 1, 5, 0, 1.0), (1, 1000003, 2, 8, 0, 1.0),
])
def test_logprobs(dtype, N, V, M, k, pad, scale):
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(V + N)
    x = (3.0 * rng.standard_normal((N, V))).astype(np.float32)
    xd, vals = _rows(x, dtype, V + pad)
    tokens = rng.integers(0, V, (N, M)).astype(np.int32)
    if M > 2:
        tokens[:, 1], tokens[0, 2] = -100, V
    what = "logprobs %s N %d V %d M %d k %d pad %d" % (dtype, N, V, M, k, pad)
    say(what)
    res = fp4.logprobs(xd, to_dev(tokens), top_k=k, scale=scale)
    check_forward(vals, scale, tokens, res, k, what)


def test_logprobs_more_rows_than_a_grid_holds():
    """70001 rows take two launches: every row's results and gradient."""
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(12)
    x = rng.standard_normal((70001, 9)).astype(np.float32)
    tokens = rng.integers(0, 9, (70001, 1)).astype(np.int32)
    say("logprobs of 70001 rows")
    res = fp4.logprobs(to_dev(x), to_dev(tokens), top_k=3)
    check_forward(x, 1.0, tokens, res, 3, "70001 rows")
    g = rng.standard_normal((70001, 1)).astype(np.float32)
    dx = to_host(fp4.logprobs_backward(to_dev(x), to_dev(tokens), res.lse, to_dev(g)))
    rows = np.r_[0:50, 65500:65600, 69951:70001]
    check_grad(x[rows], 1.0, tokens[rows], g[rows], None, dx[rows].astype(np.float64), "f32", "70001 rows")


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("kind", ["ascending", "descending", "equal", "ties", "peaked", "masked", "lowest", "one",
                                  "zeros", "large"])
def test_logprobs_orders_ties_and_masks(dtype, kind):
    """Rows on which a one-pass selection or sum could go wrong: sorted either
    way, all equal, few distinct values, one value holding all the mass, most
    logits -inf or the type's lowest value, +-0, large magnitudes."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    N, V, k = 3, 30011, 32
    rng = np.random.default_rng(4)
    low = float(torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min)
    x = rng.standard_normal((N, V)).astype(np.float32)
    if kind == "ascending":
        x = np.sort(x, axis=1)
    elif kind == "descending":
        x = -np.sort(-x, axis=1)
    elif kind == "equal":
        x[:] = 1.5
    elif kind == "ties":
        x = rng.integers(0, 3, (N, V)).astype(np.float32)
    elif kind == "peaked":
        x[:, 777] = 80.0
    elif kind == "masked":
        x[rng.random((N, V)) < 0.999] = -np.inf
    elif kind == "lowest":
        x[rng.random((N, V)) < 0.999] = low
        x[2] = low
    elif kind == "one":
        x[:] = -np.inf
        x[:, V - 1] = 3.0
    elif kind == "zeros":
        x = np.where(rng.random((N, V)) < 0.5, np.float32(-0.0), np.float32(0.0)).astype(np.float32)
    else:
        x *= 3000.0
    xd, vals = _rows(np.ascontiguousarray(x), dtype, V)
    tokens = np.stack([np.full(N, 777), np.full(N, V - 1)], 1).astype(np.int32)
    what = "logprobs %s %s" % (dtype, kind)
    say(what)
    res = fp4.logprobs(xd, to_dev(tokens), top_k=k)
    if kind == "zeros":
        vals = np.abs(vals)
    check_forward(vals, 1.0, tokens, res, k, what)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_logprobs_empty_rows_and_nan(dtype):
    """A row of -inf: lse -inf, logp -inf, entropy 0, the first indices on top;
    a NaN or +inf logit makes its row NaN and leaves the others alone."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    V, k = 9001, 4
    x = torch.randn((4, V), device="cuda")
    x[0] = -float("inf")
    x[1, 5000] = float("nan")
    x[2, 17] = float("inf")
    x = x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    tokens = to_dev(np.tile(np.array([[3, -1]], np.int32), (4, 1)))
    say("logprobs of empty and NaN rows, %s" % dtype)
    r = fp4.logprobs(x, tokens, top_k=k)
    lse, ent, lp, idx, top = (to_host(t) for t in (r.lse, r.entropy, r.logp, r.top_index, r.top_logp))
    assert lse[0] == -np.inf and ent[0] == 0 and lp[0, 0] == -np.inf and lp[0, 1] == 0
    np.testing.assert_array_equal(idx[0], [0, 1, 2, 3])
    assert np.all(top[0] == -np.inf)
    for n in (1, 2):
        assert np.isnan(lse[n]) and np.isnan(ent[n]) and np.isnan(lp[n, 0]) and lp[n, 1] == 0
        assert np.isnan(top[n]).all()
    assert idx[1, 0] == 5000 and idx[2, 0] == 17
    check_forward(x[3:].float().cpu().numpy(), 1.0, np.array([[3, -1]]),
                  fp4.LogProbs(r.logp[3:], r.entropy[3:], r.lse[3:], r.top_logp[3:], r.top_index[3:]), k, "last row")


def test_logprobs_repeats_and_streams():
    """One workspace, several shapes, a side stream: the same bits each time."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    x1, x2 = torch.randn((1, 70001), device="cuda"), torch.randn((3, 200000), device="cuda").to(torch.bfloat16)
    t1, t2 = (torch.zeros((n, 1), dtype=torch.int32, device="cuda") for n in (1, 3))
    sizes = [fp4.logprobs_workspace(1, 70001, 20), fp4.logprobs_workspace(3, 200000, 20)]
    ws = max((s for s in sizes if s is not None), key=lambda s: s.numel(), default=None)

    def both(stream=None):
        out = []
        for x, t in ((x1, t1), (x2, t2)):
            r = fp4.logprobs(x, t, top_k=20, ws=ws, stream=stream)
            out += [r.logp, r.entropy, r.lse, r.top_logp, r.top_index]
        return out

    say("logprobs, one workspace over several calls")
    want = both()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = both(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def check_grad(vals, scale, tokens, g, ge, dx, dtype, what):
    N, V = vals.shape
    sc = np.float64(np.float32(scale))
    for n in range(N):
        x = vals[n].astype(np.float64)
        gn, gen = g[n].astype(np.float64), 0.0 if ge is None else float(ge[n])
        want = ref.logprobs_grad(x, tokens[n], sc, gn, gen)
        y = sc * x
        lp = ref.log_softmax(y)
        p = np.exp(lp)
        lpf, yf = np.where(p > 0, lp, 0.0), np.where(p > 0, y, 0.0)
        lse = (yf - lpf)[p > 0][0]
        h = -(p * lpf).sum()
        ok = (tokens[n] >= 0) & (tokens[n] < V)
        gabs = np.abs(gn[ok]).sum()
        coef = np.abs(gn[ok].sum()) + np.abs(gen * (lpf + h))
        hot = np.zeros(V)
        np.add.at(hot, tokens[n][ok], np.abs(gn[ok]))
        tol = p * coef * (np.abs(yf) + abs(lse) + np.abs(lpf) + 6) * 4 * U
        tol += p * (gabs * (len(gn) + 4) + abs(gen) * (np.abs(yf) + abs(lse) + abs(h) + np.abs(lpf) + 4)) * 4 * U
        tol += hot * (len(gn) + 4) * 2 * U
        tol = sc * tol + np.abs(want) * (2.0 ** -8 if dtype == "bf16" else 4 * U)
        bad = ~(np.abs(dx[n] - want) <= tol + 1e-37)
        assert not bad.any(), "%s row %d: %d wrong, first at %s, off %g" % (
            what, n, bad.sum(), np.argwhere(bad)[:3].ravel(), np.abs(dx[n] - want).max())


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("N,V,M,ent,pad,scale", [
    (1, 1, 1, True, 0, 1.0), (2, 3, 2, True, 1, 1.0), (5, 1000, 1, False, 0, 1.0), (4, 1001, 4, True, 3, 0.5),
    (3, 33333, 1, True, 0, 1.0), (2, 70000, 8, True, 1, 2.0), (300, 513, 1, True, 0, 1.0), (1, 5000, 0, True, 0, 1.0),
    (2, 777, 100, True, 5, 1.0),
])
def test_logprobs_backward(dtype, N, V, M, ent, pad, scale):
    import torch
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(V + 13 * M)
    xd, vals = _rows((3.0 * rng.standard_normal((N, V))).astype(np.float32), dtype, V + pad)
    tokens = rng.integers(0, V, (N, M)).astype(np.int32)
    if M > 3:
        tokens[:, 1], tokens[0, 2], tokens[:, 3] = -100, V, tokens[:, 0]      # padding and a repeated token
    g, ge = rng.standard_normal((N, M)).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    what = "logprobs_backward %s N %d V %d M %d ent %d pad %d" % (dtype, N, V, M, ent, pad)
    say(what)
    fwd = fp4.logprobs(xd, to_dev(tokens), scale=scale)
    wide = torch.full((N, V + pad), -5.0, dtype=xd.dtype, device="cuda")
    dx = fp4.logprobs_backward(xd, to_dev(tokens), fwd.lse, to_dev(g), fwd.entropy if ent else None,
                               to_dev(ge) if ent else None, scale=scale, out=wide[:, :V])
    assert torch.all(wide[:, V:] == -5.0), "the gap between rows was written"
    check_grad(vals, scale, tokens, g, ge if ent else None, dx.float().cpu().numpy().astype(np.float64), dtype, what)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_logprobs_backward_masked_logits(dtype):
    """-inf and lowest-value logits get zero; a row of -inf gets zero but for its tokens' own terms."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    V = 3001
    low = float(torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min)
    x = torch.randn((3, V), device="cuda")
    x[0, ::2], x[1, 1::3], x[2] = -float("inf"), low, -float("inf")
    x = x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    tokens = to_dev(np.array([[1], [0], [-1]], np.int32))
    g = torch.ones((3, 1), device="cuda")
    ge = torch.full((3,), 0.5, device="cuda")
    say("logprobs_backward of masked logits, %s" % dtype)
    fwd = fp4.logprobs(x, tokens)
    dx = fp4.logprobs_backward(x, tokens, fwd.lse, g, fwd.entropy, ge).float().cpu().numpy()
    assert np.isfinite(dx).all()
    assert not dx[0, ::2].any() and not dx[1, 1::3].any() and not dx[2].any()
    check_grad(x[:2].float().cpu().numpy(), 1.0, np.array([[1], [0]]), np.ones((2, 1)), np.full(2, 0.5),
               dx[:2].astype(np.float64), dtype, "masked")


def test_logprobs_backward_against_differences():
    """The FP32 gradient against central differences of the FP64 loss.  With
    step d = 1e-4 the difference's own error is d^2/6 times the third
    derivative, at most (|g| + |ge| (log V + 3)) 8 d^2 scale^3, plus 1e-11 of
    rounding."""
    import block_scaled_fp4_03_amd as fp4
    V, scale, d = 37, 1.25, 1e-4
    rng = np.random.default_rng(6)
    x = rng.standard_normal((2, V)).astype(np.float32)
    tokens = np.array([[5, 5, 36], [0, -1, 7]], np.int32)
    g, ge = rng.standard_normal((2, 3)).astype(np.float32), rng.standard_normal(2).astype(np.float32)
    say("logprobs_backward against differences")
    fwd = fp4.logprobs(to_dev(x), to_dev(tokens), scale=scale)
    dx = to_host(fp4.logprobs_backward(to_dev(x), to_dev(tokens), fwd.lse, to_dev(g), fwd.entropy, to_dev(ge),
                                       scale=scale))
    for n in range(2):
        size = np.abs(g[n]).sum() + abs(ge[n]) * (np.log(V) + 3)
        for i in range(V):
            xp, xm = x[n].astype(np.float64), x[n].astype(np.float64)
            xp[i] += d
            xm[i] -= d
            diff = (ref.logprobs_loss(xp, tokens[n], scale, g[n], ge[n]) -
                    ref.logprobs_loss(xm, tokens[n], scale, g[n], ge[n])) / (2 * d)
            tol = 8 * d * d * scale ** 3 * size + 1e-11 / d + 64 * 2 * U * size * scale
            assert abs(dx[n, i] - diff) <= tol, (n, i, dx[n, i], diff)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("value", ["lowest", "largest", "half"])
def test_logprobs_of_equal_extreme_rows(dtype, value):
    """Whole rows of the type's lowest or largest value (times log2 e it is not
    finite), among ordinary ones, in rows that are not split and have no ragged
    step: lse = x + log V rounds to x, the entropy is log V (sums of ones are
    exact; the logarithm, the product and the difference round: 2^-20)."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    N, V = 520, 16384
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    big = torch.finfo(dt).min if value == "lowest" else torch.finfo(dt).max * (0.5 if value == "half" else 1.0)
    x = torch.randn((N, V), device="cuda").to(dt)
    x[::7] = big
    tokens = torch.full((N, 1), 5, dtype=torch.int32, device="cuda")
    say("logprobs of rows of %s %s" % (dtype, value))
    r = fp4.logprobs(x, tokens, top_k=4)
    torch.cuda.synchronize()
    assert torch.equal(r.lse[::7], torch.full_like(r.lse[::7], float(torch.tensor(big).to(dt).float())))
    assert ((r.entropy[::7] - np.log(V)).abs() <= 2.0 ** -20 * np.log(V)).all()
    assert torch.isfinite(r.lse).all() and torch.isfinite(r.entropy).all()
    assert torch.equal(r.top_index[::7].cpu(), torch.arange(4, dtype=torch.int32).expand(len(range(0, N, 7)), 4))
