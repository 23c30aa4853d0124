"""The operators around a layer's products together: the speculative example, the
experts between routing and joining against FP64, the gradients of the whole
path, HIP graph capture and replay, streams, shared workspaces and debug mode."""
import importlib.util
import os

import numpy as np
import pytest

import layer_reference as ref
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUNDS = -9


def _example():
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("drafts", [0, 1, 3])
def test_example_loop(drafts):
    """Every step's tokens, counts and chances are those of its logits and random
    numbers in FP64 (chances: one rounding to FP32)."""
    say("speculative example, %d drafts" % drafts)
    history = _example().run(steps=6, drafts=drafts) if drafts else []
    kept = 0
    for h in history:
        a = {n: to_host(t) for n, t in h.items()}
        for b in range(len(a["kept"])):
            want = ref.verify(a["target"][b].astype(np.float64), a["draft"][b].astype(np.float64), a["tokens"][b],
                              a["u"][b].astype(np.float64), float(a["temperature"][b]))
            assert (a["out"][b].tolist(), a["kept"][b]) == (want[0], want[1])
            np.testing.assert_allclose(a["chance"][b], want[2], rtol=2.0 ** -23, atol=1e-37)
        kept += int(a["kept"].sum())
    if drafts == 3:
        assert kept > 0


def _experts(fp4, torch, E, N, K, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = [fp4.quantize(torch.randn((N, K), generator=g, device="cuda") * K ** -0.5, fmt) for _ in range(E)]
    ts = torch.cat([w.tensor_scale for w in q]) if fmt == fp4.NVFP4 else None
    deq = np.stack([to_host(fp4.dequantize(w, out_dtype=torch.float32)).astype(np.float64) for w in q])
    return torch.stack([w.codes for w in q]), torch.stack([w.scales for w in q]), ts, deq


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (37, 8, 2), (300, 5, 3)])
def test_experts_between_routing_and_joining(T, E, k, fmt):
    """sum_j w_j W_e x over the dequantised operands in FP64: the grouped GEMM's
    1e-5 of the sum of magnitudes, weights within 1e-6, top_k FMAs; tokens of no
    expert (padding) give 0 and change nothing else."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    say("experts %d x %d of %d, format %d" % (T, k, E, fmt))
    N, K = 64, 128
    codes, scales, ts, W = _experts(fp4, torch, E, N, K, fmt, T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x = fp4.quantize(torch.randn((T, K), generator=g, device="cuda"), fmt)
    xh = to_host(fp4.dequantize(x, out_dtype=torch.float32)).astype(np.float64)
    logits = torch.randn((T, E), generator=g, device="cuda")
    ids, w = fp4.moe_route(logits, k)
    pad = torch.arange(T, device="cuda") % 3 == 1
    for hole in (False, True):
        if hole:
            ids = torch.where(pad[:, None], -1, ids).contiguous()
        off, rows, pos = fp4.moe_sort(ids, E)
        y = fp4.gemm_grouped(x, rows, off, codes, scales, N, K, fmt, b_tensor_scale=ts, out_dtype=torch.float32)
        got = to_host(fp4.moe_combine(y, pos, w)).astype(np.float64)
        i, wh = to_host(ids), to_host(w).astype(np.float64)
        live = (i >= 0)[..., None]
        each = np.where(live, np.einsum("tknc,tc->tkn", W[np.maximum(i, 0)], xh), 0.0)
        mag = np.where(live, np.einsum("tknc,tc->tkn", np.abs(W[np.maximum(i, 0)]), np.abs(xh)), 0.0)
        bound = 1.2e-5 * (wh[..., None] * mag).sum(1)
        assert (np.abs(got - (wh[..., None] * each).sum(1)) <= bound).all()


def test_gradient_of_the_whole_path():
    """Of sum(g * combine(s_e * gather(x), route(logits))) with respect to x, s and
    the logits, against central differences of the same in FP64 (step 1e-6: 1e-9);
    FP32 sums of at most 64 terms: 1e-5 of the largest gradient."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    T, E, k, H = 5, 6, 3, 64
    rng = np.random.default_rng(8)
    x, s, logits, go = (rng.standard_normal(n) for n in ((T, H), (E,), (T, E), (T, H)))
    x, s, logits, go = (np.float32(a).astype(np.float64) for a in (x, s, logits, go))

    def loss(x, s, logits, renormalise):
        ids, w = ref.route(logits, k, renormalise)
        return (go[:, None] * w[..., None] * s[ids][..., None] * x[:, None]).sum()

    for renormalise in (True, False):
        say("gradient of routing, rows and joining, %d" % renormalise)
        dx, ds, dl = np.zeros_like(x), np.zeros_like(s), np.zeros_like(logits)
        for at, d in ((x, dx), (s, ds), (logits, dl)):
            for i in np.ndindex(at.shape):
                keep = at[i]
                at[i] = keep + 1e-6
                up = loss(x, s, logits, renormalise)
                at[i] = keep - 1e-6
                d[i] = (up - loss(x, s, logits, renormalise)) / 2e-6
                at[i] = keep
        tx, ts, tl, tg = (to_dev(a.astype(np.float32)) for a in (x, s, logits, go))
        ids, w = fp4.moe_route(tl, k, renormalise=renormalise)
        off, rows, pos = fp4.moe_sort(ids, E)
        xs = fp4.moe_gather(tx, pos)
        expert = torch.empty(T * k, dtype=torch.long, device="cuda")
        expert[pos.long().flatten()] = ids.long().flatten()
        scale = ts[expert][:, None]
        dy, dw = fp4.moe_combine_backward(tg, xs * scale, pos, w)
        got = [fp4.moe_combine(dy * scale, pos), torch.zeros(E, device="cuda").index_add_(0, expert, (dy * xs).sum(1)),
               fp4.moe_route_backward(tl, ids, dw, renormalise=renormalise)]
        for a, want in zip(got, (dx, ds, dl)):
            assert np.abs(to_host(a) - want).max() <= 1e-5 * np.abs(want).max() + 1e-8


def _setup(fp4, torch, seed=0, T=40):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"qkv": torch.randn((T, 12, 128), generator=g, device="cuda").to(torch.bfloat16),
         "pos": torch.randint(0, 100000, (3, T), generator=g, device="cuda").to(torch.int32),
         "wq": torch.rand(128, generator=g, device="cuda"), "wk": torch.rand(128, generator=g, device="cuda"),
         "logits": torch.randn((T, 60), generator=g, device="cuda"),
         "x": torch.randn((T, 256), generator=g, device="cuda").to(torch.bfloat16),
         "big": torch.randint(-1, 60, (2000, 4), generator=g, device="cuda").to(torch.int32),
         "target": torch.randn((5, 4, 20011), generator=g, device="cuda"),
         "draft": torch.randn((5, 3, 20011), generator=g, device="cuda"),
         "tokens": torch.randint(0, 20011, (5, 3), generator=g, device="cuda").to(torch.int32),
         "u": torch.rand((5, 4), generator=g, device="cuda")}
    freq = torch.pow(10000.0, -torch.arange(64, device="cuda") / 64).float()
    s["rope"] = fp4.Rope(freq, sections=(16, 24, 24), cyclic=True)
    s["temperature"] = torch.tensor([0.0, 0.5, 1.0, 2.0, 0.8], device="cuda")
    s["rope_ws"] = fp4.qk_norm_rope_workspace(T, 8, 2, 128)
    s["sort_ws"] = fp4.moe_sort_workspace(2000, 4, 60)
    s["verify_ws"] = fp4.verify_workspace(5, 3, 20011)
    return s


def _step(fp4, s, stream=None):
    q, k = s["qkv"][:, :8], s["qkv"][:, 8:10]
    a = dict(stream=stream)
    oq, ok = fp4.qk_norm_rope(q, k, s["rope"], s["pos"], s["wq"], s["wk"], **a)
    grads = fp4.qk_norm_rope_backward(oq, ok, q, k, s["rope"], s["pos"], s["wq"], s["wk"], ws=s["rope_ws"], **a)
    ids, w = fp4.moe_route(s["logits"], 6, **a)
    off, rows, pos = fp4.moe_sort(ids, 60, **a)
    y = fp4.moe_gather(s["x"], pos, **a)
    out = fp4.moe_combine(y, pos, w, **a)
    dy, dw = fp4.moe_combine_backward(out, y, pos, w, **a)
    dl = fp4.moe_route_backward(s["logits"], ids, dw, **a)
    many = fp4.moe_sort(s["big"], 60, ws=s["sort_ws"], **a)
    v = fp4.verify_drafts(s["target"], s["draft"], s["tokens"], s["u"], s["temperature"], ws=s["verify_ws"], **a)
    return [oq, ok, *grads, ids, w, off, rows, pos, y, out, dy, dw, dl, *many, *v]


def _change(torch, s, turn):
    g = torch.Generator(device="cuda").manual_seed(100 + turn)
    for n in ("qkv", "logits", "x", "target", "draft"):
        s[n].copy_(torch.randn(s[n].shape, generator=g, device="cuda"))
    s["u"].copy_(torch.rand(s["u"].shape, generator=g, device="cuda"))
    s["pos"].copy_(torch.randint(0, 100000, s["pos"].shape, generator=g, device="cuda"))
    s["big"].copy_(torch.randint(-1, 60, s["big"].shape, generator=g, device="cuda"))
    s["tokens"].copy_(torch.randint(0, 20011, s["tokens"].shape, generator=g, device="cuda"))


def test_graph_replay():
    """All of it captured in one graph; every replay, on changed inputs and with
    eager work on the same workspaces between, gives the eager calls' bits."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    s = _setup(fp4, torch)
    say("layer graph: eager warm-up")
    _step(fp4, s)
    torch.cuda.synchronize()
    say("layer graph: capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(fp4, s)
    for turn in range(4):
        _change(torch, s, turn)
        torch.cuda.synchronize()
        say("layer graph: replay %d" % turn)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = _step(fp4, s)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), "turn %d output %d" % (turn, i)


def test_on_another_stream():
    """Calls on a given stream: the same bits, ordered with that stream's work."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    s = _setup(fp4, torch, 2)
    want = [t.clone() for t in _step(fp4, s)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("layer on a side stream")
    side.wait_stream(torch.cuda.current_stream())
    got = _step(fp4, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), "output %d" % i


def test_two_calls_at_once():
    """Two streams with a workspace each: the bits of one call after the other."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    states = [_setup(fp4, torch, seed) for seed in (3, 4)]
    want = [[t.clone() for t in _step(fp4, s)] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    say("layer on two streams")
    got = []
    for _ in range(3):
        got = [_step(fp4, s, stream=st) for s, st in zip(states, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), "output %d" % i


def test_one_workspace_for_calls_of_all_sizes():
    """A workspace of the largest call serves smaller ones between, and is left as
    the next call needs it."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    ws = fp4.verify_workspace(64, 7, 50000)
    g = torch.Generator(device="cuda").manual_seed(5)
    say("verify: one workspace, several sizes")
    for B, G, V in ((64, 7, 50000), (1, 1, 100), (3, 0, 9000), (64, 7, 50000), (2, 4, 40000)):
        target = torch.randn((B, G + 1, V), generator=g, device="cuda").to(torch.bfloat16)
        tokens = target[:, :G].float().argmax(2).to(torch.int32)
        u = torch.rand((B, G + 1), generator=g, device="cuda")
        a = fp4.verify_drafts(target, None, tokens, u, ws=ws)
        b = fp4.verify_drafts(target, None, tokens, u)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_debug_mode_same_bits():
    import block_scaled_fp4_03_amd as fp4
    import torch
    outs = []
    prev = fp4.fp4_set_debug(0)
    try:
        for on in (1, 0):
            fp4.fp4_set_debug(on)
            say("debug mode %d: layer" % on)
            outs.append([t.clone() for t in _step(fp4, _setup(fp4, torch, seed=6))])
    finally:
        fp4.fp4_set_debug(prev)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_debug_mode_refuses_short_buffers():
    """Buffers of exactly what a call needs pass; for one row (or entry) more they are
    refused before any launch.  (hipMalloc'd, and no whole number of pages: what the
    larger call would touch is mapped memory all the same.)"""
    import block_scaled_fp4_03_amd as fp4
    import torch
    from test_gpu_debug import _Bufs
    bufs = _Bufs()
    prev = fp4.fp4_set_debug(1)
    st = torch.cuda.current_stream().cuda_stream
    try:
        n = 1000
        wide = [bufs(n * 64 * 4) for _ in range(3)]     # rows of 64 FP32
        few = [bufs(n * 8 * 4) for _ in range(2)]       # rows of 8
        words = [bufs(n * 4) for _ in range(3)]         # one an entry
        off, ws = bufs(64), bufs(1 << 20)
        say("debug: layer buffers that fit and do not")
        for rows, status in ((n, 0), (n + 1, BOUNDS)):
            assert fp4.fp4_qk_norm_rope(None, None, wide[0], 64, 1, None, 0, 0, 64, 0, None, None, 1e-6, wide[1], 64,
                                        None, 0, rows, st) == status
            assert fp4.fp4_qk_norm_rope_backward(None, None, wide[0], 64, None, 0, None, 64, 1, None, 0, 0, 64, 0, None,
                                                 None, 1e-6, wide[1], 64, None, 0, None, None, rows, None, 0,
                                                 st) == status
            assert fp4.fp4_moe_route(few[0], 0, 8, rows, 8, 1, 1, words[0], words[1], st) == status
            assert fp4.fp4_moe_route_backward(few[0], 0, 8, rows, 8, 1, 1, words[0], words[1], few[1], st) == status
            assert fp4.fp4_moe_sort(words[0], rows, 1, 8, off, words[1], words[2], ws, 1 << 20, st) == status
            assert fp4.fp4_moe_gather(wide[0], 0, 64, words[2], rows, 1, 64, n, wide[1], st) == status
            assert fp4.fp4_moe_combine(wide[0], 0, words[2], words[0], rows, 1, 64, n, wide[1], 64, st) == status
            assert fp4.fp4_moe_combine_backward(wide[0], 64, wide[1], 0, words[2], words[0], rows, 1, 64, n, wide[2],
                                                words[1], st) == status
            assert fp4.fp4_verify_drafts(wide[0], 0, 64 * n, None, 0, 0, 0, 1, 0, rows * 64, None, off, None, words[0],
                                         words[1], None, ws, 1 << 20, st) == status
        torch.cuda.synchronize()
    finally:
        fp4.fp4_set_debug(prev)
        bufs.free()


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 elements apart or into a tensor: the bits of dense copies."""
    import block_scaled_fp4_03_amd as fp4
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    big = torch.empty(6 << 30, dtype=torch.bfloat16, device="cuda")
    say("layer: heads 2^30 apart")
    qk = [torch.randn((6, h, 64), generator=g, device="cuda").to(torch.bfloat16) for h in (3, 2)]
    far = [big.as_strided((6, h, 64), ((1 << 30) - 8, 64, 1), at) for h, at in ((3, 0), (2, 4096))]
    for a, b in zip(far, qk):
        a.copy_(b)
    rope = fp4.Rope(torch.rand(32, generator=g, device="cuda"))
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    w = torch.rand(64, generator=g, device="cuda")
    want = fp4.qk_norm_rope(*qk, rope, pos, w, w)
    grads = fp4.qk_norm_rope_backward(*want, *qk, rope, pos, w, w)
    got = fp4.qk_norm_rope_backward(*want, *far, rope, pos, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    fp4.qk_norm_rope(*far, rope, pos, w, w, q_out=far[0], k_out=far[1])
    assert all(torch.equal(a, b) for a, b in zip(far, want))

    say("layer: rows beyond 2^32 elements")
    H = 4096
    y = big[:(big.numel() // H) * H].view(-1, H)
    rows = torch.tensor([[0, 1 << 20], [y.shape[0] - 1, (1 << 20) + 7]], device="cuda")
    x = torch.randn((2, H), generator=g, device="cuda").to(torch.bfloat16)
    wt = torch.rand((2, 2), generator=g, device="cuda")
    fp4.moe_gather(x, rows.to(torch.int32), out=y)
    assert torch.equal(y[rows], x[:, None].expand(2, 2, H))
    few = y[rows.flatten()].contiguous()
    at = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    out = fp4.moe_combine(few, at, wt)
    assert torch.equal(fp4.moe_combine(y, rows.to(torch.int32), wt), out)
    dfew, dw = fp4.moe_combine_backward(x, few, at, wt)
    assert torch.equal(fp4.moe_combine_backward(x, y, rows.to(torch.int32), wt, dy=torch.empty_like(y))[1], dw)

    say("layer: logits 2^31 apart")
    V = 5003
    target = torch.randn((2, 2, V), generator=g, device="cuda").to(torch.bfloat16)
    far = big.as_strided((2, 2, V), ((1 << 32) - 8191, (1 << 31) - 3, 1), 5)
    far.copy_(target)
    tokens = target[:, :1].float().argmax(2).to(torch.int32)
    u = torch.rand((2, 2), generator=g, device="cuda")
    a, b = (fp4.verify_drafts(t, None, tokens, u) for t in (target, far))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
