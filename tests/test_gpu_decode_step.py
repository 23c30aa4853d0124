"""The decode-step operators together: the example's loop, HIP graph capture
and replay, and debug mode."""
import importlib.util
import os

import numpy as np
import pytest

import decode_reference as ref
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUNDS = -9


def _example():
    spec = importlib.util.spec_from_file_location("decode_loop", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ("bf16", "mxfp8", "mxfp4"))
def test_example_loop(cache):
    """The loop runs past an eviction; what it reports about each step's logits
    agrees with them (FP64; 2e-5 covers V = 2048 additions of 2^-24 and the
    exponentials), and the chosen token is the first of the largest."""
    say("example loop, %s cache" % cache)
    h = _example().run(steps=24, cache=cache)
    assert len(h) == 24
    assert max(int(s["lens"].max()) for s in h[1:]) <= 96 + 16
    evicted = any((h[i + 1]["lens"] < h[i]["lens"]).any() for i in range(23))
    assert evicted
    for s in h:
        y = s["logits"].double().cpu().numpy()
        lp = ref.log_softmax(y)
        t = to_host(s["token"])
        np.testing.assert_array_equal(t, y.argmax(axis=1))
        np.testing.assert_allclose(to_host(s["logp"]), lp[np.arange(len(t)), t], rtol=2e-5, atol=2e-5)
        np.testing.assert_allclose(to_host(s["entropy"]), -(np.exp(lp) * lp).sum(axis=1), rtol=2e-5, atol=2e-5)


def _setup(fp4, torch, fmt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, G, D, page, width, V = 3, 2, 4, 64, 16, 40, 50021
    cache = fp4.KVCache.empty(2 * B * width, page, Hkv, D, fmt)
    perm = torch.randperm(2 * B * width, generator=g, device="cuda").to(torch.int32)
    s = {"cache": cache, "table": perm[:B * width].view(B, width).contiguous(),
         "table2": perm[B * width:].view(B, width).contiguous(),
         "lens": to_dev(np.array([600, 37, 513], np.int32)), "k": None}
    rows = int(to_host(s["lens"]).sum())
    s["seq"] = to_dev(np.repeat([0, 1, 2], to_host(s["lens"])).astype(np.int32))
    s["pos"] = to_dev(np.concatenate([np.arange(n) for n in to_host(s["lens"])]).astype(np.int32))
    s["k"] = torch.randn((rows, Hkv, D), generator=g, device="cuda")
    s["v"] = torch.randn((rows, Hkv, D), generator=g, device="cuda")
    s["q"] = torch.randn((B, Hkv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    s["w"] = torch.rand((B, Hkv, width * page), generator=g, device="cuda")
    s["w_out"] = torch.zeros_like(s["w"])
    s["x"] = torch.randn((B, V), generator=g, device="cuda")
    s["tok"] = torch.randint(0, V, (B, 2), generator=g, device="cuda", dtype=torch.int32)
    s["g"], s["ge"] = (torch.randn(n, generator=g, device="cuda") for n in ((B, 2), (B,)))
    s["ws"] = fp4.attention_workspace(cache, B, Hkv * G, width * page, weights=True)
    s["lp_ws"] = fp4.logprobs_workspace(B, V, 10)
    return s


def _step(fp4, s):
    import torch
    fp4.kv_append(s["cache"], s["k"], s["v"], s["table"], s["seq"], s["pos"])
    out = fp4.decode_attention(s["q"], s["cache"], s["table"], s["lens"], weights=s["w"], weights_out=s["w_out"],
                               ws=s["ws"])
    lens, w, kept = fp4.kv_evict(s["cache"], s["table"], s["lens"], s["w_out"], 200, 20, s["table2"])
    r = fp4.logprobs(s["x"], s["tok"], top_k=10, ws=s["lp_ws"])
    dx = fp4.logprobs_backward(s["x"], s["tok"], r.lse, s["g"], r.entropy, s["ge"])
    # (Bytes: pages that nothing was written to hold anything, NaN too.)
    pools = [t.view(torch.uint8) for t in (s["cache"].k, s["cache"].v, s["cache"].k_scales, s["cache"].v_scales)
             if t is not None]
    return [out, s["w_out"], lens, w, kept, r.logp, r.entropy, r.lse, r.top_logp, r.top_index, dx] + pools


@pytest.mark.parametrize("fmt", (0, 1, 2))
def test_graph_replay(fmt):
    """Append, attention with weights, eviction, log probabilities and their
    gradient captured in one graph; every replay, on changed inputs and with
    eager work between, gives the eager call's bits."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    s = _setup(fp4, torch, fmt)
    say("graph: eager warm-up, format %d" % fmt)
    _step(fp4, s)
    torch.cuda.synchronize()
    say("graph: capture")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(fp4, s)
    for turn in range(4):
        for name in ("k", "v", "x", "q"):
            s[name].copy_(torch.randn(s[name].shape, device="cuda"))
        s["w"].copy_(torch.rand(s["w"].shape, device="cuda"))
        torch.cuda.synchronize()
        say("graph: replay %d" % turn)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        want = _step(fp4, s)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), "turn %d output %d" % (turn, i)


def test_debug_mode_same_bits():
    import torch
    import block_scaled_fp4_03_amd as fp4
    outs = []
    prev = fp4.fp4_set_debug(0)
    try:
        for on in (1, 0):
            fp4.fp4_set_debug(on)
            say("debug mode %d: decode step" % on)
            outs.append([t.clone() for t in _step(fp4, _setup(fp4, torch, fp4.KV_MXFP8, seed=3))[:11]])
    finally:
        fp4.fp4_set_debug(prev)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_debug_mode_refuses_short_buffers():
    """Buffers past the end of their allocation: FP4_ERR_BOUNDS, before any launch.
    (Whole allocations of the caching allocator: large ones are their own.)"""
    import torch
    import block_scaled_fp4_03_amd as fp4
    prev = fp4.fp4_set_debug(1)
    st = torch.cuda.current_stream().cuda_stream
    try:
        # 32 MB tensors have an allocation of their own.
        big = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
        p, size = big.data_ptr(), big.numel()
        small = torch.zeros(1 << 16, dtype=torch.int32, device="cuda")
        z = small.data_ptr()

        def cache(pages):
            return fp4.KVCacheStruct(p, p, None, None, pages, 16, 1, 64, fp4.KV_BF16)

        fits = size // (16 * 64 * 2)
        say("debug: caches that fit and do not")
        for pages, status in ((fits, 0), (fits + 64, BOUNDS)):
            assert fp4.fp4_kv_append(cache(pages), z, z, 1, 64, 64, z, 4, 1, z, z, 1, st) == status
            assert fp4.fp4_attn_decode(cache(pages), z, 1, 64, z, 4, z, 1, 1, 64, 0, 1.0, z + 4096, 1, None, None,
                                       None, 0, z + 8192, 1 << 16, st) == status
            assert fp4.fp4_kv_evict(cache(pages), z, 4, z, z, 64, cache(pages), z + 256, 4, z + 512, z + 1024, 64,
                                    z + 2048, 1, 64, 8, 0, None, 0, st) == status
        say("debug: logits that fit and do not")
        V = size // 4
        lse = torch.zeros(1, device="cuda")
        out = torch.empty_like(big)
        need = fp4.fp4_logprobs_workspace(1, V + 1024, 0)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        for v, status in ((V, 0), (V + 1024, BOUNDS)):
            assert fp4.fp4_logprobs(p, 0, v, 1, v, 1.0, None, 0, None, None, lse.data_ptr(), 0, None, None,
                                    ws.data_ptr(), need, st) == status
            assert fp4.fp4_logprobs_backward(p, 0, v, 1, v, 1.0, None, 0, lse.data_ptr(), None, None, None,
                                             out.data_ptr(), v, st) == status
        torch.cuda.synchronize()
    finally:
        fp4.fp4_set_debug(prev)
