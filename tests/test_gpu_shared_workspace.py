"""One zero-filled workspace of the largest size for calls of all operators that take one,
in any order: each call's bits are those of a workspace of its own, and the control
words are zero after it."""
import numpy as np
import pytest

from gpu_helpers import say, to_dev

pytestmark = pytest.mark.gpu
CONTROL_BYTES = 2048


def _calls(torch, fp4):
    """(name, workspace of its own, call of a workspace) of every operator, small and large."""
    g = torch.Generator(device="cuda").manual_seed(41)
    rng = np.random.default_rng(42)
    calls = []

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    cache = fp4.KVCache(randn(600, 2, 32, 64).to(torch.bfloat16), randn(600, 2, 32, 64).to(torch.bfloat16))
    for B, width, G in ((1, 100, 4), (200, 3, 2), (7, 60, 20)):
        table = to_dev(rng.integers(0, 600, (B, width)).astype(np.int32))
        lens = to_dev(rng.integers(0, width * 32 + 1, B).astype(np.int32))
        q = randn(B, 2 * G, 64).to(torch.bfloat16)
        calls.append(("attention of %d" % B, fp4.attention_workspace(cache, B, 2 * G, width * 32),
                      lambda ws, q=q, t=table, n=lens: [fp4.decode_attention(q, cache, t, n, ws=ws)]))
    for n, v in ((1, 60000), (300, 9000)):
        x, tok = randn(n, v), torch.zeros((n, 1), dtype=torch.int32, device="cuda")

        def logprobs(ws, x=x, tok=tok):
            r = fp4.logprobs(x, tok, top_k=20, ws=ws)
            return [r.logp, r.entropy, r.top_logp, r.top_index]
        calls.append(("log probabilities of %d" % n, fp4.logprobs_workspace(n, v, 20), logprobs))
    for B, G, V, draft in ((1, 4, 131072, True), (64, 7, 9001, True), (20, 2, 5003, False), (300, 1, 700, True),
                           (9, 3, 20011, False)):
        t = randn(B, G + 1, V)
        d = t[:, :G] + 0.3 * randn(B, G, V) if draft else None
        tokens = t[:, :G].argmax(2).to(torch.int32)
        u = torch.rand((B, G + 1), generator=g, device="cuda")
        temperature = 0.5 + torch.rand(B, generator=g, device="cuda")
        temperature[3::4] = 0.0
        calls.append(("verification of %d" % B, fp4.verify_workspace(B, G, V),
                      lambda ws, a=(t, d, tokens, u, temperature): list(fp4.verify_drafts(*a, ws=ws))))
    for T, k, E in ((4096, 4, 60), (600000, 1, 512)):
        ids = torch.randint(-1, E, (T, k), generator=g, device="cuda").to(torch.int32)
        calls.append(("sort of %d" % (T * k), fp4.moe_sort_workspace(T, k, E),
                      lambda ws, ids=ids, E=E: list(fp4.moe_sort(ids, E, ws=ws))))
    for rows, dim in ((3, 64), (2000, 128)):
        q, k, gq, gk = randn(rows, 4, dim), randn(rows, 2, dim), randn(rows, 4, dim), randn(rows, 2, dim)
        w = torch.rand(dim, generator=g, device="cuda")
        calls.append(("gradient of the norms of %d" % rows, fp4.qk_norm_rope_workspace(rows, 4, 2, dim),
                      lambda ws, a=(gq, gk, q, k, None, None, w, w): list(fp4.qk_norm_rope_backward(*a, ws=ws))))
    x = randn(32, 8192).to(torch.bfloat16)   # (the workgroups exchange the maximum)

    def quantize(ws):
        r = fp4.quantize(x, fp4.NVFP4, ws=ws)
        return [r.codes, r.scales, r.tensor_scale]
    calls.append(("NVFP4 quantisation", fp4.workspace(fp4.OP_QUANTIZE, fp4.NVFP4, 32, 0, 8192), quantize))
    return calls


def _largest(torch, calls):
    return torch.zeros(max(own.numel() for _, own, _ in calls if own is not None), dtype=torch.uint8, device="cuda")


def test_one_workspace_for_all_operators():
    import torch
    import block_scaled_fp4_03_amd as fp4
    calls = _calls(torch, fp4)
    want = []
    for name, own, call in calls:
        say("%s, a workspace of its own" % name)
        want.append([t.clone() for t in call(own)])
        torch.cuda.synchronize()
    ws = _largest(torch, calls)
    order = list(range(len(calls)))
    for turn in range(4):
        for i in order:
            say("%s, the shared workspace" % calls[i][0])
            got = calls[i][2](ws)
            assert not ws[:CONTROL_BYTES].any(), calls[i][0]
            for n, (a, b) in enumerate(zip(got, want[i])):
                assert torch.equal(a, b), "%s, output %d" % (calls[i][0], n)
        order = [order[::-1], order[::2] + order[1::2], order[::-1]][turn % 3]


def test_graphs_on_one_workspace():
    """Two graphs captured on one workspace and replayed in turn, with eager calls on it
    between: the eager calls' bits each time."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    calls = _calls(torch, fp4)
    want = [[t.clone() for t in call(own)] for _, own, call in calls]
    ws = _largest(torch, calls)
    torch.cuda.synchronize()
    graphs = []
    for part in (calls[::2], calls[1::2]):
        say("shared workspace: capture")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [call(ws) for _, _, call in part]
        graphs.append((graph, out))
    for turn in range(3):
        for half, (graph, out) in enumerate(graphs):
            say("shared workspace: replay %d of graph %d" % (turn, half))
            for r in out:
                for t in r:
                    t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for r, w in zip(out, want[half::2]):
                assert all(torch.equal(a, b) for a, b in zip(r, w))
            i = (5 * turn + half) % len(calls)
            assert all(torch.equal(a, b) for a, b in zip(calls[i][2](ws), want[i]))
            torch.cuda.synchronize()


def test_a_workspace_serves_smaller_calls():
    """Sizes where a smaller call has more counters or parts than the larger one that the
    workspace was made for."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    g = torch.Generator(device="cuda").manual_seed(43)
    ws = fp4.moe_sort_workspace(131072, 8, 128)
    for T in (131072, 65536, 2000):
        say("sort of %d, a larger call's workspace" % (T * 8))
        ids = torch.randint(-1, 128, (T, 8), generator=g, device="cuda").to(torch.int32)
        assert all(torch.equal(a, b) for a, b in zip(fp4.moe_sort(ids, 128, ws=ws), fp4.moe_sort(ids, 128)))
    ws = fp4.verify_workspace(64, 3, 131072)
    for B, G, draft in ((64, 3, True), (58, 3, True), (33, 2, False), (9, 1, True), (1, 0, False)):
        say("verification of %d, a larger call's workspace" % B)
        target = torch.randn((B, G + 1, 131072), generator=g, device="cuda").to(torch.bfloat16)
        d = target[:, :G] * 0.9 if draft else None
        tokens = target[:, :G].float().argmax(2).to(torch.int32)
        u = torch.rand((B, G + 1), generator=g, device="cuda")
        a, b = (fp4.verify_drafts(target, d, tokens, u, ws=w) for w in (ws, None))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
