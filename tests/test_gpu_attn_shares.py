"""fp4_attn_decode over many sequences against FP64, with the tolerances of
test_gpu_attn_decode.py: many short sequences, whose units are never cut (the
workspace has no room for pieces), and shares in which the change of units is
counted (attn_share_cases.py; the CPU replay shows that the cases reach this)."""
import numpy as np
import pytest

import attn_share_cases as cases
import test_gpu_attn_decode as attn
from gpu_helpers import say, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weights", (False, True))
@pytest.mark.parametrize("case", cases.SHORT + cases.COUNTED, ids=lambda c: "%s-f32=%d-%dx%dx%dx%d-%d" % c)
def test_many_units(case, weights):
    fmt, f32, B, kv_heads, group, D, most = case
    lens = [int(n) for n in cases.lens_of(case)]
    attn.run_case(B + D, fmt, lens, kv_heads, group, D, 32, f32=f32, weights=weights)


def test_many_units_on_a_kept_workspace():
    """Short sequences by the hundred, counted shares and one long sequence in
    turn on one workspace: each call's bits are those of a workspace of its own,
    and the counters are zero after each."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    rng = np.random.default_rng(8)
    cache = attn.cache_of(attn.make(8, "bf16", 900, 8, 32, 128))
    calls = []
    for B, width, weights in ((264, 4, False), (80, 32, False), (193, 4, True), (1, 900, False), (97, 30, True)):
        table = to_dev(rng.integers(0, 900, (B, width)).astype(np.int32))
        lens = to_dev(rng.integers(0, width * 32 + 1, B).astype(np.int32))
        q = torch.randn((B, 16, 128), device="cuda").to(torch.bfloat16)
        w = torch.rand((B, 8, width * 32), device="cuda") if weights else None
        size = fp4.fp4_attn_decode_workspace(cache.struct, B, 16, width * 32, int(weights))

        def call(ws, q=q, t=table, n=lens, w=w):
            w_out = None if w is None else torch.zeros_like(w)
            out = fp4.decode_attention(q, cache, t, n, weights=w, weights_out=w_out, ws=ws)
            return [out] + ([] if w is None else [w_out])
        calls.append((size, call))
    say("attention of many units, workspaces of their own")
    want = [f(None) for _, f in calls]
    torch.cuda.synchronize()
    ws = torch.zeros(max(n for n, _ in calls), dtype=torch.uint8, device="cuda")
    for i in list(range(len(calls))) * 2 + list(range(len(calls)))[::-1]:
        say("attention of many units, one workspace, call %d" % i)
        got = calls[i][1](ws)
        torch.cuda.synchronize()
        assert not ws[:2048].any(), i
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
