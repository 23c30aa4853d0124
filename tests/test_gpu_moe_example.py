"""examples/moe_decode.py without drafts: one token a step, drawn from the head's logits."""
import numpy as np
import pytest

import layer_reference as ref
from gpu_helpers import say, to_host
from test_gpu_moe_layer import _example

pytestmark = pytest.mark.gpu


def test_loop_without_drafts():
    say("speculative example without drafts")
    history = _example().run(steps=6, drafts=0)
    assert len(history) == 6
    for i, h in enumerate(history):
        assert h["draft"] is None and h["tokens"].shape == (4, 0) and h["chance"].shape == (4, 0)
        assert (to_host(h["lens"]) == 40 + i).all() and not to_host(h["kept"]).any()
        target, u, t, out = (to_host(h[n]) for n in ("target", "u", "temperature", "out"))
        for b in range(4):
            want = ref.verify(target[b].astype(np.float64), None, np.zeros(0, np.int64), u[b].astype(np.float64), float(t[b]))
            assert out[b].tolist() == want[0]
