"""Scales that the decode-step calls take and refuse (CPU: argument checks).
They multiply it by log2 e in FP32: beyond 2^127 that is not finite, and a
difference of zero times it is NaN."""
import numpy as np
import pytest

import test_decode_abi as abi

L = abi.L
NAN, INF, BIG = float("nan"), float("inf"), float(np.nextafter(np.float32(2.0) ** 127, np.float32(np.inf)))


@pytest.mark.parametrize("scale", (BIG, 3e38, INF, NAN))
def test_refused(scale):
    assert abi.logprobs(scale=scale) == abi.SHAPE
    assert abi.backward(scale=scale) == abi.SHAPE
    assert abi.attn(abi.cache(), scale=scale) == abi.SHAPE
    assert abi.attn(abi.cache(), scale=-scale) == abi.SHAPE


@pytest.mark.parametrize("scale", (2.0 ** 127, 1e-40, 1.0))
def test_taken(scale):
    """(A missing workspace or pointer is then what stops the call.)"""
    assert abi.logprobs(scale=scale, x=None) == abi.NULL
    assert abi.backward(scale=scale, x=None) == abi.NULL
    for s in (scale, -scale, 0.0):
        assert abi.attn(abi.cache(), scale=s, q=None) == abi.NULL
