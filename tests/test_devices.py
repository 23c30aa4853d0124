"""Calls on operands of a device that is not the current one (CPU: the library's calls and the
current device are stand-ins).  The null stream is the current device's, so that such a call
runs with the operands' device current and leaves the current one as it was."""
import contextlib

import pytest

import block_scaled_fp4_03_amd as fp4

torch = pytest.importorskip("torch")
CALLS = ("kv_append", "decode_attention", "kv_evict", "logprobs", "logprobs_backward", "qk_norm_rope",
         "qk_norm_rope_backward", "moe_route", "moe_route_backward", "moe_sort", "moe_gather", "moe_combine",
         "moe_combine_backward", "verify_drafts")


class OnDevice1(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 1)


class Stream:
    def __init__(self, raw, index):
        self.cuda_stream, self.device = raw, torch.device("cuda", index)


@pytest.fixture
def two_devices(monkeypatch):
    """(library function, stream, current device) of every call; the current device."""
    seen, current = [], [0]

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, args[-1], current[0]))
                return 0
            return call

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        try:
            yield
        finally:
            current[0] = before

    # The streams of device 1: its null stream, unless this is another.
    other = [0]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: other[0] if index == 1 else 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(fp4, "lib", Library)
    return seen, current, other


def tensor(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice1)


def calls():
    i32, bf16 = torch.int32, torch.bfloat16
    cache = fp4.KVCache(tensor(4, 2, 16, 64, dtype=bf16), tensor(4, 2, 16, 64, dtype=bf16))
    k, rows = tensor(3, 2, 64), tensor(3, dtype=i32)
    q, table = tensor(2, 4, 64), tensor(2, 2, dtype=i32)
    y, pos, g = tensor(8, 64), tensor(4, 2, dtype=i32), tensor(4, 64)
    return {
        "fp4_kv_append": lambda **a: fp4.kv_append(cache, k, k, table, rows, rows, **a),
        "fp4_attn_decode": lambda **a: fp4.decode_attention(q, cache, table, tensor(2, dtype=i32), out=tensor(2, 4, 64),
                                                            ws=tensor(1 << 16, dtype=torch.uint8), **a),
        "fp4_qk_norm_rope": lambda **a: fp4.qk_norm_rope(q, q, None, None, q_out=tensor(2, 4, 64),
                                                         k_out=tensor(2, 4, 64), **a),
        "fp4_moe_gather": lambda **a: fp4.moe_gather(g, pos, out=y, **a),
        "fp4_moe_combine": lambda **a: fp4.moe_combine(y, pos, out=g, **a)}


@pytest.mark.parametrize("name", ["fp4_kv_append", "fp4_attn_decode", "fp4_qk_norm_rope", "fp4_moe_gather",
                                  "fp4_moe_combine"])
def test_operands_of_another_device(two_devices, name):
    seen, current, other = two_devices
    call = calls()[name]
    call()                                   # device 1's null stream
    call(stream=Stream(0, 1))                # the same, given
    call(stream=Stream(0, 0))                # device 0's, for operands of device 1
    call(stream=Stream(77, 1))
    other[0] = 55
    call()                                   # a stream of device 1's own
    assert seen == [(name, 0, 1), (name, 0, 1), (name, 0, 0), (name, 77, 0), (name, 55, 0)]
    assert current == [0]
    other[0], current[0] = 0, 1
    del seen[:]
    call()
    assert seen == [(name, 0, 1)] and current == [1]


def test_an_error_leaves_the_current_device(two_devices, monkeypatch):
    class Refuses:
        def __getattr__(self, name):
            return lambda *args: b"FP4_ERR_SHAPE" if name == "fp4_status_string" else -2

    monkeypatch.setattr(fp4, "lib", Refuses)
    with pytest.raises(fp4.Fp4Error):
        calls()["fp4_moe_combine"]()
    assert two_devices[1] == [0]


def test_every_call_that_takes_a_stream_of_its_operands():
    """Those above stand for all: each goes through the same way to its stream."""
    for name in CALLS:
        assert hasattr(getattr(fp4, name), "__wrapped__"), name
