"""How fp4_attn_decode cuts a call into workgroups' shares, and whether the
workspace that it asks for has room for what the cut units leave there (CPU:
csrc/attn_split.h, the source of both, in a host replay of the kernel's walk).

Checked of every call: each unit's tiles are taken once and in order; a unit is
cut only where the workspace has room for its pieces; every place and every
arrival counter lies within it and is used by one unit alone; the arrays do not
overlap; and the size is what the library asks for."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import attn_share_cases as cases
import block_scaled_fp4_03_amd as fp4

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_fp4_03_amd", "csrc")
FORMATS = {"bf16": (0, 2.0), "mxfp8": (1, 1.0), "mxfp4": (2, 0.5)}


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "attn_split_check.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "attn_split_check.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).attn_split_check
    I64, P = ctypes.c_int64, ctypes.c_void_p
    f.argtypes = [I64] * 5 + [ctypes.c_int, I64, I64, P, ctypes.c_int, P, P, ctypes.c_char_p, ctypes.c_size_t]
    if not os.path.exists(fp4.LIB_PATH):
        import block_scaled_fp4_03_amd.build as b
        b.build()

    def run(B, kv_heads, group, D, fmt, max_len, lens, exact=False, window=0, weights=False):
        code, width = FORMATS[fmt]
        lens = np.ascontiguousarray(lens, np.int32)
        assert lens.shape == (B,)
        seen, size, msg = (ctypes.c_uint32 * 4)(), ctypes.c_size_t(), ctypes.create_string_buffer(256)
        rc = f(B, kv_heads, group, D, int(D * width), exact, max_len, window, lens.ctypes.data, weights, seen,
               ctypes.byref(size), msg, 256)
        what = "B %d kv %d group %d D %d %s max_len %d exact %d window %d weights %d: " % (
            B, kv_heads, group, D, fmt, max_len, exact, window, weights)
        assert rc == 0, what + msg.value.decode()
        cache = fp4.KVCacheStruct(None, None, None, None, 0, 16, kv_heads, D, code)
        assert fp4.fp4_attn_decode_workspace(cache, B, kv_heads * group, max_len, int(weights)) == size.value, what
        return {"more": seen[0], "cut": seen[1], "pieces": seen[2], "share": seen[3]}

    return run


@pytest.mark.parametrize("B,kv_heads,D,fmt", [(49, 32, 128, "bf16"), (97, 8, 256, "bf16"), (193, 8, 128, "bf16"),
                                              (264, 8, 128, "bf16"), (449, 8, 128, "mxfp8"), (705, 8, 128, "mxfp4")])
def test_many_short_sequences_are_not_cut(replay, B, kv_heads, D, fmt):
    """Sequences of at most 128 tokens: the workspace has no room for pieces."""
    for weights in (False, True):
        got = replay(B, kv_heads, 4, D, fmt, 128, np.full(B, 128), weights=weights)
        assert got["cut"] == 0 and got["pieces"] == 1


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("D", (64, 128, 192, 256))
def test_short_calls(replay, fmt, D):
    """max_len up to 128 over batches to 2048 and 1 to 64 kv heads."""
    rng = np.random.default_rng(D)
    for kv_heads in (1, 2, 3, 8, 32, 64):
        for B in sorted(set([1, 2, 31, 64, 129, 2048] + [int(n) for n in rng.integers(1, 2049, 20)])):
            max_len = int(rng.choice([0, 1, 32, 33, 100, 128]))
            got = replay(B, kv_heads, int(rng.choice([1, 5, 16, 17, 40])), D, fmt, max_len,
                         rng.integers(-2, max_len + 2, B), exact=bool(rng.integers(2)), weights=bool(rng.integers(2)),
                         window=int(rng.choice([0, 0, 7])))
            assert got["cut"] == 0


@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("D", (64, 128, 192, 256))
def test_calls_of_all_lengths(replay, fmt, D):
    """Lengths mixed in every way: equal, ragged, mostly empty, one long one
    among short ones; shares with and without the change of units counted, and
    units in many pieces."""
    rng = np.random.default_rng(7 * D)
    counted = plain = most = 0
    for _ in range(400):
        B = int(round(np.exp(rng.uniform(0, np.log(2048)))))
        kv_heads, group = int(rng.choice([1, 2, 3, 8, 32, 64])), int(rng.choice([1, 4, 16, 17, 40]))
        max_len = int(round(np.exp(rng.uniform(np.log(100), np.log(200000)))))
        # (As fp4_attn_decode bounds it; a pass over the units stays short.)
        if (max_len // 32 + 32) * B * kv_heads * -(-group // 16) >= 1 << 32 or B * kv_heads > 40000:
            continue
        kind = int(rng.integers(5))
        lens = (np.full(B, max_len) if kind == 0 else rng.integers(0, max_len + 1, B) if kind == 1 else
                rng.integers(0, max_len + 1, B) * (rng.random(B) < 0.2) if kind == 2 else
                rng.integers(0, min(200, max_len + 1), B) if kind == 3 else np.full(B, -1))
        lens[0] = max_len if kind in (1, 3) else lens[0]
        got = replay(B, kv_heads, group, D, fmt, max_len, lens, exact=bool(rng.integers(2)),
                     weights=bool(rng.integers(2)), window=int(rng.choice([0, 0, 1, 500])))
        counted, plain = counted + (got["more"] > 0), plain + (got["more"] == 0)
        most = max(most, got["pieces"])
    assert counted > 40 and plain > 40 and most > 64, (counted, plain, most)


def test_few_long_sequences(replay):
    """Units in two and three levels of joins."""
    for D, fmt in ((64, "bf16"), (128, "mxfp8"), (256, "mxfp4")):
        for n in (2100, 2180, 13405, 33000, 66000, 131071, 1 << 20):
            for lens in ([n], [n, 5, n // 2], [70, n], [n, n, n, n]):
                for kv_heads in (1, 8):
                    replay(len(lens), kv_heads, 4, D, fmt, max(lens), np.array(lens))
    assert replay(1, 1, 4, 128, "mxfp8", 131071, np.array([131071]))["pieces"] == 512


def test_cases_of_the_gpu_tests(replay):
    """They reach what they are for: many units a workgroup and no room for
    pieces; the change of units counted, more than 512 units, some of them cut."""
    for case in cases.SHORT:
        fmt, f32, B, kv_heads, group, D, most = case
        got = replay(B, kv_heads, group, D, fmt, most, cases.lens_of(case), exact=f32)
        assert got["cut"] == 0 and B * kv_heads > 2 * 256
    for case in cases.COUNTED:
        fmt, f32, B, kv_heads, group, D, most = case
        for weights in (False, True):
            got = replay(B, kv_heads, group, D, fmt, most, cases.lens_of(case), exact=f32, weights=weights)
            assert got["more"] > 0 and got["cut"] > 100 and B * kv_heads > 512, case
