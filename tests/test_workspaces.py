"""The operators' workspaces: their sizes, and where a verification's data lie (CPU)."""
import ctypes
import os
import subprocess

import pytest

import block_scaled_fp4_03_amd as fp4

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_fp4_03_amd", "csrc")
# Vocabularies around what a workgroup, a lane's run of chunks and all splits take.
VOCABS = (1, 511, 513, 4095, 8191, 8192, 40000, 100003, 131072, 131073, 300001, 1 << 24)


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(fp4.LIB_PATH):
        import block_scaled_fp4_03_amd.build as b
        b.build()
    fp4.lib()


def test_empty_calls_need_none():
    assert fp4.fp4_verify_drafts_workspace(0, 4, 1000) == 0
    assert fp4.fp4_verify_drafts_workspace(0, 0, 1) == 0
    assert fp4.fp4_moe_sort_workspace(0, 4, 8) == 0 and fp4.fp4_moe_sort_workspace(4, 0, 8) == 0
    assert fp4.fp4_qk_norm_rope_workspace(0, 4, 2, 64) == 0 and fp4.fp4_qk_norm_rope_workspace(4, 0, 0, 64) == 0


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("workspace") / "workspace_check.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "workspace_check.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    I64 = ctypes.c_int64
    L.verify_layout_check.argtypes = [I64, I64, I64, ctypes.c_void_p, ctypes.c_char_p, ctypes.c_size_t]
    L.control_bytes.restype = ctypes.c_size_t
    return L


def test_verification_keeps_to_its_places(layout):
    """Row counters within the control words, everything else behind them and apart,
    and all of it within the size that the library asks for."""
    total, msg = ctypes.c_size_t(), ctypes.create_string_buffer(256)
    for B in (1, 2, 3, 5, 8, 16, 17, 33, 64, 100, 129, 255, 256):
        for G in (0, 1, 4, 7, 32):
            for V in VOCABS:
                need = fp4.fp4_verify_drafts_workspace(B, G, V)
                for rows in {G + 1, 2 * G + 1}:
                    what = "%d sequences, %d rows of %d: " % (B, rows, V)
                    rc = layout.verify_layout_check(B, rows, V, ctypes.byref(total), msg, 256)
                    assert rc == 0, what + msg.value.decode()
                    assert total.value <= need, what


def test_partial_sums_have_room_behind_the_control_words(layout):
    """The least data of a sort and of a gradient of norms, and the control words."""
    words = layout.control_bytes()
    for E in (1, 32, 512):
        for T in (2049, 8192, 524288, 524289, 1 << 22):
            chunk = 2048 if T <= 524288 else 8192
            assert fp4.fp4_moe_sort_workspace(T, 1, E) >= words + (-(-T // chunk) + 1) * (E + 1) * 4
    for D in (32, 64, 256):
        for rows, q, k in ((1, 1, 0), (1, 1, 1), (7, 5, 1), (640, 1, 1), (1 << 20, 64, 8)):
            assert fp4.fp4_qk_norm_rope_workspace(rows, q, k, D) >= words + min(rows * (q + k), 1281) * D * 4


def never_less(size, *ranges):
    """size(*args) never falls as any one of its arguments grows over its range."""
    for at in range(len(ranges)):
        others = [[]]
        for i, r in enumerate(ranges):
            others = [o + [v] for o in others for v in ([None] if i == at else r)]
        for o in others:
            before = 0
            for v in ranges[at]:
                args = o[:at] + [v] + o[at + 1:]
                now = size(*args)
                assert now >= before, "%s: %d, %d with one argument less" % (args, now, before)
                before = now


def test_a_sort_workspace_serves_smaller_calls():
    T = sorted({m * n + d for m in (1, 64, 256, 1024, 2048, 8192) for n in (1, 3, 16, 63, 64, 65, 255, 256, 257, 1000)
                for d in (-1, 0, 1)})
    never_less(fp4.fp4_moe_sort_workspace, T, range(65), (1, 2, 32, 128, 512))
    assert fp4.fp4_moe_sort_workspace(131072, 8, 128) >= fp4.fp4_moe_sort_workspace(65536, 8, 128)


def test_a_workspace_of_the_norms_gradient_serves_smaller_calls():
    never_less(fp4.fp4_qk_norm_rope_workspace, (0, 1, 2, 5, 100, 128, 255, 1024, 1025, 1 << 20), range(0, 65, 3), range(17),
               (32, 64, 72, 128, 256))


def test_a_verification_workspace_serves_smaller_calls():
    size = fp4.fp4_verify_drafts_workspace
    never_less(size, list(range(0, 300)) + [1000, 20000], (0, 1, 2, 3, 4, 7, 8, 31, 32), (1, 5003, 8192, 100003, 131072, 1 << 19))
    never_less(size, (1, 2, 58, 64, 227, 256), range(33), VOCABS)
    assert size(256, 4, 131072) >= size(227, 4, 131072) and size(64, 3, 131072) >= size(58, 3, 131072)
