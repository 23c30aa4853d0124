"""The entry points around a layer's products (norms with rotary positions,
routing to experts, verification of drafts) refuse bad arguments before any HIP
call, and their plain FP64 forms agree with differences and brute force (CPU)."""
import ctypes

import numpy as np
import pytest

import block_scaled_fp4_03_amd as fp4
import layer_reference as ref

FAKE = 0x100000
NULL, SHAPE, ALIGN, FMT, DTYPE, WORKSPACE, HIP, FLAGS = -1, -2, -3, -4, -5, -6, -7, -8
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def L():
    import os
    if not os.path.exists(fp4.LIB_PATH):
        import block_scaled_fp4_03_amd.build as b
        b.build()
    return fp4.lib()


def rope(freq=FAKE, rot=64, axes=1, sections=(0, 0, 0, 0), flags=0):
    return fp4.RopeStruct(freq, rot, axes, (ctypes.c_int32 * 4)(*sections), flags)


def forward(r, **kw):
    a = dict(pos=FAKE, q=FAKE, qs=256, hq=4, k=FAKE, ks=128, hk=2, D=64, dt=1, wq=FAKE, wk=FAKE, eps=1e-6, qo=FAKE,
             qos=256, ko=FAKE, kos=128, rows=3)
    a.update(kw)
    return fp4.fp4_qk_norm_rope(r, a["pos"], a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["hk"], a["D"], a["dt"],
                                a["wq"], a["wk"], a["eps"], a["qo"], a["qos"], a["ko"], a["kos"], a["rows"], None)


def backward(r, **kw):
    a = dict(pos=FAKE, gq=FAKE, gqs=256, gk=FAKE, gks=128, q=FAKE, qs=256, hq=4, k=FAKE, ks=128, hk=2, D=64, dt=1,
             wq=FAKE, wk=FAKE, eps=1e-6, dq=FAKE, dqs=256, dk=FAKE, dks=128, dwq=FAKE, dwk=FAKE, rows=3, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_qk_norm_rope_backward(r, a["pos"], a["gq"], a["gqs"], a["gk"], a["gks"], a["q"], a["qs"], a["hq"],
                                         a["k"], a["ks"], a["hk"], a["D"], a["dt"], a["wq"], a["wk"], a["eps"],
                                         a["dq"], a["dqs"], a["dk"], a["dks"], a["dwq"], a["dwk"], a["rows"], a["ws"],
                                         a["wsb"], None)


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,status", [
    (dict(rot=-8), SHAPE), (dict(rot=4), SHAPE), (dict(rot=72), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
    (dict(axes=2, sections=(16, 15, 0, 0)), SHAPE), (dict(axes=2, sections=(33, -1, 0, 0)), SHAPE),
    (dict(axes=3, sections=(0, 0, 31, 1)), SHAPE), (dict(flags=4), FLAGS), (dict(freq=None), NULL),
    (dict(freq=FAKE + 2), ALIGN)])
def test_rope_faults(call, kw, status):
    assert call(rope(**kw)) == status


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(D=24), SHAPE), (dict(D=68), SHAPE), (dict(D=264), SHAPE), (dict(hq=-1), SHAPE),
    (dict(hk=65536), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 40), SHAPE), (dict(rows=1 << 62), SHAPE),
    (dict(rows=1 << 25), SHAPE),
    (dict(qs=255), SHAPE), (dict(ks=127), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=NAN), SHAPE),
    (dict(eps=INF), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL),
    (dict(pos=FAKE + 2), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(k=FAKE + 2), ALIGN), (dict(qs=260), ALIGN),
    (dict(dt=0, ks=130), ALIGN), (dict(wq=FAKE + 2), ALIGN), (dict(wk=FAKE + 1), ALIGN)])
def test_norm_rope_arguments(call, kw, status):
    assert call(rope(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(qo=None), NULL), (dict(ko=None), NULL), (dict(qo=FAKE + 8), ALIGN), (dict(qos=255), SHAPE),
    (dict(kos=132), ALIGN), (dict(rows=0, q=None, pos=None), 0), (dict(hq=0, hk=0), 0)])
def test_norm_rope_outputs(kw, status):
    assert forward(rope(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(gq=None), NULL), (dict(gk=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dwq=None), NULL),
    (dict(dwk=None), NULL), (dict(gqs=255), SHAPE), (dict(dks=100), SHAPE), (dict(gk=FAKE + 8), ALIGN),
    (dict(dwq=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(ws=FAKE + 8), ALIGN),
    (dict(hq=0, hk=0), 0), (dict(rows=0, wq=None, wk=None), 0)])
def test_norm_rope_backward_outputs(kw, status):
    assert backward(rope(), **kw) == status


def test_norm_rope_workspace():
    n = fp4.fp4_qk_norm_rope_workspace(3, 4, 2, 64)
    assert 0 < n <= 1024 * 2 * 64 * 4
    assert backward(rope(), wsb=n - 1) == WORKSPACE
    assert fp4.fp4_qk_norm_rope_workspace(1 << 20, 64, 8, 256) == 1024 * 2 * 256 * 4
    assert fp4.fp4_qk_norm_rope_workspace(3, 4, 2, 20) == 0
    assert fp4.fp4_qk_norm_rope_workspace(-1, 4, 2, 64) == 0


def route(**kw):
    a = dict(x=FAKE, dt=1, st=32, T=5, E=32, k=4, re=1, ids=FAKE, w=FAKE)
    a.update(kw)
    return fp4.fp4_moe_route(a["x"], a["dt"], a["st"], a["T"], a["E"], a["k"], a["re"], a["ids"], a["w"], None)


def route_back(**kw):
    a = dict(x=FAKE, dt=1, st=32, T=5, E=32, k=4, re=1, ids=FAKE, w=FAKE, dx=FAKE)
    a.update(kw)
    return fp4.fp4_moe_route_backward(a["x"], a["dt"], a["st"], a["T"], a["E"], a["k"], a["re"], a["ids"], a["w"],
                                      a["dx"], None)


@pytest.mark.parametrize("call", [route, route_back])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 61), SHAPE), (dict(E=0), SHAPE), (dict(E=513, st=513), SHAPE),
    (dict(k=0), SHAPE), (dict(k=17), SHAPE), (dict(E=3, k=4), SHAPE), (dict(st=31), SHAPE), (dict(x=None), NULL),
    (dict(ids=None), NULL), (dict(w=None), NULL), (dict(x=FAKE + 1), ALIGN), (dict(dt=0, x=FAKE + 2), ALIGN),
    (dict(ids=FAKE + 2), ALIGN), (dict(w=FAKE + 1), ALIGN), (dict(T=0, x=None), 0)])
def test_route_arguments(call, kw, status):
    assert call(**kw) == status


def test_route_backward_output():
    assert route_back(dx=None) == NULL and route_back(dx=FAKE + 1) == ALIGN


def sort(**kw):
    a = dict(ids=FAKE, T=5, k=4, E=32, off=FAKE, rows=FAKE, pos=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_moe_sort(a["ids"], a["T"], a["k"], a["E"], a["off"], a["rows"], a["pos"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(k=-1), SHAPE), (dict(k=65), SHAPE), (dict(T=1 << 29, k=4), SHAPE), (dict(E=0), SHAPE),
    (dict(E=513), SHAPE), (dict(ids=None), NULL), (dict(off=None), NULL), (dict(rows=None), NULL),
    (dict(pos=None), NULL), (dict(T=0, off=None), NULL), (dict(ids=FAKE + 2), ALIGN), (dict(pos=FAKE + 1), ALIGN),
    (dict(T=1 << 20, ws=None), WORKSPACE), (dict(T=1 << 20, wsb=64), WORKSPACE), (dict(T=1 << 20, ws=FAKE + 8), ALIGN)])
def test_sort_arguments(kw, status):
    assert sort(**kw) == status


def test_sort_workspace():
    n = fp4.fp4_moe_sort_workspace(1 << 20, 4, 32)
    assert n > 0 and sort(T=1 << 20, wsb=n - 1) == WORKSPACE
    assert fp4.fp4_moe_sort_workspace(4, 4, 0) == 0 and fp4.fp4_moe_sort_workspace(-4, 4, 8) == 0


def gather(**kw):
    a = dict(x=FAKE, dt=1, st=64, pos=FAKE, T=5, k=4, H=64, rows=20, out=FAKE, w=FAKE)
    a.update(kw)
    return fp4.fp4_moe_gather(a["x"], a["dt"], a["st"], a["pos"], a["T"], a["k"], a["H"], a["rows"], a["out"], None)


def combine(**kw):
    a = dict(x=FAKE, dt=1, st=64, pos=FAKE, T=5, k=4, H=64, rows=20, out=FAKE, w=FAKE)
    a.update(kw)
    return fp4.fp4_moe_combine(a["x"], a["dt"], a["pos"], a["w"], a["T"], a["k"], a["H"], a["rows"], a["out"],
                               a["st"], None)


def combine_back(**kw):
    a = dict(x=FAKE, dt=1, st=64, pos=FAKE, T=5, k=4, H=64, rows=20, out=FAKE, w=FAKE, y=FAKE, dw=FAKE)
    a.update(kw)
    return fp4.fp4_moe_combine_backward(a["x"], a["st"], a["y"], a["dt"], a["pos"], a["w"], a["T"], a["k"], a["H"],
                                        a["rows"], a["out"], a["dw"], None)


@pytest.mark.parametrize("call", [gather, combine, combine_back])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(T=-1), SHAPE), (dict(k=-1), SHAPE), (dict(k=65), SHAPE), (dict(H=0), SHAPE),
    (dict(H=60), SHAPE), (dict(dt=0, H=62), SHAPE), (dict(st=56), SHAPE), (dict(rows=-1), SHAPE),
    (dict(T=1 << 26, H=1 << 16, st=1 << 16, k=1), SHAPE), (dict(T=1 << 30, k=2), SHAPE), (dict(T=1 << 24, k=1), SHAPE), (dict(x=None), NULL),
    (dict(pos=None), NULL), (dict(out=None), NULL), (dict(x=FAKE + 8), ALIGN), (dict(out=FAKE + 4), ALIGN),
    (dict(st=68), ALIGN), (dict(pos=FAKE + 2), ALIGN), (dict(T=0, x=None), 0)])
def test_row_arguments(call, kw, status):
    assert call(**kw) == status


def test_row_arguments_of_one_call():
    assert combine(w=FAKE + 2) == ALIGN
    assert combine_back(w=None) == NULL and combine_back(dw=None) == NULL and combine_back(y=None) == NULL
    assert combine_back(y=FAKE + 8) == ALIGN and combine_back(dw=FAKE + 2) == ALIGN
    assert gather(rows=0, out=None) == 0 and gather(k=0, pos=None) == 0 and combine_back(k=0, pos=None) == 0


def verify(**kw):
    a = dict(t=FAKE, ts=400, tr=100, d=FAKE, ds=300, dr=100, dt=0, B=2, G=3, V=100, tok=FAKE, u=FAKE, temp=FAKE,
             out=FAKE, acc=FAKE, ch=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_verify_drafts(a["t"], a["ts"], a["tr"], a["d"], a["ds"], a["dr"], a["dt"], a["B"], a["G"], a["V"],
                                 a["tok"], a["u"], a["temp"], a["out"], a["acc"], a["ch"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(G=-1), SHAPE), (dict(G=33), SHAPE),
    (dict(V=0), SHAPE), (dict(V=(1 << 24) + 1), SHAPE), (dict(B=65535, V=1 << 24), SHAPE), (dict(ts=-1), SHAPE),
    (dict(tr=-1), SHAPE), (dict(ds=-1), SHAPE), (dict(dr=1 << 41), SHAPE), (dict(t=None), NULL), (dict(tok=None), NULL),
    (dict(u=None), NULL), (dict(out=None), NULL), (dict(acc=None), NULL), (dict(ch=None), NULL), (dict(t=FAKE + 2), ALIGN),
    (dict(d=FAKE + 1), ALIGN), (dict(dt=1, t=FAKE + 1), ALIGN), (dict(tok=FAKE + 2), ALIGN), (dict(temp=FAKE + 2), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE), (dict(ws=FAKE + 8), ALIGN), (dict(B=0, t=None), 0)])
def test_verify_arguments(kw, status):
    assert verify(**kw) == status


def test_verify_workspace():
    n = fp4.fp4_verify_drafts_workspace(2, 3, 100)
    assert n > 0 and verify(wsb=n - 1) == WORKSPACE
    assert fp4.fp4_verify_drafts_workspace(2, 33, 100) == 0 and fp4.fp4_verify_drafts_workspace(2, 3, 0) == 0


def test_wrappers_refuse_before_the_library():
    """Host tensors, wrong types and shapes stop in the Python wrappers."""
    torch = pytest.importorskip("torch")
    f, i32 = torch.zeros, torch.int32
    with pytest.raises(ValueError):
        fp4.Rope(f(32))
    with pytest.raises(TypeError):
        fp4.Rope(f(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        fp4.qk_norm_rope(f((2, 4, 64)), f((2, 2, 64)), None, None)
    with pytest.raises(TypeError):
        fp4.qk_norm_rope(f((2, 4, 64), dtype=torch.float16), f((2, 2, 64)), None, None)
    with pytest.raises(ValueError):
        fp4.qk_norm_rope_backward(f((2, 4, 64)), f((2, 2, 64)), f((2, 4, 64)), f((2, 2, 64)), None, None)
    with pytest.raises(ValueError):
        fp4.moe_route(f((4, 8)), 2)
    with pytest.raises(TypeError):
        fp4.moe_route(f((4, 8), dtype=i32), 2)
    with pytest.raises(ValueError):
        fp4.moe_route_backward(f((4, 8)), f((4, 2), dtype=i32), f((4, 2)))
    with pytest.raises(TypeError):
        fp4.moe_sort(f((4, 2)), 8)
    with pytest.raises(ValueError):
        fp4.moe_sort(f((4, 2), dtype=i32), 8)
    with pytest.raises(ValueError):
        fp4.moe_gather(f((4, 64)), f((4, 2), dtype=i32))
    with pytest.raises(ValueError):
        fp4.moe_combine(f((8, 64)), f((4, 2), dtype=i32))
    with pytest.raises(ValueError):
        fp4.moe_combine_backward(f((4, 64)), f((8, 64)), f((4, 2), dtype=i32), None)
    with pytest.raises(ValueError):
        fp4.verify_drafts(f((2, 4, 9)), None, f((2, 3), dtype=i32), f((2, 4)))
    with pytest.raises(ValueError):
        fp4.verify_drafts(f((2, 5, 9)), None, f((2, 3), dtype=i32), f((2, 4)))
    with pytest.raises(TypeError):
        fp4.verify_drafts(f((2, 4, 9), dtype=i32), None, f((2, 3), dtype=i32), f((2, 4)))


def test_null_stream_of_another_device(monkeypatch):
    """The null stream is the current device's: operands on another one are refused
    there, and run on a stream of their own."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    assert fp4._run_on(None, torch.device("cuda", 0)) == 0
    with pytest.raises(ValueError):
        fp4._run_on(None, torch.device("cuda", 1))
    assert fp4._run_on(Stream(), torch.device("cuda", 1)) == 77


def test_struct_layout():
    assert ctypes.sizeof(fp4.RopeStruct) == 40
    assert fp4.RopeStruct.sections.offset == 16 and fp4.RopeStruct.flags.offset == 32


# ---- the plain forms themselves ------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_norm_rope_gradient_against_differences(interleaved):
    rng = np.random.default_rng(2)
    x, w, g = rng.standard_normal((2, 2, 16)), rng.standard_normal(16), rng.standard_normal((2, 2, 16))
    c, s = ref.cos_sin(np.array([[3, -7], [5, 100]]), rng.random(4).astype(np.float32), [0, 0, 1, 1])

    def loss(x, w):
        return (ref.norm_rope(x, w, 0.1, c, s, 8, interleaved) * g).sum()

    dx, dw, _, _ = ref.norm_rope_grad(x, w, 0.1, c, s, 8, interleaved, g)
    for at, d in ((x, dx), (w, dw)):
        for i in np.ndindex(at.shape):
            keep = at[i]
            at[i] = keep + 1e-6
            up = loss(x, w)
            at[i] = keep - 1e-6
            down = loss(x, w)
            at[i] = keep
            assert abs((up - down) / 2e-6 - d[i]) < 1e-7


def test_plain_axes():
    assert ref.axis_of_pairs([2, 1, 3], False) == [0, 0, 1, 2, 2, 2]
    assert ref.axis_of_pairs([2, 1, 3], True) == [0, 1, 2, 0, 2, 2]


@pytest.mark.parametrize("renormalise", [True, False])
def test_plain_route_gradient_against_differences(renormalise):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 2))
    ids, w = ref.route(x, 2, renormalise)
    want, _, _ = ref.route_grad(x, ids, g, renormalise)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-6
        up, down = (ref.route(x + e, 2, renormalise)[1] for e in (d, -d))
        assert abs(((up - down) * g).sum() / 2e-6 - want[i]) < 1e-8


def test_plain_sort():
    off, rows, pos = ref.sort(np.array([[2, 0], [-1, 2], [0, 9]]), 3)
    assert list(off) == [0, 2, 2, 6] and list(rows) == [0, 2, 0, 1, 1, 2]
    assert pos.tolist() == [[2, 0], [-5, 3], [1, -6]]


def test_plain_verification_keeps_the_target_distribution():
    """Over many random numbers, the first emitted token follows p, whatever the
    draft (30000 draws: 5 standard deviations are below 0.015)."""
    rng = np.random.default_rng(4)
    target, draft = rng.standard_normal((2, 5)), rng.standard_normal((1, 5))
    p, q = ref.probabilities(target[0], 0.7), ref.probabilities(draft[0], 0.7)
    n, count = 30000, np.zeros(5)
    for d in rng.choice(5, size=n, p=q):
        out, kept, _ = ref.verify(target, draft, [d], rng.random(2), 0.7)
        count[out[0]] += 1
        assert kept == (1 if out[1] >= 0 else 0)
    assert np.abs(count / n - p).max() < 0.015


def test_plain_verification_edges():
    t = np.array([[0.0, 1.0, 1.0], [5.0, 0.0, 0.0]])
    assert ref.verify(t, None, [1], [0.5, 0.5], 0.0) == ([1, 0], 1, [1.0])
    assert ref.verify(t, None, [2], [0.5, 0.5], -1.0) == ([1, -1], 0, [0.0])
    assert ref.verify(t, None, [3], [0.5, 0.0], 1.0) == ([0, -1], 0, [0.0])
    assert ref.verify(t, t[:1], [0], [0.999, 0.9], 1.0)[1] == 1
    bad = np.array([[0.0, np.nan, 1.0], [5.0, 0.0, 0.0]])
    assert ref.verify(bad, None, [1], [0.5, 0.5], 1.0) == ([-1, -1], 0, [0.0])
    masked = np.array([[-np.inf, 0.0, -np.inf], [5.0, 0.0, 0.0]])
    assert ref.verify(masked, masked[:1], [0], [0.0, 0.0], 1.0)[:2] == ([1, -1], 0)
