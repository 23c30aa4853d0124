"""The decode-step entry points refuse bad arguments before any HIP call, and
their plain FP64 forms agree with differences and brute force (CPU)."""
import ctypes

import numpy as np
import pytest

import block_scaled_fp4_03_amd as fp4
import decode_reference as ref

FAKE = 0x100000
NULL, SHAPE, ALIGN, FMT, DTYPE, WORKSPACE = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module", autouse=True)
def L():
    import os
    if not os.path.exists(fp4.LIB_PATH):
        import block_scaled_fp4_03_amd.build as b
        b.build()
    return fp4.lib()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, pages=8, page_size=16, kv_heads=2, head_dim=64, fmt=0)
    a.update(kw)
    return fp4.KVCacheStruct(**a)


CACHE_FAULTS = [(dict(fmt=3), FMT), (dict(fmt=-1), FMT), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
                (dict(page_size=8192), SHAPE), (dict(head_dim=32), SHAPE), (dict(head_dim=96), SHAPE),
                (dict(head_dim=320), SHAPE), (dict(kv_heads=0), SHAPE), (dict(pages=-1), SHAPE), (dict(k=None), NULL),
                (dict(v=None), NULL), (dict(fmt=1, k_scales=None), NULL), (dict(fmt=2, v_scales=None), NULL),
                (dict(k=FAKE + 8), ALIGN), (dict(v=FAKE + 2), ALIGN), (dict(fmt=1, k_scales=FAKE + 4), ALIGN)]


def append(c, **kw):
    a = dict(k=FAKE, v=FAKE, dt=1, ks=128, vs=128, table=FAKE, width=4, seqs=2, seq=FAKE, pos=FAKE, rows=3)
    a.update(kw)
    return fp4.fp4_kv_append(c, a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["table"], a["width"], a["seqs"], a["seq"],
                             a["pos"], a["rows"], None)


def attn(c, **kw):
    a = dict(q=FAKE, qdt=1, qs=256, table=FAKE, width=4, lens=FAKE, B=2, Hq=4, max_len=64, window=0, scale=0.1,
             out=FAKE, odt=1, lse=None, win=None, wout=None, wst=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_attn_decode(c, a["q"], a["qdt"], a["qs"], a["table"], a["width"], a["lens"], a["B"], a["Hq"],
                               a["max_len"], a["window"], a["scale"], a["out"], a["odt"], a["lse"], a["win"],
                               a["wout"], a["wst"], a["ws"], a["wsb"], None)


def evict(c, d=None, **kw):
    a = dict(st=FAKE, sw=4, lens=FAKE, w=FAKE, wst=64, dt=FAKE, dw=2, ol=FAKE, ow=FAKE, ost=32, kept=FAKE, B=2,
             max_len=64, budget=32, recent=4, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_kv_evict(c, a["st"], a["sw"], a["lens"], a["w"], a["wst"], c if d is None else d, a["dt"], a["dw"],
                            a["ol"], a["ow"], a["ost"], a["kept"], a["B"], a["max_len"], a["budget"], a["recent"],
                            a["ws"], a["wsb"], None)


def logprobs(**kw):
    a = dict(x=FAKE, dt=0, st=100, N=2, V=100, scale=1.0, tok=FAKE, M=1, lp=FAKE, ent=FAKE, lse=FAKE, k=4, tl=FAKE,
             ti=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return fp4.fp4_logprobs(a["x"], a["dt"], a["st"], a["N"], a["V"], a["scale"], a["tok"], a["M"], a["lp"], a["ent"],
                            a["lse"], a["k"], a["tl"], a["ti"], a["ws"], a["wsb"], None)


def backward(**kw):
    a = dict(x=FAKE, dt=0, st=100, N=2, V=100, scale=1.0, tok=FAKE, M=1, lse=FAKE, ent=FAKE, g=FAKE, ge=FAKE, dx=FAKE,
             dst=100)
    a.update(kw)
    return fp4.fp4_logprobs_backward(a["x"], a["dt"], a["st"], a["N"], a["V"], a["scale"], a["tok"], a["M"], a["lse"],
                                     a["ent"], a["g"], a["ge"], a["dx"], a["dst"], None)


@pytest.mark.parametrize("call", [append, attn, evict])
@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults(call, fault, status):
    assert call(cache(**fault)) == status


@pytest.mark.parametrize("call", [append, attn, evict])
def test_missing_cache(call):
    assert call(None) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(rows=-1), SHAPE), (dict(seqs=-1), SHAPE), (dict(width=-1), SHAPE),
    (dict(ks=127), SHAPE), (dict(vs=64), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(table=None), NULL), (dict(seq=None), NULL), (dict(pos=None), NULL),
    (dict(k=FAKE + 8), ALIGN), (dict(ks=132), ALIGN), (dict(dt=0, vs=130), ALIGN), (dict(seq=FAKE + 2), ALIGN),
    (dict(rows=0, k=None), 0), (dict(seqs=0), 0), (dict(width=0), 0)])
def test_append_arguments(kw, status):
    assert append(cache(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(qdt=2), DTYPE), (dict(odt=-1), DTYPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(Hq=3), SHAPE),
    (dict(Hq=-2), SHAPE), (dict(max_len=65), SHAPE), (dict(max_len=-1), SHAPE), (dict(window=-1), SHAPE),
    (dict(qs=255), SHAPE), (dict(wout=FAKE, wst=63), SHAPE), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(lens=None), NULL), (dict(table=None), NULL), (dict(win=FAKE), NULL), (dict(q=FAKE + 8), ALIGN),
    (dict(out=FAKE + 4), ALIGN), (dict(qs=260), ALIGN), (dict(lse=FAKE + 1), ALIGN), (dict(B=0, q=None), 0),
    (dict(Hq=0), 0)])
def test_attention_arguments(kw, status):
    assert attn(cache(), **kw) == status


def test_attention_workspace():
    c = cache(kv_heads=1, head_dim=128)
    n = fp4.fp4_attn_decode_workspace(c, 1, 8, 1 << 17, 0)
    if n:
        assert attn(c, B=1, Hq=8, qs=1024, width=1 << 13, max_len=1 << 17, ws=None, wsb=0) == WORKSPACE
        assert attn(c, B=1, Hq=8, qs=1024, width=1 << 13, max_len=1 << 17, wsb=n - 1) == WORKSPACE
        assert attn(c, B=1, Hq=8, qs=1024, width=1 << 13, max_len=1 << 17, ws=FAKE + 8) == ALIGN
    assert fp4.fp4_attn_decode_workspace(c, 1, 8, 1 << 17, 1) >= n
    assert fp4.fp4_attn_decode_workspace(cache(fmt=9), 1, 8, 64, 0) == 0
    assert fp4.fp4_attn_decode_workspace(cache(), 1, 3, 64, 0) == 0
    assert fp4.fp4_attn_decode_workspace(None, 1, 2, 64, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), SHAPE), (dict(max_len=65), SHAPE), (dict(budget=-1), SHAPE), (dict(recent=-1), SHAPE),
    (dict(budget=33, ost=33), SHAPE), (dict(wst=63), SHAPE), (dict(ost=31), SHAPE), (dict(sw=-1), SHAPE),
    (dict(lens=None), NULL), (dict(w=None), NULL), (dict(st=None), NULL), (dict(dt=None), NULL), (dict(ol=None), NULL),
    (dict(ow=None), NULL), (dict(kept=None), NULL), (dict(w=FAKE + 2), ALIGN), (dict(kept=FAKE + 2), ALIGN),
    (dict(B=0, lens=None), 0)])
def test_evict_arguments(kw, status):
    assert evict(cache(), **kw) == status


def test_evict_pools_must_agree():
    assert evict(cache(), cache(fmt=1)) == FMT
    assert evict(cache(), cache(kv_heads=4)) == SHAPE
    assert evict(cache(), cache(head_dim=128)) == SHAPE
    assert evict(cache(), cache(page_size=32)) == SHAPE


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(V=0), SHAPE), (dict(N=-1), SHAPE), (dict(st=99), SHAPE), (dict(M=-1), SHAPE),
    (dict(M=1025), SHAPE), (dict(k=33), SHAPE), (dict(k=-1), SHAPE), (dict(scale=0.0), SHAPE),
    (dict(scale=-1.0), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(x=None), NULL), (dict(tok=None), NULL), (dict(lp=None), NULL), (dict(tl=None), NULL), (dict(ti=None), NULL),
    (dict(x=FAKE + 2), ALIGN), (dict(dt=1, x=FAKE + 1), ALIGN), (dict(tok=FAKE + 2), ALIGN), (dict(ti=FAKE + 1), ALIGN),
    (dict(N=0, x=None), 0)])
def test_logprobs_arguments(kw, status):
    assert logprobs(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), DTYPE), (dict(V=0), SHAPE), (dict(st=99), SHAPE), (dict(dst=99), SHAPE), (dict(M=1025), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(x=None), NULL), (dict(dx=None), NULL), (dict(lse=None), NULL),
    (dict(tok=None), NULL), (dict(g=None), NULL), (dict(ent=None), NULL), (dict(dx=FAKE + 2), ALIGN),
    (dict(lse=FAKE + 2), ALIGN), (dict(N=0, x=None), 0)])
def test_backward_arguments(kw, status):
    assert backward(**kw) == status


def test_wrappers_refuse_before_the_library():
    """Host tensors, wrong types and shapes stop in the Python wrappers."""
    torch = pytest.importorskip("torch")
    f = torch.zeros
    with pytest.raises(ValueError):
        fp4.KVCache(f((2, 1, 16, 64), dtype=torch.bfloat16), f((2, 1, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        fp4.KVCache(f((2, 1, 16, 64)), f((2, 1, 16, 64)))
    with pytest.raises(TypeError):
        fp4.decode_attention(f((1, 2, 64)), "cache", f((1, 1)), f(1))
    with pytest.raises(TypeError):
        fp4.kv_append(None, f((1, 2, 64)), f((1, 2, 64)), f((1, 1)), f(1), f(1))
    with pytest.raises(TypeError):
        fp4.logprobs(f((2, 5), dtype=torch.int32), f((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        fp4.logprobs(f((2, 5)), f((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        fp4.logprobs(f((5, 2)).t(), f((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError):
        fp4.logprobs(f(5), f((2, 1), dtype=torch.int32))
    with pytest.raises(TypeError):
        fp4.logprobs([1.0], f((2, 1), dtype=torch.int32))


def test_struct_layout():
    """The ctypes structure has the C struct's layout (8-byte pointers, int64, four int32)."""
    assert ctypes.sizeof(fp4.KVCacheStruct) == 56
    assert fp4.KVCacheStruct.pages.offset == 32 and fp4.KVCacheStruct.fmt.offset == 52


# ---- the plain forms themselves ------------------------------------------------
def test_plain_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, tokens = rng.standard_normal(23), np.array([4, 4, 22, -1, 23])
    g, ge, sc, d = rng.standard_normal(5), 0.7, 1.3, 1e-5
    want = ref.logprobs_grad(x, tokens, sc, g, ge)
    for i in range(23):
        e = np.zeros(23)
        e[i] = d
        diff = (ref.logprobs_loss(x + e, tokens, sc, g, ge) - ref.logprobs_loss(x - e, tokens, sc, g, ge)) / (2 * d)
        assert abs(diff - want[i]) < 1e-7


def test_plain_eviction():
    w = np.array([1.0, 5.0, 2.0, 2.0, np.nan, 2.0, 0.0, 9.0])
    assert ref.evict(w, 8, 8, 2) == list(range(8))
    assert ref.evict(w, 8, 4, 1) == [1, 2, 4, 7]
    assert ref.evict(w, 8, 3, 3) == [5, 6, 7]
    assert ref.evict(w, 8, 2, 0) == [4, 7]
    assert ref.evict(w, 8, 0, 5) == []


def test_plain_rows():
    codes = np.array([[0x21] + [0] * 15], np.uint8)
    assert list(ref.row_values(codes, np.array([[128]]), "mxfp4")[0, :3]) == [1.0, 2.0, 0.0]
    assert ref.row_values(np.array([[0x38] + [0] * 31], np.uint8), np.array([[126]]), "mxfp8")[0, 0] == 0.5


def test_attention_counts_fit():
    """The bound on sequences x heads x tiles that the kernel counts in 32 bits."""
    c = cache(kv_heads=64, page_size=4096, head_dim=64)
    big = dict(B=65535, Hq=64, qs=4096, width=1 << 15)
    assert attn(c, max_len=1 << 20, **big) == SHAPE
    assert fp4.fp4_attn_decode_workspace(c, 65535, 64, 1 << 20, 0) == 0
    assert fp4.fp4_attn_decode_workspace(c, 65535, 64, 1 << 14, 0) > 0
