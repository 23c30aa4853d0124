"""fp4_kv_append and fp4_kv_evict on the GPU: rows and scales against the
oracle's quantiser bit for bit, kept tokens and moved rows against the plain
selection exactly."""
import numpy as np
import pytest

import decode_reference as ref
import synth
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu

FMTS = ("bf16", "mxfp8", "mxfp4")


def _fmt(fp4, name):
    return {"bf16": fp4.KV_BF16, "mxfp8": fp4.KV_MXFP8, "mxfp4": fp4.KV_MXFP4}[name]


def _pools(cache):
    return [t for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None]


def _fill(cache, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in _pools(cache):
        raw = torch.randint(0, 256, (t.numel() * t.element_size(),), generator=g, device="cuda", dtype=torch.int16)
        t.view(torch.uint8).copy_(raw.to(torch.uint8).view(t.view(torch.uint8).shape))


def _bits(t):
    return to_host(t) if t.dtype.itemsize == 1 else to_host(t).view(np.uint16)


def _expected_rows(orc, x, fmt):
    """The oracle's codes and scales (dense per row) of rows x (n x D float32 values)."""
    if fmt == "bf16":
        return synth.to_bf16_bits(x), None
    f = orc.FMT_MXFP8 if fmt == "mxfp8" else orc.FMT_MXFP4
    r = orc.quantize(x, f)
    n, D = x.shape
    scales = np.array([[r[1][orc.scale_offset(f, n, D, i, b)] for b in range(D // 32)] for i in range(n)], np.uint8)
    return r[0].reshape(n, -1), scales


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("heads,dim,page,rows", [(1, 64, 16, 1), (3, 128, 16, 37), (8, 128, 64, 5), (2, 192, 32, 19),
                                                 (1, 256, 128, 130)])
def test_append_matches_the_quantiser(orc, fmt, dtype, heads, dim, page, rows):
    import torch
    import block_scaled_fp4_03_amd as fp4
    say("append %s %s heads %d dim %d page %d rows %d" % (fmt, dtype, heads, dim, page, rows))
    seqs, width = 3, -(-(rows + 20) // page)
    cache = fp4.KVCache.empty(seqs * width + 1, page, heads, dim, _fmt(fp4, fmt))
    _fill(cache, 5)
    before = [_bits(t).copy() for t in _pools(cache)]
    xk = synth.gaussian(100 + rows, (rows, heads * dim), std=2.0, bernoulli=0.01)
    xv = synth.gaussian(200 + rows, (rows, heads * dim), std=0.1)
    xk[0, :32] = 0.0
    if dtype == "bf16":
        kh, vh = synth.to_bf16_bits(xk), synth.to_bf16_bits(xv)
        xk, xv = ((h.astype(np.uint32) << 16).view(np.float32) for h in (kh, vh))
    else:
        kh, vh = xk, xv
    # Columns of a wider matrix: the rows have a stride of their own.
    wide = torch.zeros((rows, 3 * heads * dim), dtype=torch.float32 if dtype == "f32" else torch.bfloat16,
                       device="cuda")
    wide[:, :heads * dim] = to_dev(kh)
    wide[:, 2 * heads * dim:] = to_dev(vh)
    k = wide[:, :heads * dim].unflatten(1, (heads, dim))
    v = wide[:, 2 * heads * dim:].unflatten(1, (heads, dim))
    rng = np.random.default_rng(rows)
    table = rng.permutation(seqs * width).reshape(seqs, width).astype(np.int32)
    seq = (np.arange(rows) % seqs).astype(np.int32)
    pos = (np.arange(rows) // seqs + 3).astype(np.int32)
    fp4.kv_append(cache, k, v, to_dev(table), to_dev(seq), to_dev(pos))
    got = [_bits(t) for t in _pools(cache)]
    for which, x in ((0, xk), (1, xv)):
        codes, scales = _expected_rows(orc, x.reshape(rows * heads, dim), fmt)
        for i in range(rows):
            p, s = table[seq[i], pos[i] // page], pos[i] % page
            before[which][p, :, s] = codes.reshape(rows, heads, -1)[i]
            if scales is not None:
                before[2 + which][p, :, s] = scales.reshape(rows, heads, -1)[i]
    for a, b in zip(got, before):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_skips_what_has_no_place(orc, fmt):
    """Rows padded with seq -1, past the sequences or the table, with a negative
    position or a page outside the pool leave every byte alone."""
    import block_scaled_fp4_03_amd as fp4
    cache = fp4.KVCache.empty(4, 16, 2, 64, _fmt(fp4, fmt))
    _fill(cache, 6)
    before = [_bits(t).copy() for t in _pools(cache)]
    table = np.array([[0, 1], [4, -1]], np.int32)
    seq = np.array([-1, 2, 0, 0, 1, 1, 7], np.int32)
    pos = np.array([0, 0, 32, -1, 3, 20, 2 ** 31 - 1], np.int32)
    x = to_dev(synth.gaussian(9, (7, 2, 64)))
    say("append of rows without a place, %s" % fmt)
    fp4.kv_append(cache, x, x, to_dev(table), to_dev(seq), to_dev(pos))
    for t, b in zip(_pools(cache), before):
        np.testing.assert_array_equal(_bits(t), b)
    fp4.kv_append(cache, x[:0], x[:0], to_dev(table), to_dev(seq[:0]), to_dev(pos[:0]))


def test_append_rounds_special_values_to_bf16():
    """FP32 into a BF16 cache: NaN stays NaN, infinities stay, ties go to even."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.4e38, 1.00390625, 1.01171875, -0.0, 1e-41] * 8,
                     device="cuda").view(1, 1, 64)
    cache = fp4.KVCache.empty(1, 16, 1, 64)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("append of special values")
    fp4.kv_append(cache, x, x, z.view(1, 1), z, z)
    torch.testing.assert_close(cache.k[0, 0, 0].cpu(), x.cpu().view(64).to(torch.bfloat16), rtol=0, atol=0,
                               equal_nan=True)


def _evict_case(fmt, lens, heads, dim, page, budget, recent, weights, seed, other_pool=False):
    import torch
    import block_scaled_fp4_03_amd as fp4
    B = len(lens)
    width, width2 = -(-max(max(lens), 1) // page), -(-max(min(max(lens), budget), 1) // page)
    pages = B * (width + width2)
    src = fp4.KVCache.empty(pages, page, heads, dim, _fmt(fp4, fmt))
    _fill(src, seed)
    dst = src
    if other_pool:
        dst = fp4.KVCache.empty(pages + 3, page, heads, dim, _fmt(fp4, fmt))
        _fill(dst, seed + 1)
    rng = np.random.default_rng(seed)
    perm = rng.permutation(pages).astype(np.int32)
    table, table2 = perm[:B * width].reshape(B, width), perm[B * width:].reshape(B, width2)
    before = [_bits(t).copy() for t in _pools(src)]
    want = before if dst is src else [_bits(t).copy() for t in _pools(dst)]
    say("evict %s lens %s heads %d dim %d page %d budget %d recent %d" % (fmt, lens, heads, dim, page, budget, recent))
    out_lens, out_w, kept = fp4.kv_evict(src, to_dev(table), to_dev(np.array(lens, np.int32)), to_dev(weights),
                                         budget, recent, to_dev(table2), out_cache=None if dst is src else dst)
    got = [_bits(t) for t in _pools(dst)]
    want = [w.copy() for w in want]
    exp_kept = np.full((B, heads, budget), -1, np.int32)
    exp_w = np.zeros(tuple(out_w.shape), np.float32)
    for b, n in enumerate(lens):
        for h in range(heads):
            keep = ref.evict(weights[b, h], n, budget, recent)
            exp_kept[b, h, :len(keep)] = keep
            exp_w[b, h, :len(keep)] = weights[b, h, keep]
            for i, t in enumerate(keep):
                for w, old in zip(want, before):
                    w[table2[b, i // page], h, i % page] = old[table[b, t // page], h, t % page]
    np.testing.assert_array_equal(to_host(out_lens), np.minimum(lens, budget))
    np.testing.assert_array_equal(to_host(kept), exp_kept)
    np.testing.assert_array_equal(to_host(out_w), exp_w)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,heads,dim,page,budget,recent", [
    ([1], 1, 64, 16, 1, 0), ([0, 1, 2], 2, 64, 16, 1, 1), ([17, 40, 33], 3, 128, 16, 33, 5),
    ([1100, 1030], 2, 64, 32, 1024, 128), ([5000, 700], 1, 128, 64, 600, 600), ([3000], 2, 192, 16, 77, 0),
    ([130, 0, 64], 1, 256, 64, 64, 1000), ([2049], 1, 64, 16, 2048, 1),
])
def test_evict_matches_plain_selection(fmt, lens, heads, dim, page, budget, recent):
    rng = np.random.default_rng(len(lens) * 1000 + budget)
    cap = -(-max(max(lens), 1) // page) * page
    w = np.exp(2.0 * rng.standard_normal((len(lens), heads, cap))).astype(np.float32)
    _evict_case(fmt, lens, heads, dim, page, budget, recent, w, 11 + budget)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "special", "denormal", "ascending"])
def test_evict_ties_and_special_weights(kind):
    """Ties go to the lowest token; -0 ties with +0; NaN and infinity count as
    the largest; weights that differ in their last bit are told apart."""
    n, heads, page, budget, recent = 1500, 2, 16, 400, 30
    rng = np.random.default_rng(3)
    cap = -(-n // page) * page
    if kind == "equal":
        w = np.full((1, heads, cap), 0.25, np.float32)
    elif kind == "few":
        w = rng.integers(0, 4, (1, heads, cap)).astype(np.float32)
    elif kind == "zeros":
        w = np.where(rng.random((1, heads, cap)) < 0.5, np.float32(-0.0), np.float32(0.0)).astype(np.float32)
    elif kind == "special":
        w = rng.standard_normal((1, heads, cap)).astype(np.float32)
        w[..., ::7], w[..., 3::50], w[..., 5::11] = np.inf, np.nan, -np.inf
    elif kind == "denormal":
        w = (rng.integers(0, 3000, (1, heads, cap)).astype(np.uint32)).view(np.float32)
    else:
        w = (np.uint32(0x3F800000) + np.arange(heads * cap, dtype=np.uint32)).view(np.float32).reshape(1, heads, cap)
    _evict_case("bf16", [n], heads, 64, page, budget, recent, np.ascontiguousarray(w), 21)


def test_evict_into_another_pool():
    rng = np.random.default_rng(8)
    w = rng.random((2, 2, 256)).astype(np.float32)
    _evict_case("mxfp4", [250, 90], 2, 128, 64, 100, 10, w, 31, other_pool=True)


def test_evict_zero_budget_and_masked_pages():
    """budget 0 keeps nothing; a kept token of a page outside the pool is left out of the copy alone."""
    import torch
    import block_scaled_fp4_03_amd as fp4
    cache = fp4.KVCache.empty(4, 16, 1, 64)
    _fill(cache, 40)
    before = _bits(cache.k).copy()
    table = to_dev(np.array([[0, 9]], np.int32))
    lens = to_dev(np.array([32], np.int32))
    w = torch.zeros((1, 1, 32), device="cuda")
    say("evict to nothing")
    out_lens, out_w, kept = fp4.kv_evict(cache, table, lens, w, 0, 0, to_dev(np.array([[2]], np.int32)))
    assert to_host(out_lens)[0] == 0 and kept.numel() == 0 and not to_host(out_w).any()
    np.testing.assert_array_equal(_bits(cache.k), before)
    say("evict with a page outside the pool")
    out_lens, out_w, kept = fp4.kv_evict(cache, table, lens, w, 20, 8, to_dev(np.array([[2, 3]], np.int32)))
    np.testing.assert_array_equal(to_host(kept)[0, 0], list(range(12)) + list(range(24, 32)))
    before[2, :, :12] = before[0, :, :12]
    np.testing.assert_array_equal(_bits(cache.k), before)


@pytest.mark.parametrize("n,budget,recent,levels", [(40000, 5000, 100, 0), (70001, 33000, 7, 50), (33000, 32999, 0, 3),
                                                    (32768, 1, 0, 0), (32769, 32768, 32768, 0), (100000, 70000, 0, 1)])
def test_evict_long_sequences(n, budget, recent, levels):
    """Sequences past what a workgroup holds in registers; weights of few distinct levels tie across its pieces."""
    rng = np.random.default_rng(n)
    cap = -(-n // 64) * 64
    w = rng.random((1, 1, cap)) if levels == 0 else rng.integers(0, levels, (1, 1, cap))
    _evict_case("mxfp4", [n], 1, 64, 64, budget, recent, w.astype(np.float32), 51)
