"""fp4_attn_decode where NaN lies in valid places: a sequence whose query or
keys hold one has NaN in its output, its log-sum-exp and the weights of the
tokens it attends to, whichever wave and piece meets it; other sequences, other
kv heads and masked tokens are left alone."""
import numpy as np
import pytest

import test_gpu_attn_decode as attn
from gpu_helpers import say, to_dev, to_host

pytestmark = pytest.mark.gpu


def _call(pools, q, table, lens, window=0, f32=False):
    import torch
    import block_scaled_fp4_03_amd as fp4
    cache = attn.cache_of(pools)
    B, Hq = q.shape[:2]
    cap = table.shape[1] * cache.page_size
    w_in = np.random.default_rng(0).random((B, cache.kv_heads, cap)).astype(np.float32)
    w_out, lse = torch.full((B, cache.kv_heads, cap), -7.0, device="cuda"), torch.empty((B, Hq), device="cuda")
    qd = torch.from_numpy(q).cuda().to(torch.float32 if f32 else torch.bfloat16)
    out = fp4.decode_attention(qd, cache, to_dev(table), to_dev(np.array(lens, np.int32)), window=window, lse=lse,
                               weights=to_dev(w_in), weights_out=w_out)
    return out.float().cpu().numpy(), to_host(lse), w_in, to_host(w_out)


@pytest.mark.parametrize("f32", (False, True))
@pytest.mark.parametrize("n", (1, 20, 300, 3000, 20000))
def test_nan_query(n, f32):
    """One element of one head's query: that head's results, and its kv head's weights."""
    page, D, G = 16, 64, 2
    width = -(-n // page)
    pools = attn.make(5, "bf16", 2 * width, 2, page, D)
    q = np.random.default_rng(n).standard_normal((2, 2 * G, D)).astype(np.float32)
    q[0, 1, 7] = np.nan
    say("attention, NaN in a query, %d tokens, f32 %d" % (n, f32))
    table = np.arange(2 * width, dtype=np.int32).reshape(2, width)
    out, lse, w_in, w_out = _call(pools, q, table, [n, n], f32=f32)
    bad = np.zeros((2, 2 * G), bool)
    bad[0, 1] = True
    assert (np.isnan(out).all(axis=2) == bad).all() and np.isfinite(out[~bad]).all()
    assert (np.isnan(lse) == bad).all() and np.isfinite(lse[~bad]).all()
    assert np.isnan(w_out[0, 0, :n]).all()
    assert np.isfinite(w_out[0, 1]).all() and np.isfinite(w_out[1]).all()


@pytest.mark.parametrize("n,tile", [(100, 0), (300, 1), (300, 2), (300, 3), (300, 9), (5000, 70), (20000, 623)])
def test_a_tile_of_nan_keys(n, tile):
    """32 tokens, all of one wave's step: every score there is NaN, others are not."""
    page, D, G = 16, 64, 3
    width = -(-n // page)
    pools = attn.make(6, "bf16", width, 2, page, D)
    for t in range(32 * tile, min(32 * tile + 32, n)):
        pools[0][0][t // page, 1, t % page] = 0x7FC0
    q = np.random.default_rng(n).standard_normal((1, 2 * G, D)).astype(np.float32)
    say("attention, a tile of NaN keys, %d tokens, tile %d" % (n, tile))
    out, lse, w_in, w_out = _call(pools, q, np.arange(width, dtype=np.int32).reshape(1, width), [n])
    assert np.isfinite(out[0, :G]).all() and np.isfinite(lse[0, :G]).all() and np.isfinite(w_out[0, 0, :n]).all()
    assert np.isnan(out[0, G:]).all()
    assert np.isnan(lse[0, G:]).all()
    assert np.isnan(w_out[0, 1, :n]).all()


@pytest.mark.parametrize("window", (0, 40, 75))
def test_masked_tokens_beside_nan(window):
    """Tokens before the window and in pages outside the pool keep their weights."""
    page, D, n = 16, 64, 150
    pools = attn.make(7, "bf16", 10, 1, page, D)
    table = np.arange(10, dtype=np.int32).reshape(1, 10)
    table[0, 6] = -1
    pools[0][0][9, 0, :] = 0x7FC0                         # tokens 144 .. 149, attended to
    q = np.random.default_rng(1).standard_normal((1, 2, D)).astype(np.float32)
    say("attention, masked tokens beside NaN, window %d" % window)
    out, lse, w_in, w_out = _call(pools, q, table, [n], window=window)
    t = np.arange(n)
    masked = (t // page == 6) | (t < n - window if window else False)
    assert np.isnan(out).all() and np.isnan(lse).all()
    np.testing.assert_array_equal(w_out[0, 0, :n][masked], w_in[0, 0, :n][masked])
    assert np.isnan(w_out[0, 0, :n][~masked]).all()
    assert (w_out[0, 0, n:] == -7.0).all()
