"""Plain FP64 forms of the decode-step operators (paged cache attention,
eviction, log probabilities and their gradient), for their tests.  Written
from the definitions in include/fp4.h; no code of the library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def e4m3(codes):
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where(c & 128, -mag, mag)


def row_values(codes, scales, fmt):
    """FP64 values of cache rows (..., row bytes): fmt "bf16" (uint16 bits), "mxfp8" or "mxfp4"."""
    if fmt == "bf16":
        return (np.asarray(codes).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    if fmt == "mxfp8":
        x = e4m3(codes)
    else:
        x = E2M1[np.stack([codes & 15, codes >> 4], -1)].reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    s = 2.0 ** (np.asarray(scales).astype(np.float64) - 127.0)
    return x * np.repeat(s, 32, axis=-1)


def softmax(s):
    m = s.max(axis=-1, keepdims=True)
    e = np.exp(s - m)
    return e / e.sum(axis=-1, keepdims=True)


def attend(q, K, V, scale):
    """q: G x D, K, V: T x D.  Returns out G x D, lse G, p G x T, s G x T."""
    if len(K) == 0:
        return np.zeros((len(q), V.shape[1])), np.full(len(q), -np.inf), np.zeros((len(q), 0)), np.zeros((len(q), 0))
    s = scale * (q @ K.T)
    p = softmax(s)
    m = s.max(axis=1)
    return p @ V, m + np.log(np.exp(s - m[:, None]).sum(axis=1)), p, s


def evict(weights, n, budget, recent):
    """The kept token numbers of one (sequence, head) with n tokens, ascending."""
    if n <= budget:
        return list(range(n))
    last = min(recent, budget)
    order = sorted(range(n - last), key=lambda t: (-np.inf if np.isnan(weights[t]) else -weights[t], t))
    # A NaN sorts with +inf here; it goes before it.
    order.sort(key=lambda t: 0 if np.isnan(weights[t]) else 1)
    return sorted(order[:budget - last]) + list(range(n - last, n))


def log_softmax(y):
    m = y.max(axis=-1, keepdims=True)
    return y - (m + np.log(np.exp(y - m).sum(axis=-1, keepdims=True)))


def logprobs_loss(x, tokens, scale, g, ge):
    """sum_j g_j logp_j + ge * entropy of one row, in the precision of x."""
    lp = log_softmax(scale * x)
    ok = (tokens >= 0) & (tokens < len(x))
    p = np.exp(lp)
    ent = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum()
    return (g[ok] * lp[tokens[ok]]).sum() + ge * ent


def logprobs_grad(x, tokens, scale, g, ge):
    """The gradient's formula for one row."""
    with np.errstate(invalid="ignore"):
        lp = log_softmax(scale * x)
    p = np.exp(lp)
    h = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum()
    ok = (tokens >= 0) & (tokens < len(x))
    d = np.where(p > 0, -p * (g[ok].sum() + ge * (np.where(p > 0, lp, 0.0) + h)), 0.0)
    np.add.at(d, tokens[ok], g[ok])
    return scale * d
