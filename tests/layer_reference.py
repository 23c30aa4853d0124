"""Plain FP64 forms of the operators around a layer's products (norms with
rotary positions, routing to experts, verification of drafts), for their tests.
Written from the definitions in include/fp4.h; no code of the library."""
import numpy as np


# ---- norms and rotary positions ----------------------------------------------
def axis_of_pairs(sections, cyclic):
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, order = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                order.append(a)
    return order


def cos_sin(pos, freq, axis):
    """pos: axes x rows, freq: FP32 pairs.  The angle in 64-bit mantissas."""
    angle = np.asarray(pos).astype(np.longdouble)[list(axis)].T * np.asarray(freq).astype(np.longdouble)
    return np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]


def _pairs(x, R, interleaved):
    return (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])


def rotate(x, c, s, R, interleaved):
    out = x.copy()
    a, b = _pairs(x, R, interleaved)
    oa, ob = _pairs(out, R, interleaved)
    oa[...] = a * c - b * s
    ob[...] = b * c + a * s
    return out


def norm_rope(x, w, eps, c, s, R, interleaved):
    """x: rows x heads x D."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(x, c, s, R, interleaved)


def norm_rope_grad(x, w, eps, c, s, R, interleaved, g):
    """dx, dw (None without w), and the sums of magnitudes that bound their rounding."""
    g = rotate(g, c, -s, R, interleaved)
    mag = rotate_magnitude(g, R, interleaved)
    if w is None:
        return g, None, mag, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xn, t = x * r, g * w
    dx = r * (t - xn * (xn * t).mean(-1, keepdims=True))
    dmag = r * (mag * np.abs(w) + np.abs(xn) * (np.abs(xn) * mag * np.abs(w)).mean(-1, keepdims=True))
    return dx, (g * xn).sum((0, 1)), dmag, (mag * np.abs(xn)).sum((0, 1))


def rotate_magnitude(x, R, interleaved):
    """|a| + |b| of every value's pair: what the rotation's rounding goes by."""
    out = np.abs(x)
    a, b = _pairs(out, R, interleaved)
    total = a + b
    a[...] = total
    b[...] = total
    return out


# ---- routing -----------------------------------------------------------------
def route(x, k, renormalise):
    """ids, weights of each token."""
    T, E = x.shape
    ids, weights = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        key = [(0 if np.isnan(v) else 1, 0.0 if np.isnan(v) else -v, e) for e, v in enumerate(x[t])]
        ids[t] = [e for _, _, e in sorted(key)[:k]]
        over = x[t, ids[t]] if renormalise else x[t]
        top = over.max()
        if top == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            weights[t] = np.exp(x[t, ids[t]] - top) / np.exp(over - top).sum()
    return ids, weights


def route_grad(x, ids, g, renormalise):
    T, E = x.shape
    full, chosen = np.zeros((T, E)), np.zeros((T, E), bool)
    for t in range(T):
        for e, v in zip(ids[t], g[t]):
            if 0 <= e < E:
                full[t, e] += v
                chosen[t, e] = True
    y = np.where(chosen, x, -np.inf) if renormalise else x
    top = y.max(1, keepdims=True)
    p = np.exp(y - np.where(top == -np.inf, 0.0, top))
    z = p.sum(1, keepdims=True)
    p = p / np.where(z == 0.0, 1.0, z)
    return p * (full - (p * full).sum(1, keepdims=True)), p, full


def sort(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    b = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(b, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    off = np.concatenate([[0], np.cumsum(np.bincount(b, minlength=E + 1))[:E]])
    off[E] = T * k
    return off, order // max(k, 1), np.where(b < E, pos, -1 - pos).reshape(T, k)


# ---- drafts ------------------------------------------------------------------
def probabilities(x, temperature):
    """The softmax over the temperature, or None without a distribution."""
    if np.isnan(x).any() or x.max() in (np.inf, -np.inf):
        return None
    with np.errstate(over="ignore", under="ignore"):
        p = np.exp((x - x.max()) / temperature) if np.isfinite(temperature) else (x > -np.inf).astype(np.float64)
    return p / p.sum()


def verify(target, draft, tokens, u, temperature):
    """One sequence: target (G + 1) x V, draft G x V or None.  (tokens, kept, chances)."""
    G, V = len(tokens), target.shape[1]
    greedy = not temperature > 0.0
    out, kept, chance = [], None, []
    for i in range(G + 1):
        x = target[i]
        if greedy:
            p = probabilities(x, 1.0)
            if p is not None:
                p = np.eye(1, V, int(np.argmax(x)))[0]
        else:
            p = probabilities(x, temperature)
        live = i < G and 0 <= tokens[i] < V
        q = np.zeros(V)
        keep, odds = False, 0.0
        if live and p is not None:
            d = tokens[i]
            if greedy:
                keep, odds = p[d] == 1.0, p[d]
            else:
                q1 = np.eye(1, V, d)[0] if draft is None else probabilities(draft[i], temperature)
                if q1 is not None:
                    q = q1
                    keep = u[i] * q[d] < p[d]
                    odds = float(p[d] > 0.0) if p[d] >= q[d] else p[d] / q[d]
        if i < G:
            chance.append(odds)
        if kept is not None:
            continue
        if keep:
            out.append(int(tokens[i]))
            continue
        kept = i
        if p is None:
            continue
        r = np.maximum(p - q, 0.0)
        if r.sum() == 0.0:
            r = p
        c = np.cumsum(r)
        past = np.nonzero((c > u[G] * c[-1]) & (r > 0.0))[0]
        out.append(int(past[0]))
    return out + [-1] * (G + 1 - len(out)), kept, chance
