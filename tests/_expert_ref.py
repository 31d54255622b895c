"""Plain 64-bit implementations of the expert operators (numpy), for the tests:
the gate, its gradient, row quantisation and the experts' products, written
from their formulas, one token or one expert at a time."""
import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def scores(l, softmax):
    """l float64 [E] -> (scores, clamped logits, available)."""
    ok = l > -np.inf  # False for NaN
    x = np.where(ok, np.minimum(l, F32_MAX), 0.0)
    s = np.zeros_like(x)
    if not ok.any():
        return s, x, ok
    if softmax:
        e = np.exp(x[ok] - x[ok].max())
        s[ok] = e / e.sum()
    else:
        with np.errstate(over="ignore"):
            s[ok] = 1.0 / (1.0 + np.exp(-x[ok]))
    return s, x, ok


def gate_row(l, K, softmax, bias, groups, topk_groups, group_top, renorm, scale):
    """One token: (ids, weights, keys) in 64 bits; keys are -inf where an expert
    cannot be picked."""
    E = l.shape[0]
    s, x, ok = scores(l, softmax)
    c = s if bias is None else s + bias
    key = x.copy() if bias is None else c.copy()
    key[~ok] = -np.inf
    key[~(key > -np.inf)] = -np.inf
    if groups > 1 and topk_groups < groups:
        per = E // groups
        gs = []
        for g in range(groups):
            part = slice(g * per, (g + 1) * per)
            live = key[part] > -np.inf
            if group_top == 1:
                gs.append(key[part].max())
            else:
                two = np.sort(c[part][live])[::-1][:2]
                gs.append(two.sum() if two.size else -np.inf)
        order = sorted(range(groups), key=lambda g: (-gs[g], g))
        for g in order[topk_groups:]:
            key[g * per:(g + 1) * per] = -np.inf
    order = sorted(range(E), key=lambda e: (-key[e], e))[:K]
    ids = [e if key[e] > -np.inf else -1 for e in order]
    return np.array(ids), weights_of(l, ids, softmax, renorm, scale), key


def shares(x, softmax):
    """s_k / sum_j s_j of picks with logits x, by the scores' logarithms."""
    log_s = x if softmax else -np.logaddexp(0.0, -x)
    q = np.exp(log_s - log_s.max())
    return q / q.sum()


def weights_of(l, ids, softmax, renorm, scale):
    s, x, _ = scores(l, softmax)
    ids = np.asarray(ids)
    w = np.zeros(len(ids))
    at = np.nonzero(ids >= 0)[0]
    if at.size:
        w[at] = shares(x[ids[at]], softmax) if renorm else s[ids[at]]
    return w * scale


def gate_grad_row(l, ids, g, softmax, renorm, scale):
    """Gradient of sum_k g_k w_k with respect to one token's logits."""
    s, x, ok = scores(l, softmax)
    d = np.zeros_like(s)
    at = [(k, e) for k, e in enumerate(ids) if 0 <= e < len(s) and ok[e]]
    if not at:
        return d
    up = scale * np.array([g[k] for k, _ in at])
    e = np.array([e for _, e in at])
    if renorm:
        q = shares(x[e], softmax)
        d[e] = (up - (up * q).sum()) * q
        if not softmax:
            d[e] *= np.exp(-np.logaddexp(0.0, x[e]))  # 1 - s
        return d
    sk = s[e]
    if softmax:
        d[e] = up
        return s * (d - (up * sk).sum())
    with np.errstate(over="ignore"):
        d[e] = up * sk / (1.0 + np.exp(x[e]))
    return d


def quantize(v):
    """v float64 [rows, cols] -> (exact v / scale, scale)."""
    top = np.abs(v).max(1)
    scale = np.where(top > 0, top / 127.0, 1.0)
    return v / scale[:, None], scale


def swiglu(x):
    c = x.shape[1] // 2
    a, b = x[:, :c], x[:, c:]
    with np.errstate(over="ignore"):
        return a / (1.0 + np.exp(-a)) * b


def matmul(x, xs, w, ws, offs, layout, cap, row_src, rows):
    """(out, magnitude, written): magnitude = the same sum over |x||w|."""
    E, Nc, Kd = w.shape
    out = np.zeros((rows, Nc))
    mag = np.zeros((rows, Nc))
    written = np.zeros(rows, dtype=bool)
    for e in range(E):
        n = int(offs[e + 1]) - int(offs[e])
        if layout == 1:
            n = min(n, cap)
        we = w[e].astype(np.float64)
        for i in range(n):
            r = e * cap + i if layout == 1 else int(offs[e]) + i
            src = r if row_src is None else int(row_src[int(offs[e]) + i])
            written[r] = True
            if not 0 <= src < x.shape[0]:
                continue
            xr = x[src].astype(np.float64)
            f = float(xs[src]) * ws[e].astype(np.float64)
            out[r] = (we @ xr) * f  # integers below 2^53: exact
            mag[r] = (np.abs(we) @ np.abs(xr)) * np.abs(f)
    return out, mag, written
