"""Norm and rotation of heads and the draw of a token, restated plainly in 64 bits (numpy). Shares no code with the
library."""
import numpy as np


def norm_rope(x, weight=None, eps=0.0, rows=None, interleaved=False):
    """x [n, heads, dim]; rows [n, turn] (cos | sin) or None. fp64. Also returns, for each element, the magnitudes that its
    sum was made of."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    size = np.abs(y)
    if rows is None:
        return y, size
    turn = rows.shape[1]
    c, s = (r.astype(np.float64)[:, None] for r in np.split(rows, 2, axis=1))
    out, size = y.copy(), size.copy()
    a = np.arange(turn // 2) * 2 if interleaved else np.arange(turn // 2)
    b = a + (1 if interleaved else turn // 2)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a], size[..., b] = (np.abs(y[..., a] * c) + np.abs(y[..., b] * s), np.abs(y[..., b] * c) + np.abs(y[..., a] * s))
    return out, size


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, probability, kept token numbers). logits 1-D, finite or -inf."""
    x = logits.astype(np.float64)
    ids = np.flatnonzero(x > -np.inf)
    if ids.size == 0:
        return -1, 0.0, ids
    m = x.max()
    if not temperature > 0:
        first = np.flatnonzero(x == m)[:1]
        return int(first[0]), 1.0, first
    w = np.exp((x - m) / np.float64(temperature))
    order = ids[np.lexsort((ids, -x[ids]))]                # falling, the lowest index first among equals
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
        take = before < np.float64(top_p) * w[order].sum()
        take[0] = True
        order = order[take]
    order = order[w[order] >= min(np.float64(min_p), 1.0)]
    kept = np.sort(order)
    sums = np.cumsum(w[kept])
    at = min(int((sums <= np.float64(u) * sums[-1]).sum()), len(kept) - 1)
    return int(kept[at]), float(w[kept[at]] / sums[-1]), kept
