"""The router, rows in expert order and back, and the few-token 4-bit products
(oracle; test infrastructure): float64 numpy from the definitions, one token
and one slot at a time where that is plainest."""

import numpy as np

from .formats import decode_e2m1, decode_e8m0, unpack_e2m1x2


def scores(logits, gate: str) -> np.ndarray:
    """softmax over a row (a row without any expert: zeros) or the sigmoid."""
    x = np.asarray(logits, dtype=np.float64)
    if gate == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def gate_weights(logits, ids, gate: str, renormalize: bool, scale: float = 1.0) -> np.ndarray:
    """Weights of given ids (outside [0, E): 0).  The renormalized sigmoid is formed as
    e^(log sigma - max log sigma) over its sum, so that far negative logits stay apart."""
    x = np.asarray(logits, dtype=np.float64)
    ids = np.asarray(ids)
    on = (ids >= 0) & (ids < x.shape[1])
    at = np.where(on, ids, 0)
    if renormalize:
        v = np.where(on, np.take_along_axis(x, at, 1), -np.inf)
        if gate == "sigmoid":
            v = -np.logaddexp(0.0, -v)
        top = v.max(axis=1, keepdims=True)
        e = np.exp(v - np.where(np.isneginf(top), 0.0, top))
        s = e.sum(axis=1, keepdims=True)
        w = e / np.where(s == 0, 1.0, s)
    else:
        w = np.take_along_axis(scores(x, gate), at, 1)
    return np.where(on, scale * w, 0.0)


def moe_route(logits, k: int, gate="softmax", bias=None, renormalize=False, scale: float = 1.0):
    """(ids [T, k], weights [T, k] float64); no NaN or +inf here (see gate_weights for the weights)."""
    x = np.asarray(logits, dtype=np.float64)
    key = x if bias is None else np.where(np.isneginf(x), -np.inf, scores(x, gate) + np.asarray(bias, np.float64))
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids = np.where(np.isneginf(np.take_along_axis(key, ids, 1)), -1, ids).astype(np.int32)
    return ids, gate_weights(x, ids, gate, renormalize, scale)


def moe_route_backward(logits, ids, dw, gate="softmax", renormalize=False, scale: float = 1.0) -> np.ndarray:
    """d/dlogits of sum(dw * gate_weights), by the chain rule written out per token."""
    x = np.asarray(logits, dtype=np.float64)
    dw = np.asarray(dw, dtype=np.float64)
    T, E = x.shape
    s = scores(x, gate)
    out = np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        e = [int(ids[t, j]) for j in on]
        u = scale * dw[t, on]
        if renormalize:
            p = gate_weights(x[t:t + 1], ids[t:t + 1], gate, True)[0, on]
            d = p * (u - np.dot(u, p))                     # softmax of the chosen (log) scores
            if gate == "sigmoid":
                d = d * (1.0 - s[t, e])                    # d log sigma / dl
            np.add.at(out[t], e, d)
        elif gate == "sigmoid":
            np.add.at(out[t], e, u * s[t, e] * (1.0 - s[t, e]))
        else:
            g = np.zeros(E)
            np.add.at(g, e, u)
            out[t] = s[t] * (g - np.dot(g, s[t]))
    return out


def rows_from_tokens(tokens, w, src_to_row, total: int, rows) -> np.ndarray:
    """A copy of `rows` with [0, total) zeroed and each pair's row set to w * token."""
    tokens = np.asarray(tokens, dtype=np.float64)
    out = np.array(rows, dtype=np.float64)
    out[:min(total, out.shape[0])] = 0.0
    k = src_to_row.size // tokens.shape[0]
    for p, r in enumerate(src_to_row):
        if 0 <= r < out.shape[0]:
            out[r] = (1.0 if w is None else float(w.reshape(-1)[p])) * tokens[p // k]
    return out


def tokens_from_rows(rows, w, src_to_row, T: int) -> np.ndarray:
    rows = np.asarray(rows, dtype=np.float64)
    out = np.zeros((T, rows.shape[1]))
    k = src_to_row.size // T
    for p, r in enumerate(src_to_row):
        if 0 <= r < rows.shape[0]:
            out[p // k] += (1.0 if w is None else float(w.reshape(-1)[p])) * rows[r]
    return out


def pair_dots(tokens, rows, src_to_row) -> np.ndarray:
    tokens, rows = np.asarray(tokens, dtype=np.float64), np.asarray(rows, dtype=np.float64)
    T = tokens.shape[0]
    k = src_to_row.size // T
    out = np.zeros((T, k))
    for p, r in enumerate(src_to_row):
        if 0 <= r < rows.shape[0]:
            out[p // k, p % k] = np.dot(tokens[p // k], rows[r])
    return out


def fp4_weights(b, b_scales) -> np.ndarray:
    """[..., N, K/2] codes and [..., N, K/32] E8M0 bytes to [..., N, K] values."""
    v = decode_e2m1(unpack_e2m1x2(b))
    return v * np.repeat(decode_e8m0(b_scales), 32, axis=-1)


def moe_gemv_fp4(x, weights, ids=None, w=None, silu_mul=False):
    """x [T, K] or [T, k, K], weights [G, N, K] (fp4_weights).  Returns (result, magnitude):
    magnitude is the same sum over absolute products, the scale that rounding errors are
    measured against (with silu_mul: of the gate and up halves, [..., 2, N])."""
    x = np.asarray(x, dtype=np.float64)
    T = x.shape[0]
    G, rows, _ = weights.shape
    k = 1 if ids is None else ids.shape[1]
    y, mag = np.zeros((T, k, rows)), np.zeros((T, k, rows))
    for t in range(T):
        for j in range(k):
            e = 0 if ids is None else int(ids[t, j])
            if 0 <= e < G:
                xt = x[t, j] if x.ndim == 3 else x[t]
                y[t, j] = weights[e] @ xt
                mag[t, j] = np.abs(weights[e]) @ np.abs(xt)
    if w is not None:
        on = (ids >= 0) & (ids < G)
        wt = np.where(on, np.asarray(w, dtype=np.float64), 0.0)[..., None]
        return (y * wt).sum(1), (mag * np.abs(wt)).sum(1)
    if silu_mul:
        h = rows // 2
        g, u = y[..., :h], y[..., h:]
        with np.errstate(over="ignore"):
            y = g / (1.0 + np.exp(-g)) * u
        mag = np.stack((mag[..., :h], mag[..., h:]), axis=-2)
        return (y, mag, g, u)
    return (y[:, 0], mag[:, 0]) if ids is None else (y, mag)
