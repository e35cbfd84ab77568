"""Reference of the second half of a block in numpy float64, written out from the definitions: the residual add between
norms and the gated feed-forward product, each with its gradients.  Test infrastructure: shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v)


def act(v, how):
    v = np.asarray(v, dtype=np.float64)
    if how == "relu":
        return np.maximum(v, 0.0)
    if how == "gelu":
        return v * 0.5 * (1.0 + erf(v / math.sqrt(2.0)))
    if how == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    y = 0.5 * (1.0 + np.tanh(0.5 * v))
    return y if how == "sigmoid" else v * y


def slope(v, how):
    """The derivative of act."""
    v = np.asarray(v, dtype=np.float64)
    if how == "relu":
        return (v > 0).astype(np.float64)
    if how == "gelu":
        return 0.5 * (1.0 + erf(v / math.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if how == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (v + 0.044715 * v ** 3))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * v * v)
    y = 0.5 * (1.0 + np.tanh(0.5 * v))
    return y * (1.0 - y) if how == "sigmoid" else y + v * y * (1.0 - y)


def glu(x, wg, wu, bg=None, bu=None, how="silu"):
    """(h, g, u)"""
    g = x @ wg.T + (0.0 if bg is None else bg)
    u = x @ wu.T + (0.0 if bu is None else bu)
    return act(g, how) * u, g, u


def glu_bwd(dh, x, wg, wu, bg=None, bu=None, how="silu"):
    """(dx, dwg, dwu, dbg, dbu)"""
    _, g, u = glu(x, wg, wu, bg, bu, how)
    dg, du = dh * u * slope(g, how), dh * act(g, how)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg.sum(0), du.sum(0)


def rows_of(v, rows, C, none):
    """A vector as one per row: [C], or [groups, C] with the rows cut into that many runs; none where it is None."""
    if v is None:
        return np.full((rows, C), none)
    v = np.asarray(v, dtype=np.float64).reshape(-1, C)
    return np.repeat(v, rows // len(v), axis=0)


def to_vector(t, like, C):
    """Rows summed to the shape of the vector `like`."""
    if like is None:
        return t.sum(0)
    groups = np.asarray(like).size // C
    return t.reshape(groups, -1, C).sum(1).reshape(np.shape(like))


def moments(v, kind, eps):
    """Mean (zeros for root mean square) and inverse deviation of each row."""
    mean = v.mean(-1) if kind == "layer" else np.zeros(len(v))
    d = v - mean[:, None]
    return mean, 1.0 / np.sqrt((d * d).mean(-1) + eps)


def addnorm(x, y, w=None, b=None, gate=None, post_w=None, post_b=None, norm="layer", post="none", scale=1.0, residual=1.0,
            eps=1e-5):
    """{s, h, mean, rstd, post_mean, post_rstd} of [rows, C]; None for what a missing norm has not."""
    rows, C = x.shape
    V = lambda v, none: rows_of(v, rows, C, none)
    out = dict.fromkeys(("s", "h", "mean", "rstd", "post_mean", "post_rstd"))
    z = y
    if post != "none":
        m, r = out["post_mean"], out["post_rstd"] = moments(y, post, eps)
        z = (y - m[:, None]) * r[:, None] * V(post_w, 1.0) + V(post_b, 0.0)
    out["s"] = residual * x + scale * V(gate, 1.0) * z
    if norm != "none":
        m, r = out["mean"], out["rstd"] = moments(out["s"], norm, eps)
        out["h"] = (out["s"] - m[:, None]) * r[:, None] * V(w, 1.0) + V(b, 0.0)
    return out


def addnorm_bwd(dh, ds, s, y, w=None, gate=None, post_w=None, post_b=None, norm="layer", post="none", scale=1.0, residual=1.0,
                mean=None, rstd=None, post_mean=None, post_rstd=None, b=None):
    """{dx, dy, dw, db, dgate, dpost_w, dpost_b} at the given statistics (b: only for the shape of db)."""
    rows, C = y.shape
    V = lambda v, none: rows_of(v, rows, C, none)
    column = lambda v: 0.0 if v is None else np.asarray(v, dtype=np.float64).reshape(rows, 1)

    def back(q, f, r, kind):
        out = q - f * (q * f).mean(-1, keepdims=True)
        return r * (out - q.mean(-1, keepdims=True) if kind == "layer" else out)

    out = {}
    D = np.zeros((rows, C)) if ds is None else ds
    if norm != "none":
        e = (s - column(mean)) * column(rstd)
        D = D + back(dh * V(w, 1.0), e, column(rstd), norm)
        out["dw"], out["db"] = to_vector(dh * e, w, C), to_vector(dh, w if b is None else b, C)
    out["dx"] = residual * D
    f = y if post == "none" else (y - column(post_mean)) * column(post_rstd)
    q = scale * D * V(gate, 1.0)
    out["dgate"] = to_vector(scale * D * (f * V(post_w, 1.0) + V(post_b, 0.0)), gate, C)
    if post != "none":
        out["dpost_w"], out["dpost_b"] = (q * f).sum(0), q.sum(0)
        out["dy"] = back(q * V(post_w, 1.0), f, column(post_rstd), post)
    else:
        out["dy"] = q
    return out
