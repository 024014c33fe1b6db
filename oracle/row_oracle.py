"""Plain float64 definitions of the row passes around the attention: the norm
and several-axis rotation of Q and K, the modulated norm, the gated residual
update, and their gradients, written from the formulas.

Arrays are numpy float64, or anything with the same +, -, *, mean, sum,
indexing and an rsqrt method (the tests put numbers with error bounds through
the same lines)."""
from __future__ import annotations

import numpy as np

__all__ = ["rope_ladder", "grid_positions", "rope_angles", "rotate", "rotate_back", "qk_norm_rope",
           "qk_norm_rope_backward", "gate_residual_norm", "gate_residual_norm_backward"]


def _rsqrt(v):
    return v.rsqrt() if hasattr(v, "rsqrt") else 1.0 / np.sqrt(v)


# ------------------------------------------------------------- rotations --
def rope_ladder(pairs, theta, scale=(1.0, 1.0, 1.0), shared=False):
    """(axis, frequency) of every rotated pair."""
    axis, freq, total = [], [], sum(pairs)
    for a in range(3):
        for i in range(pairs[a]):
            freq.append(scale[a] * (theta[0] ** (-len(freq) / total) if shared else theta[a] ** (-i / pairs[a])))
            axis.append(a)
    return np.array(axis, dtype=int), np.array(freq, dtype=np.float64)


def grid_positions(rows, offset, T, H, W):
    n = np.arange(rows, dtype=np.int64) + offset
    return np.stack([n // (H * W), n // W % H, n % W], axis=1)


def rope_angles(positions, axis, freq, d, text_tokens=0):
    """cos, sin [rows, 1, d / 2]; pairs past the ladder and the last
    text_tokens rows do not turn."""
    a = np.zeros((positions.shape[0], d // 2))
    a[:, : len(axis)] = positions[:, axis].astype(np.float64) * freq
    if text_tokens:
        a[positions.shape[0] - text_tokens:] = 0.0
    return np.cos(a)[:, None, :], np.sin(a)[:, None, :]


def _pairs(d, style):
    i = np.arange(d // 2)
    return (2 * i, 2 * i + 1) if style == "interleaved" else (i, i + d // 2)


def _place(first, second, d, style):
    """Pair halves [..., d / 2] back in channel order."""
    f, s = _pairs(d, style)
    order = np.empty(d, dtype=int)
    order[f], order[s] = np.arange(d // 2), np.arange(d // 2) + d // 2
    both = first.joined(second) if hasattr(first, "joined") else np.concatenate([first, second], axis=-1)
    return both[..., order]


def rotate(x, cos, sin, style):
    f, s = _pairs(x.shape[-1], style)
    a, b = x[..., f], x[..., s]
    return _place(a * cos - b * sin, a * sin + b * cos, x.shape[-1], style)


def rotate_back(x, cos, sin, style):
    f, s = _pairs(x.shape[-1], style)
    a, b = x[..., f], x[..., s]
    return _place(a * cos + b * sin, b * cos - a * sin, x.shape[-1], style)


def _qk_rstd(x, norm, eps):
    axes = (1, 2) if norm == "token" else (2,)
    return _rsqrt((x * x).mean(axis=axes, keepdims=True) + eps), axes


def qk_norm_rope(x, weight, cos, sin, norm, eps, style):
    """One of Q and K, [rows, heads, d]; weight [heads, d] or [1, d]."""
    if norm != "none":
        x = x * _qk_rstd(x, norm, eps)[0] * weight
    return rotate(x, cos, sin, style)


def qk_norm_rope_backward(g, x, weight, cos, sin, norm, eps, style):
    """(dx, dweight [heads, d] or [1, d])."""
    u = rotate_back(g, cos, sin, style)
    if norm == "none":
        return u, None
    r, axes = _qk_rstd(x, norm, eps)
    n = x * r
    dw = (u * n).sum(axis=(0,) if norm == "token" else (0, 1), keepdims=True)[0]
    u = u * weight
    return r * (u - n * (u * n).mean(axis=axes, keepdims=True)), dw


# ------------------------------------------------------------ row passes --
def _normed(x, kind, eps):
    """(xhat, rstd)."""
    if kind == "layer":
        x = x - x.mean(axis=(1,), keepdims=True)
    r = _rsqrt((x * x).mean(axis=(1,), keepdims=True) + eps)
    return x * r, r


def _normed_backward(u, hat, r, kind):
    d = u - hat * (u * hat).mean(axis=(1,), keepdims=True)
    if kind == "layer":
        d = d - u.mean(axis=(1,), keepdims=True)
    return r * d


def _rows_of(m, rows):
    """A parameter [groups, dim] spread over the rows."""
    return m if m.shape[0] in (1, rows) else m[np.repeat(np.arange(m.shape[0]), rows // m.shape[0])]


def _one(m):
    return 1.0 if m is None else m


def gate_residual_norm(x, y, p, norm, eps, post_norm, post_eps, residual_scale):
    """(x_out, h); y None: x_out is x; norm None: h is None.  p: dict of
    gate, scale, shift [groups, dim] and weight, bias, post_weight [1, dim],
    each None for the identity."""
    rows = x.shape[0]
    if y is not None:
        if post_norm != "none":
            y = _normed(y, post_norm, post_eps)[0]
        if p["post_weight"] is not None:
            y = y * p["post_weight"]
        if p["gate"] is not None:
            y = y * _rows_of(p["gate"], rows)
        x = x + y * residual_scale
    if norm is None:
        return x, None
    h = _normed(x, norm, eps)[0]
    h = h * _one(p["weight"]) if p["weight"] is not None else h
    h = h + p["bias"] if p["bias"] is not None else h
    h = h * (_rows_of(p["scale"], rows) + 1.0) if p["scale"] is not None else h
    return x, (h + _rows_of(p["shift"], rows) if p["shift"] is not None else h)


def gate_residual_norm_backward(dx_out, dh, x, y, p, norm, eps, post_norm, post_eps, residual_scale, groups=1):
    """dict of x, y and every parameter's gradient (modulations [groups, dim],
    weights [1, dim]); dx_out or dh None: no such gradient comes in."""
    out = {}

    def per_group(t):
        if groups == t.shape[0]:
            return t
        return t.reshape(groups, t.shape[0] // groups, t.shape[1]).sum(axis=(1,), keepdims=True)[:, 0]

    rows = (x if x is not None else dx_out).shape[0]
    yhat = yr = affine_y = None
    if y is not None:
        yhat, yr = (y, None) if post_norm == "none" else _normed(y, post_norm, post_eps)
        affine_y = yhat * p["post_weight"] if p["post_weight"] is not None else yhat
    g = dx_out
    if norm is not None:
        if y is not None:
            b = affine_y * _rows_of(p["gate"], rows) if p["gate"] is not None else affine_y
            x = x + b * residual_scale
        hat, r = _normed(x, norm, eps)
        affine = hat * p["weight"] if p["weight"] is not None else hat
        affine = affine + p["bias"] if p["bias"] is not None else affine
        out["shift"] = per_group(dh)
        out["scale"] = per_group(dh * affine)
        u = dh * (_rows_of(p["scale"], rows) + 1.0) if p["scale"] is not None else dh
        out["weight"] = (u * hat).sum(axis=(0,), keepdims=True)
        out["bias"] = u.sum(axis=(0,), keepdims=True)
        u = u * p["weight"] if p["weight"] is not None else u
        d = _normed_backward(u, hat, r, norm)
        g = d + g if g is not None else d
        out["x"] = g
    if y is not None:
        v = g * residual_scale
        out["gate"] = per_group(v * affine_y)
        v = v * _rows_of(p["gate"], rows) if p["gate"] is not None else v
        out["post_weight"] = (v * yhat).sum(axis=(0,), keepdims=True)
        v = v * p["post_weight"] if p["post_weight"] is not None else v
        out["y"] = _normed_backward(v, yhat, yr, post_norm) if yr is not None else v
    return out
