"""The attention block's linear layers and position rotation (oracle; test infrastructure only).

The pages describe none of these, so they are the plain definitions:

* linear: h = x W^T + b in float64 on the decoded weight, then SiLU, GELU (by
  the error function) or SwiGLU (rows [0, N/2) gate, [N/2, N) up), then the
  residual;
* rotation: pairs (i, i + rot/2) or (2i, 2i + 1) of a head's first ``rot``
  elements, (a, b) -> (a cos - b sin, b cos + a sin), the two products and the
  sum each rounded to float32.
"""

from __future__ import annotations

import math

import numpy as np

from . import formats

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def linear(x, w, scale, bias=None, act=None, residual=None):
    """float64 [T, columns] and ``slack``, the change of each result for a change of every h by the given share of
    ``size`` = sum |x w| + |b|: |result(h + e size) - result(h)| <= e slack + O(e^2), the residual's own size on top."""
    x = np.asarray(x, np.float64)
    W = formats.e2m1_decode(formats.unpack_nibbles(w)) * np.repeat(formats.e8m0_decode(scale), 32, axis=-1)
    h = x @ W.T
    size = np.abs(x) @ np.abs(W).T
    if bias is not None:
        h = h + np.asarray(bias, np.float64)
        size = size + np.abs(np.asarray(bias, np.float64))
    if act == "swiglu":
        n = h.shape[1] // 2
        g, u = h[:, :n], h[:, n:]
        s = _silu(g)
        out = s * u
        slack = 1.1 * size[:, :n] * np.abs(u) + np.abs(s) * size[:, n:]  # |SiLU'| < 1.1
    elif act == "silu":
        out, slack = _silu(h), 1.1 * size
    elif act == "gelu":
        out, slack = 0.5 * h * _erfc(-h / math.sqrt(2.0)), 1.13 * size  # |GELU'| < 1.13
    else:
        out, slack = h, size
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
    return out, slack


def _silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def rotate(x, row, interleaved=False):
    """float32 rows [..., D] rotated by one table row (rot/2 cosines, rot/2 sines)."""
    x, row = np.asarray(x, np.float32), np.asarray(row, np.float32)
    rot = len(row)
    c, s = row[: rot // 2], row[rot // 2:]
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        if interleaved:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
        else:
            a, b = x[..., : rot // 2], x[..., rot // 2: rot]
            y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    return y
