"""Float64 CPU oracle of the 4-bit weights, straight from

  w[o][k] = scale[o][k / group] (code[o][k] - zero[o][k / group])
  Y = X W^T + bias,  dX = dY W

and of the rule by which codes are made (a scale rounded to bf16 first; codes to
the nearest, ties to even).  Besides a product's values it returns the sum of the
magnitudes of its terms: what a bound on a rounding error scales with.
"""
from __future__ import annotations

import numpy as np

from input_adaptive_rank_amd.synth import round_bf16


def _wide(t, group, c1):
    return np.repeat(np.asarray(t, dtype=np.float64), group, axis=1)[:, :c1]


def weight(codes, scale, zero, group):
    """codes [c2][c1] 0 .. 15; zero None: 8."""
    c1 = codes.shape[1]
    return _wide(scale, group, c1) * (codes - (8.0 if zero is None else _wide(zero, group, c1)))


def unpack(nibbles):
    """[c2][c1 / 2] bytes to [c2][c1] codes, the even column in the low half."""
    out = np.empty((nibbles.shape[0], 2 * nibbles.shape[1]))
    out[:, 0::2], out[:, 1::2] = nibbles & 15, nibbles >> 4
    return out


def quantise(W, group, zero_points):
    """(codes, scale, zero or None); W as the storage holds it.  Quotients are
    formed in float32, as the device forms them."""
    f = np.float32
    c2, c1 = W.shape
    groups = -(-c1 // group)
    codes, scale = np.empty((c2, c1)), np.empty((c2, groups))
    zero = np.empty((c2, groups)) if zero_points else None
    for q in range(groups):
        w = W[:, q * group:(q + 1) * group].astype(f)
        lo, hi = np.minimum(w.min(1), f(0)), np.maximum(w.max(1), f(0))
        span = hi / f(15) - lo / f(15) if zero_points else np.maximum(hi, -lo) / f(7)
        s = round_bf16(span.astype(np.float64))
        scale[:, q] = s
        safe = np.where(s > 0, s, 1).astype(f)
        if zero_points:
            zero[:, q] = np.where(s > 0, np.clip(np.rint(-lo / safe), 0, 15), 0)
        z = zero[:, q] if zero_points else np.full(c2, 8.0)
        v = np.where(s[:, None] > 0, np.rint(w / safe[:, None]), 0) + z[:, None]
        codes[:, q * group:(q + 1) * group] = np.clip(v, 0, 15)
    return codes, scale, zero


def forward(X, W, bias=None):
    b = 0.0 if bias is None else bias[None, :]
    return X @ W.T + b, np.abs(X) @ np.abs(W).T + np.abs(b)


def backward(dY, W):
    return dY @ W, np.abs(dY) @ np.abs(W)
