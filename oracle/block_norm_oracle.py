"""Float64 CPU oracle of the norms around a block, straight from

  u = post(y),  x' = alpha x + g * u,  z = pre(x'),
  norm(v) = w * (v - mean) / sqrt(mean((v - mean)^2) + eps) + b  (mean 0 for "rms")

and the gradients of these, one row at a time where rows matter.
"""
from __future__ import annotations

import numpy as np


def hat(v, kind, eps):
    m = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    inv = 1.0 / np.sqrt(((v - m) ** 2).mean(1, keepdims=True) + eps)
    return (v - m) * inv, inv


def affine(v, w, b):
    v = v if w is None else v * w
    return v if b is None else v + b


def gate_rows(gate, offsets, n):
    if gate is None:
        return np.ones((n, 1))
    if gate.ndim == 1:
        return gate[None, :]
    out = np.zeros((n, gate.shape[1]))
    for b in range(gate.shape[0]):
        out[offsets[b]:offsets[b + 1]] = gate[b]
    return out


def branch(y, post, w, b, eps):
    return y if post == "none" else affine(hat(y, post, eps)[0], w, b)


def forward(x, y, pre, post, par, offsets=None, alpha=1.0, eps=1e-6):
    g = gate_rows(par["gate"], offsets, x.shape[0])
    xn = alpha * x + g * branch(y, post, par["post_weight"], par["post_bias"], eps)
    return xn, affine(hat(xn, pre, eps)[0], par["pre_weight"], par["pre_bias"])


def hat_grad(d, h, inv, kind):
    """The gradient of v from d, the gradient of hat(v): the derivative of
    (v - mean) inv along v, applied row by row."""
    c = h.shape[1]
    out = inv * (d - h * (d * h).sum(1, keepdims=True) / c)
    return out - inv * d.sum(1, keepdims=True) / c if kind == "layer" else out


def backward(xn, y, dz, dxn, pre, post, par, offsets=None, alpha=1.0, eps=1e-6):
    n = xn.shape[0]
    one = lambda w: 1.0 if w is None else w  # noqa: E731
    h, inv = hat(xn, pre, eps)
    d = hat_grad(dz * one(par["pre_weight"]), h, inv, pre) + (0.0 if dxn is None else dxn)
    g = gate_rows(par["gate"], offsets, n)
    u = branch(y, post, par["post_weight"], par["post_bias"], eps)
    out = {"dx": alpha * d, "d_pre_weight": (dz * h).sum(0), "d_pre_bias": dz.sum(0)}
    du = g * d
    gate = par["gate"]
    if gate is not None and gate.ndim == 1:
        out["d_gate"] = (d * u).sum(0)
    elif gate is not None:
        out["d_gate"] = np.stack([(d * u)[offsets[b]:offsets[b + 1]].sum(0) for b in range(gate.shape[0])])
    if post != "none":
        hy, iy = hat(y, post, eps)
        out["d_post_weight"], out["d_post_bias"] = (du * hy).sum(0), du.sum(0)
        du = hat_grad(du * one(par["post_weight"]), hy, iy, post)
    out["dy"] = du
    return out
