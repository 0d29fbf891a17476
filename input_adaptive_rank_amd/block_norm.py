"""The norms before and after a block, fused with its gate and residual scale.

Per row, y the block's output and x the residual stream:

  block_norm_forward    u = post(y),  x' = residual_scale x + gate * u,
                        z = pre(x')          (what the next block reads)
  block_norm_backward   d = dx' + pre^T(dz), dx = residual_scale d,
                        dy = post^T(gate * d), and the gradients of weights,
                        biases and gate

pre is "rms" or "layer", post also "none".  The gate is absent, one vector
[c], or one row per request [requests][c] with offsets int32 [requests + 1]
(request b is rows offsets[b] .. offsets[b + 1] - 1, from 0 to n without
decreasing).  Weights and biases are [c] or None (1 and 0).

All tensors are on one GPU, bf16 or fp32 (one type throughout), contiguous;
c is a multiple of 8 up to 16384.  Parameter gradients are float32.  Every step
runs in libdyra.so's HIP kernels on the given stream, without synchronising;
results and workspace that are made here are allocated on that stream, and the
caller orders it after the work that makes the operands, and its own use of the
results after it.
"""
from __future__ import annotations

import ctypes

import torch

from . import dyra as D
from .adapters import _DTYPES, _apart, _flat, _on, _output

MAX_C = 16384   # DYRA_BLOCK_NORM_MAX_C
_KINDS = {"none": 0, "rms": 1, "layer": 2}


def _params(x, name, pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, offsets, residual_scale, eps):
    """Checks the parameters against x; the library's struct, n, requests, offsets."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    dev, dtype = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if pre not in ("rms", "layer") or post not in _KINDS:
        raise ValueError(f'pre must be "rms" or "layer", post "none", "rms" or "layer": got {pre!r}, {post!r}')
    n, c = x.shape
    if not c or c % 8 or c > MAX_C:
        raise ValueError(f"the width must be a multiple of 8 up to {MAX_C}, got {c}")
    if post == "none" and (post_weight is not None or post_bias is not None):
        raise ValueError('post is "none": it takes no weight or bias')
    kind, nb, gp, op = 0, 0, None, None
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() not in (1, 2):
            raise ValueError("gate must be a 1-D or 2-D tensor")
        kind = gate.dim()
        if kind == 2:
            nb = gate.shape[0]
            if offsets is None:
                raise ValueError("a gate per request needs the requests' offsets")
            if n and not nb:
                raise ValueError("rows of no request have no gate")
            op = _flat(offsets, "offsets", (nb + 1,), torch.int32, dev)
        gp = _flat(gate, "gate", (c,) if kind == 1 else (nb, c), dtype, dev)
    p = D.BlockNorm(c, _KINDS[pre], _KINDS[post], kind, eps, residual_scale,
                    _flat(pre_weight, "pre_weight", (c,), dtype, dev), _flat(pre_bias, "pre_bias", (c,), dtype, dev),
                    _flat(post_weight, "post_weight", (c,), dtype, dev),
                    _flat(post_bias, "post_bias", (c,), dtype, dev), gp)
    return p, dt, n, c, nb, op


def _no_overlap(out, name, inputs, others):
    """An output may be one of the row inputs itself; it overlaps nothing else."""
    lo = out.data_ptr()
    for other, t in inputs:
        if t is not None and t.data_ptr() != lo:
            _apart(out, name, [(other, t)])
    _apart(out, name, others)


def block_norm_forward(x, y, pre="rms", post="none", pre_weight=None, pre_bias=None, post_weight=None, post_bias=None,
                       gate=None, offsets=None, residual_scale=1.0, eps=1e-6, x_new=None, z=None, stream=None):
    """(x', z), both [n][c] (asynchronous).  x_new, z: tensors that receive
    them; each may be x or y itself, not both the same."""
    p, dt, n, c, nb, off = _params(x, "x", pre, post, pre_weight, pre_bias, post_weight, post_bias, gate, offsets,
                                   residual_scale, eps)
    dev, dtype = x.device, x.dtype
    handle = _on(dev, stream)
    shape = (n, c)
    xp, yp = _flat(x, "x", shape, dtype, dev), _flat(y, "y", shape, dtype, dev)
    if yp is None:
        raise ValueError("y must be a tensor")
    if x_new is not None or z is not None:
        fixed = [("pre_weight", pre_weight), ("pre_bias", pre_bias), ("post_weight", post_weight),
                 ("post_bias", post_bias), ("gate", gate)]
        for t, name in ((x_new, "x_new"), (z, "z")):
            if t is not None:
                _flat(t, name, shape, dtype, dev)
                _no_overlap(t, name, [("x", x), ("y", y)], fixed)
        if x_new is not None and z is not None:
            _apart(x_new, "x_new", [("z", z)])
    x_new, z = _output(x_new, shape, dtype, dev, stream), _output(z, shape, dtype, dev, stream)
    D._check("dyra_block_norm_forward",
             D.lib().dyra_block_norm_forward(p, xp, yp, x_new.data_ptr(), z.data_ptr(), n, nb, off, dt, handle))
    return x_new, z


def block_norm_backward(x_new, y, dz, dx_new=None, pre="rms", post="none", pre_weight=None, pre_bias=None,
                        post_weight=None, post_bias=None, gate=None, offsets=None, residual_scale=1.0, eps=1e-6,
                        dx=None, dy=None, workspace=None, stream=None):
    """The gradients of block_norm_forward (asynchronous): a dict of dx, dy
    and d_pre_weight, d_pre_bias, d_post_weight, d_post_bias, d_gate (float32;
    None for a parameter that is None).

    x_new: the x' the forward pass stored; dz, dx_new: the gradients that
    reach z and x' (dx_new None: zero).  dx, dy: tensors that receive those;
    each may be one of the row inputs itself, not both the same.
    """
    p, dt, n, c, nb, off = _params(x_new, "x_new", pre, post, pre_weight, pre_bias, post_weight, post_bias, gate,
                                   offsets, residual_scale, eps)
    dev, dtype = x_new.device, x_new.dtype
    handle = _on(dev, stream)
    shape = (n, c)
    rows = [("x_new", x_new), ("y", y), ("dz", dz), ("dx_new", dx_new)]
    ptr = [_flat(t, name, shape, dtype, dev) for name, t in rows]
    if y is None or dz is None:
        raise ValueError("y and dz must be tensors")
    params = [("pre_weight", pre_weight), ("pre_bias", pre_bias), ("post_weight", post_weight),
              ("post_bias", post_bias), ("gate", gate)]
    for t, name in ((dx, "dx"), (dy, "dy")):
        if t is not None:
            _flat(t, name, shape, dtype, dev)
            _no_overlap(t, name, rows, params)
    if dx is not None and dy is not None:
        _apart(dx, "dx", [("dy", dy)])
    dx, dy = _output(dx, shape, dtype, dev, stream), _output(dy, shape, dtype, dev, stream)
    # one allocation: a row for each vector, the gate's rows last
    vectors = [name for name, t in params if t is not None and t.dim() == 1]
    buf = _output(None, (len(vectors) + (nb if gate is not None and gate.dim() == 2 else 0), c), torch.float32, dev,
                  stream)
    rows_of = dict(zip(vectors, buf[:len(vectors)].unbind(0))) if vectors else {}
    if gate is not None and gate.dim() == 2:
        rows_of["gate"] = buf[len(vectors):]
    grads = {"d_" + name: rows_of.get(name) for name, _ in params}
    g = D.BlockNormGrads(*[None if t is None else t.data_ptr() for t in grads.values()])
    need = ctypes.c_size_t()
    L = D.lib()
    D._check("dyra_block_norm_workspace_size", L.dyra_block_norm_workspace_size(p, n, nb, dt, need))
    if workspace is None:
        workspace = D._new((need.value,), torch.uint8, dev, stream)
    else:
        D._expect_bytes(workspace, "workspace", need.value)
        D._expect_device([("workspace", workspace)], dev)
    D._check("dyra_block_norm_backward",
             L.dyra_block_norm_backward(p, *ptr, dx.data_ptr(), dy.data_ptr(), g, n, nb, off, dt,
                                        workspace.data_ptr(), workspace.numel(), handle))
    return {"dx": dx, "dy": dy, **grads}
