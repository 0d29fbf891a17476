"""Projections with 4-bit weights and group scales.

A weight W [c2][c1] (output-major, as a linear layer stores it) is held as codes
0 .. 15 with a bf16 scale and a zero point for each group of 32, 64 or 128
columns of a row:  w = scale (code - zero).

  q4_quantise   codes, scales and zero points of a matrix
  q4_pack       a Q4Weight from them: laid out for the products, once
  q4_forward    Y = X W^T + bias     single tokens and long prompts alike
  q4_backward   dX = dY W            the frozen weight's input gradient
  q4_dense      the weight as a dense matrix

Such a projection stands where the layer or a dense product stands: what it
gives is the `base` of adapters.adapter_forward, and its gradient the `dX_base`
of adapters.adapter_backward.

Tensors (GPU; X, bias, Y and gradients bf16 or fp32, one type throughout):
  codes uint8 [c2][c1 / 2]: two to a byte, the even column in the low half
  scale bfloat16 [c2][groups], zero uint8 [c2][groups] (None: 8 everywhere),
      groups = ceil(c1 / group); all contiguous
  X, dX [n][c1], Y, dY [n][c2]: rows may be further apart than their width, by a
      multiple of 16 bytes, elements of a row adjacent; widths multiples of 8

Every step runs in libdyra.so's HIP kernels on the given stream, without
synchronising; results and workspace that are made here are allocated on that
stream, and the caller orders it after the work that makes the operands, and its
own use of the results after it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import dyra as D
from .adapters import _DTYPES, _apart, _flat, _on, _output, _rows

GROUPS = (32, 64, 128)


def _widths(c1, c2, group):
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    if c1 % 8 or c2 % 8 or not c1 or not c2:
        raise ValueError(f"widths must be multiples of 8: W is [{c2}][{c1}]")


@functools.lru_cache(maxsize=1024)
def q4_packed_size(c1: int, c2: int, group: int) -> int:
    """Bytes of a packed weight."""
    need = ctypes.c_size_t()
    D._check("dyra_q4_packed_size", D.lib().dyra_q4_packed_size(c1, c2, group, ctypes.byref(need)))
    return need.value


@functools.lru_cache(maxsize=1024)
def q4_workspace_size(c1: int, c2: int, n: int, dtype, backward=False) -> int:
    """Workspace bytes of a call of n rows (0: it needs none); dtype: a torch or library type."""
    dtype = _DTYPES.get(dtype, dtype)
    if dtype not in (D.DT_BF16, D.DT_F32):
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    need = ctypes.c_size_t()
    D._check("dyra_q4_workspace_size",
             D.lib().dyra_q4_workspace_size(c1, c2, n, dtype, int(bool(backward)), ctypes.byref(need)))
    return need.value


class Q4Weight:
    """A packed weight: shape (c2, c1), group, device, and the uint8 tensor
    `packed` that holds it."""

    def __init__(self, c1: int, c2: int, group: int, packed):
        _widths(c1, c2, group)
        if not isinstance(packed, torch.Tensor) or packed.device.type != "cuda":
            raise ValueError("packed must be a GPU tensor")
        D._expect_bytes(packed, "packed", q4_packed_size(c1, c2, group))
        D._expect_device([("packed", packed)], packed.device)
        if packed.data_ptr() & 15:
            raise ValueError("packed must be 16-byte aligned")
        self.c1, self.c2, self.group, self.packed = c1, c2, group, packed
        self.shape, self.device = (c2, c1), packed.device
        self._handle = D.Q4(c1, c2, group, packed.data_ptr())


def q4_quantise(W, group=128, zero_points=False, stream=None):
    """(codes, scale, zero) of a dense matrix [c2][c1], bf16 or fp32, finite
    (asynchronous).  zero is None without zero_points: code 8 stands for 0 and
    a group's largest magnitude for 7 scales; with them a group's lowest and highest
    value (0 among them) are 15 scales apart."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D tensor")
    dt = _DTYPES.get(W.dtype)
    if dt is None:
        raise ValueError(f"W must be torch.bfloat16 or torch.float32, got {W.dtype}")
    dev = W.device
    if dev.type != "cuda":
        raise ValueError("W must be a GPU tensor")
    c2, c1 = W.shape
    _widths(c1, c2, group)
    handle = _on(dev, stream)
    wp = _flat(W, "W", (c2, c1), W.dtype, dev)
    if wp & 15:
        raise ValueError("W must be 16-byte aligned")
    groups = -(-c1 // group)
    codes = _output(None, (c2, c1 // 2), torch.uint8, dev, stream)
    scale = _output(None, (c2, groups), torch.bfloat16, dev, stream)
    zero = _output(None, (c2, groups), torch.uint8, dev, stream) if zero_points else None
    D._check("dyra_q4_quantise",
             D.lib().dyra_q4_quantise(wp, c1, c2, group, dt, codes.data_ptr(), scale.data_ptr(),
                                      None if zero is None else zero.data_ptr(), handle))
    return codes, scale, zero


def q4_pack(codes, scale, zero=None, group=128, stream=None) -> Q4Weight:
    """The packed weight of codes [c2][c1 / 2], scales and zero points
    (asynchronous); the operands are not needed afterwards."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a 2-D tensor")
    dev = codes.device
    if dev.type != "cuda":
        raise ValueError("codes must be a GPU tensor")
    c2, c1 = codes.shape[0], 2 * codes.shape[1]
    _widths(c1, c2, group)
    groups = -(-c1 // group)
    if scale is None:
        raise ValueError("scale must be a tensor")
    cp = _flat(codes, "codes", (c2, c1 // 2), torch.uint8, dev)
    sp = _flat(scale, "scale", (c2, groups), torch.bfloat16, dev)
    zp = _flat(zero, "zero", (c2, groups), torch.uint8, dev)
    if cp & 3:
        raise ValueError("codes must be 4-byte aligned")
    handle = _on(dev, stream)
    packed = _output(None, (q4_packed_size(c1, c2, group),), torch.uint8, dev, stream)
    D._check("dyra_q4_pack", D.lib().dyra_q4_pack(c1, c2, group, cp, sp, zp, packed.data_ptr(), handle))
    return Q4Weight(c1, c2, group, packed)


def _call(t, name, weight, back):
    """Checks the rows of a call against the weight; type, device, rows, the
    stride of its rows and where they lie."""
    if not isinstance(weight, Q4Weight):
        raise ValueError("weight must be a Q4Weight (q4_pack)")
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    dev, width = weight.device, weight.c2 if back else weight.c1
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the weight on {dev}")
    n, c = t.shape
    if c != width:
        raise ValueError(f"{name} must have {width} columns, got {tuple(t.shape)}")
    p = t.data_ptr()
    if p & 15 or not t.is_contiguous():
        return dt, dev, n, *_rows(t, name, n, width, t.dtype, dev)
    return dt, dev, n, p, width


def _result(t, out, name, n, width, stream):
    """Where a result goes: out, or a new tensor beside t."""
    if out is None and stream is None:
        out = t.new_empty((n, width))
        return out, out.data_ptr(), width
    out = _output(out, (n, width), t.dtype, t.device, stream)
    return out, *_rows(out, name, n, width, t.dtype, t.device)


def _workspace(workspace, need, device, stream):
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = D._new((need,), torch.uint8, device, stream)
    else:
        D._expect_bytes(workspace, "workspace", need)
        D._expect_device([("workspace", workspace)], device)
    return workspace.data_ptr(), workspace.numel(), workspace


def q4_forward(X, weight, bias=None, out=None, workspace=None, stream=None):
    """Y = X W^T + bias (asynchronous).  out: receives Y."""
    dt, dev, n, xp, ldx = _call(X, "X", weight, False)
    c1, c2 = weight.c1, weight.c2
    handle = _on(dev, stream)
    bp = None
    if bias is not None:
        bp = _flat(bias, "bias", (c2,), X.dtype, dev)
        if bp & 15:
            raise ValueError("bias must be 16-byte aligned")
    Y, yp, ldy = _result(X, out, "out", n, c2, stream)
    if out is not None:
        _apart(out, "out", [("X", X), ("bias", bias), ("weight", weight.packed)])
    wp, wn, workspace = _workspace(workspace, q4_workspace_size(c1, c2, n, dt), dev, stream)
    D._check("dyra_q4_forward",
             D.lib().dyra_q4_forward(weight._handle, xp, ldx, bp, yp, ldy, n, dt, wp, wn, handle))
    return Y


def q4_backward(dY, weight, dX=None, workspace=None, stream=None):
    """dX = dY W, the gradient of q4_forward's X (asynchronous).  dX: a tensor
    that receives it."""
    dt, dev, n, gp, ldg = _call(dY, "dY", weight, True)
    c1, c2 = weight.c1, weight.c2
    handle = _on(dev, stream)
    given = dX
    dX, op, ldo = _result(dY, dX, "dX", n, c1, stream)
    if given is not None:
        _apart(dX, "dX", [("dY", dY), ("weight", weight.packed)])
    wp, wn, workspace = _workspace(workspace, q4_workspace_size(c1, c2, n, dt, True), dev, stream)
    D._check("dyra_q4_backward",
             D.lib().dyra_q4_backward(weight._handle, gp, ldg, op, ldo, n, dt, wp, wn, handle))
    return dX


def q4_dense(weight, dtype=torch.bfloat16, stream=None):
    """The weight as a dense [c2][c1] matrix: exact in fp32, rounded once in
    bf16 (asynchronous)."""
    if not isinstance(weight, Q4Weight):
        raise ValueError("weight must be a Q4Weight (q4_pack)")
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    handle = _on(weight.device, stream)
    out = _output(None, (weight.c2, weight.c1), dtype, weight.device, stream)
    D._check("dyra_q4_dense", D.lib().dyra_q4_dense(weight._handle, out.data_ptr(), _DTYPES[dtype], handle))
    return out
