"""Softmax cross entropy over a vocabulary, without its logits in memory.

For hidden rows H [n][c], a head W [v][c] and targets [n]

  vocab_loss_forward    a = logit_scale H W^T,  lse_t = log sum_v exp a_tv,
                        loss_t = lse_t - a_t,target
  vocab_loss_backward   d_tv = logit_scale dloss_t (exp(a_tv - lse_t) - [v = target_t]),
                        dH = d W,  dW = d^T H

A row whose target is outside 0 .. v - 1 (by convention -1) is ignored: its
loss and its row of dH are 0 and it adds nothing to dW, whatever its row of H,
lse and dloss hold; its lse is computed.  A mean over the rows that count is
the caller's: dloss = 1 / their number gives its gradient.

The backward pass multiplies the logits again, one piece of the vocabulary at
a time, and rounds d to W's precision for the two products, relative to the
largest weight logit_scale |dloss_t|: rows of equal weights, as a mean's are, lose
nothing by the weight.  Results do not
depend on the order in which workgroups run: the same call gives the same bits.

Tensors (GPU, bf16 or fp32, one type throughout):
  H, dH [n][c]: rows may be further apart than their width, by a multiple of
      16 bytes, elements of a row adjacent; c a multiple of 8
  W, dW [v][c]: contiguous; v is any
  targets int32 [n]; loss, lse, dloss float32 [n]

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


@functools.lru_cache(maxsize=1024)
def vocab_loss_workspace_size(n: int, c: int, v: int, dtype, backward=False, need_dh=True, need_dw=True) -> int:
    """Workspace bytes of a call with these sizes; dtype: a torch or library type."""
    dtype = _DTYPES.get(dtype, dtype)
    if dtype not in (D.DT_BF16, D.DT_F32):
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    need = ctypes.c_size_t()
    D._check("dyra_vocab_loss_workspace_size",
             D.lib().dyra_vocab_loss_workspace_size(n, c, v, dtype, int(bool(backward)), int(bool(need_dh)),
                                                    int(bool(need_dw)), ctypes.byref(need)))
    return need.value


def _operands(H, W, targets, logit_scale):
    """Checks what both passes read; sizes and pointers."""
    for name, t, dims in (("H", H, 2), ("W", W, 2), ("targets", targets, 1)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D tensor")
    dt = _DTYPES.get(H.dtype)
    if dt is None:
        raise ValueError(f"H must be torch.bfloat16 or torch.float32, got {H.dtype}")
    dev = H.device
    if dev.type != "cuda":
        raise ValueError("H must be a GPU tensor")
    n, c = H.shape
    v = W.shape[0]
    if not c or c % 8 or not v:
        raise ValueError(f"the width must be a multiple of 8 and the vocabulary not empty: H is {tuple(H.shape)}, "
                         f"W {tuple(W.shape)}")
    if not 0.0 < logit_scale <= 2.0 ** 126:
        raise ValueError(f"logit_scale must be positive and finite, at most 2^126, got {logit_scale}")
    hp, ldh = _rows(H, "H", n, c, H.dtype, dev)
    wp = _flat(W, "W", (v, c), H.dtype, dev)
    if wp & 15:
        raise ValueError("W must be 16-byte aligned")
    return dt, dev, n, c, v, hp, ldh, wp, _flat(targets, "targets", (n,), torch.int32, dev)


def _workspace(workspace, need, device, stream):
    if workspace is None:
        workspace = D._new((need,), torch.uint8, device, stream)
    else:
        D._expect_bytes(workspace, "workspace", need)
        D._expect_device([("workspace", workspace)], device)
    return workspace


def vocab_loss_forward(H, W, targets, logit_scale=1.0, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse), float32 [n] each (asynchronous).  loss, lse: tensors that
    receive them.  The backward pass needs lse."""
    dt, dev, n, c, v, hp, ldh, wp, tp = _operands(H, W, targets, logit_scale)
    handle = _on(dev, stream)
    inputs = [("H", H), ("W", W), ("targets", targets)]
    given = [(t, name) for t, name in ((loss, "loss"), (lse, "lse")) if t is not None]
    loss, lse = _output(loss, (n,), torch.float32, dev, stream), _output(lse, (n,), torch.float32, dev, stream)
    lp, ep = _flat(loss, "loss", (n,), torch.float32, dev), _flat(lse, "lse", (n,), torch.float32, dev)
    for t, name in given:
        _apart(t, name, inputs)
    if len(given) == 2:
        _apart(loss, "loss", [("lse", lse)])
    ws = _workspace(workspace, vocab_loss_workspace_size(n, c, v, dt), dev, stream)
    D._check("dyra_vocab_loss_forward",
             D.lib().dyra_vocab_loss_forward(hp, ldh, wp, tp, logit_scale, lp, ep, n, c, v, dt, ws.data_ptr(),
                                             ws.numel(), handle))
    return loss, lse


def vocab_loss_backward(H, W, targets, lse, dloss, logit_scale=1.0, dH=None, dW=None, need_dh=True, need_dw=True,
                        workspace=None, stream=None):
    """(dH, dW) from dloss, the gradient of vocab_loss_forward's loss, and
    the lse it returned (asynchronous).  dH, dW: tensors that receive them,
    every element written.  need_dh / need_dw False (a frozen head): that
    result is None and its work is not done."""
    dt, dev, n, c, v, hp, ldh, wp, tp = _operands(H, W, targets, logit_scale)
    if not need_dh and not need_dw:
        raise ValueError("nothing is asked for: need_dh and need_dw are both False")
    handle = _on(dev, stream)
    ep, gp = _flat(lse, "lse", (n,), torch.float32, dev), _flat(dloss, "dloss", (n,), torch.float32, dev)
    if lse is None or dloss is None:
        raise ValueError("lse and dloss must be tensors")
    inputs = [("H", H), ("W", W), ("targets", targets), ("lse", lse), ("dloss", dloss)]
    op, ldo, wo = None, 0, None
    if need_dh:
        given = dH is not None
        dH = _output(dH, (n, c), H.dtype, dev, stream)
        op, ldo = _rows(dH, "dH", n, c, H.dtype, dev)
        if given:
            _apart(dH, "dH", inputs)
    else:
        dH = None
    if need_dw:
        given = dW is not None
        dW = _output(dW, (v, c), H.dtype, dev, stream)
        wo = _flat(dW, "dW", (v, c), H.dtype, dev)
        if given:
            if wo & 15:
                raise ValueError("dW must be 16-byte aligned")
            _apart(dW, "dW", inputs + [("dH", dH)])
    else:
        dW = None
    ws = _workspace(workspace, vocab_loss_workspace_size(n, c, v, dt, True, need_dh, need_dw), dev, stream)
    D._check("dyra_vocab_loss_backward",
             D.lib().dyra_vocab_loss_backward(hp, ldh, wp, tp, ep, gp, logit_scale, op, ldo, wo, n, c, v, dt,
                                              ws.data_ptr(), ws.numel(), handle))
    return dH, dW
