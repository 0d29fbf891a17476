"""Low-rank adapters of many requests beside a shared projection.

Rows of all requests are concatenated; request b is rows offsets[b] ..
offsets[b + 1] - 1 and uses adapter slots[b] of a pool (a value outside the
pool, by convention -1: none).  For a row t of a request with adapter a

  adapter_forward    H_t = X_t A_a^T,  Y_t = base_t + scale_a H_t B_a^T
  adapter_backward   dX_t = dX_base_t + G_t A_a,  G_t = scale_a dY_t B_a,
                     dA_a = sum_t G_t^T X_t,  dB_a = sum_t scale_a dY_t^T H_t

`base` is what the shared projection gives (dyra.forward, dyra.dense_ref, any
other).  Every step runs in libdyra.so's HIP kernels on the given stream; the
calls do not synchronise, and offsets and slots are read on the device, so a
captured graph may be replayed with other requests of the same total rows.
Another stream than the current one is given as `stream`: results and
workspace that are made here are then allocated on it, and the caller orders it
after the work that makes the operands, and its own use of the results after it.

Tensors (GPU, bf16 or fp32, one type throughout):
  X [n][c1], base / Y / dY [n][c2], dX_base / dX [n][c1]: rows may be further
      apart than their width (a column range of a wider matrix), by a multiple
      of 16 bytes, elements of a row adjacent
  A [slots][r][c1], B [slots][c2][r]: contiguous; r a multiple of 8, <= 128
  rank int32 [slots], scale float32 [slots]: optional
  offsets int32 [requests + 1], from 0 to n without decreasing; slots int32
      [requests]
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import dyra as D

MAX_SLOTS = 2048   # DYRA_ADAPTER_MAX_SLOTS
_DTYPES = {torch.bfloat16: D.DT_BF16, torch.float32: D.DT_F32}


def _expect(t, name, shape, dtype, device):
    """Raises ValueError unless t is a tensor of this shape and type on device."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, name, n, c, dtype, device):
    """Pointer and row stride of an [n][c] operand whose rows are dense."""
    _expect(t, name, (n, c), dtype, device)
    p = t.data_ptr()
    if t.is_contiguous():
        ld = c
    else:
        ld, one = t.stride()
        if n == 1:
            ld = c
        if one != 1 or ld < c or ld * t.element_size() & 15:
            raise ValueError(f"{name}: rows must be dense, 16-byte aligned and not overlapping "
                             f"(strides {t.stride()})")
    if p & 15:
        raise ValueError(f"{name} must be 16-byte aligned")
    return p, ld


def _flat(t, name, shape, dtype, device):
    """Pointer of a contiguous tensor of exactly this shape, or None."""
    if t is None:
        return None
    _expect(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _span(t):
    """First and past-the-last byte a tensor reaches."""
    lo = t.data_ptr()
    return lo, lo + (sum((s - 1) * d for s, d in zip(t.shape, t.stride())) + 1) * t.element_size() if t.numel() else lo


def _overlap(a, b):
    """Whether two tensors share a byte.  Column ranges of one wide matrix are
    told apart row by row; tensors of other shapes by their spans."""
    (lo, hi), (first, last) = _span(a), _span(b)
    if not (lo < last and first < hi):
        return False
    if a.dim() != 2 or b.dim() != 2 or a.stride(1) != 1 or b.stride(1) != 1:
        return True
    # a single row may take the other's row stride
    pitch = {t.stride(0) * t.element_size() for t in (a, b) if t.shape[0] > 1}
    wide, other = (t.shape[1] * t.element_size() for t in (a, b))
    if len(pitch) != 1 or max(wide, other) > (step := pitch.pop()):
        return True
    # row i of a begins `at` bytes into row `row` + i of b's grid
    row, at = divmod(lo - first, step)
    meets = lambda k: -a.shape[0] < k < b.shape[0]  # noqa: E731
    return at < other and meets(row) or step - at < wide and meets(row + 1)


def _apart(out, name, others):
    """An output overlaps no other operand (the kernels read those while others write)."""
    for other, t in others:
        if t is not None and _overlap(out, t):
            raise ValueError(f"{name} must not overlap {other}")


def _same(a, b):
    """Whether two row operands of one shape are the same memory (a single row has no stride)."""
    return a.data_ptr() == b.data_ptr() and (a.shape[0] < 2 or a.stride() == b.stride())


def _pool(X, A, B, offsets, slots, rank, scale):
    """Checks the pool and the requests; the library's struct and sizes."""
    for name, t, dims in (("X", X, 2), ("A", A, 3), ("B", B, 3), ("offsets", offsets, 1), ("slots", slots, 1)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must be a {dims}-D tensor")
    dt = _DTYPES.get(X.dtype)
    if dt is None:
        raise ValueError(f"X must be torch.bfloat16 or torch.float32, got {X.dtype}")
    dev = X.device
    if dev.type != "cuda":
        raise ValueError("X must be a GPU tensor")
    ns, r, c1 = A.shape
    c2, B0 = B.shape[1], slots.shape[0]
    if not 1 <= ns <= MAX_SLOTS or r % 8 or not 8 <= r <= 128 or c1 % 8 or c2 % 8 or not c1 or not c2:
        raise ValueError(f"the pool must have 1 to {MAX_SLOTS} slots, a rank that is a multiple of 8 up to 128 and "
                         f"widths that are multiples of 8: A is {tuple(A.shape)}, B {tuple(B.shape)}")
    ad = D.Adapters(ns, r, c1, c2, _flat(A, "A", (ns, r, c1), X.dtype, dev), _flat(B, "B", (ns, c2, r), X.dtype, dev),
                    _flat(rank, "rank", (ns,), torch.int32, dev), _flat(scale, "scale", (ns,), torch.float32, dev))
    return (ad, dt, X.shape[0], c1, c2, r, B0, _flat(offsets, "offsets", (B0 + 1,), torch.int32, dev),
            _flat(slots, "slots", (B0,), torch.int32, dev))


@functools.lru_cache(maxsize=1024)
def adapter_workspace_size(slots: int, r: int, c1: int, c2: int, n: int, requests: int, dtype, backward=False) -> int:
    """Workspace bytes of a call with these sizes (0: it needs none); dtype: a torch or library type."""
    dtype = _DTYPES.get(dtype, dtype)
    if dtype not in (D.DT_BF16, D.DT_F32):
        raise ValueError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    need = ctypes.c_size_t()
    D._check("dyra_adapter_workspace_size",
             D.lib().dyra_adapter_workspace_size(slots, r, c1, c2, n, requests, dtype,
                                                 int(bool(backward)), ctypes.byref(need)))
    return need.value


def _workspace(workspace, ad, n, requests, dt, backward, device, stream):
    """Pointer, bytes and owner of the workspace (a temporary one if none is given)."""
    need = adapter_workspace_size(ad.slots, ad.r, ad.c1, ad.c2, n, requests, dt, backward)
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = D._new((need,), torch.uint8, device, stream)
    else:
        D._expect_bytes(workspace, "workspace", need)
        D._expect_device([("workspace", workspace)], device)
    return workspace.data_ptr(), workspace.numel(), workspace


def _on(device, stream):
    """The stream's handle; the library launches on the current device."""
    here = torch.cuda.current_device()
    if here != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{here}")
    if stream is None:
        # the handle alone: making a Stream object of it takes as long as a small kernel's launch
        return torch._C._cuda_getCurrentRawStream(here)
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors are on {device}")
    return stream.cuda_stream


def _output(t, shape, dtype, device, stream):
    """t, or a new tensor for a result, which the caller may use on the current stream."""
    return D._result(shape, dtype, device, stream) if t is None else t


def adapter_forward(X, A, B, offsets, slots, base=None, rank=None, scale=None, out=None, save_h=False, H=None,
                    workspace=None, stream=None):
    """Y = base + scale (X A^T) B^T by each request's adapter (asynchronous).

    base None: zero.  out: receives Y (may be base itself).  save_h: also
    return H = X A^T (float32 [n][r], 0 past an adapter's rank), which
    adapter_backward needs; H: a tensor that receives it.
    """
    ad, dt, n, c1, c2, r, nb, off, ids = _pool(X, A, B, offsets, slots, rank, scale)
    dev = X.device
    handle = _on(dev, stream)
    xp, ldx = _rows(X, "X", n, c1, X.dtype, dev)
    bp, ldb = (None, 0) if base is None else _rows(base, "base", n, c2, X.dtype, dev)
    Y = _output(out, (n, c2), X.dtype, dev, stream)
    yp, ldy = _rows(Y, "out", n, c2, X.dtype, dev)
    if out is not None:
        _apart(out, "out", [("X", X), ("A", A), ("B", B)])
        if base is not None and not _same(out, base):
            _apart(out, "out", [("base (other than base itself)", base)])
    given = H is not None
    if save_h:
        H = _output(H, (n, r), torch.float32, dev, stream)
    hp = _flat(H, "H", (n, r), torch.float32, dev)
    if given:
        _apart(H, "H", [("X", X), ("A", A), ("B", B), ("base", base), ("out", out)])
    wp, wn, workspace = _workspace(workspace, ad, n, nb, dt, 0, dev, stream)
    D._check("dyra_adapter_forward",
             D.lib().dyra_adapter_forward(ad, xp, ldx, bp, ldb, yp, ldy, hp, n, nb, off, ids, dt, wp, wn, handle))
    return (Y, H) if save_h or H is not None else Y


def adapter_backward(X, dY, H, A, B, offsets, slots, dX_base=None, rank=None, scale=None, dX=None, dA=None, dB=None,
                     need_dx=True, need_weights=True, workspace=None, stream=None):
    """(dX, dA, dB) from dY, the gradient of adapter_forward's Y (asynchronous).

    H: what the forward pass kept (may be None if need_weights is False).
    dX_base: the shared projection's input gradient (None: zero); dX may be
    dX_base itself.  dA, dB are float32, every element written.  need_dx /
    need_weights False: that result is None and its work is not done.
    """
    ad, dt, n, c1, c2, r, nb, off, ids = _pool(X, A, B, offsets, slots, rank, scale)
    dev = X.device
    if not need_dx and not need_weights:
        raise ValueError("nothing is asked for: need_dx and need_weights are both False")
    handle = _on(dev, stream)
    xp, ldx = _rows(X, "X", n, c1, X.dtype, dev)
    gp, ldg = _rows(dY, "dY", n, c2, X.dtype, dev)
    if need_weights and H is None:
        raise ValueError("H, kept by the forward pass, is needed for the weights' gradients")
    hp = _flat(H, "H", (n, r), torch.float32, dev)
    inputs = [("X", X), ("dY", dY), ("H", H), ("A", A), ("B", B)]
    bp, ldb, op, ldo = None, 0, None, 0
    if need_dx:
        if dX_base is not None:
            bp, ldb = _rows(dX_base, "dX_base", n, c1, X.dtype, dev)
        given = dX is not None
        dX = _output(dX, (n, c1), X.dtype, dev, stream)
        op, ldo = _rows(dX, "dX", n, c1, X.dtype, dev)
        if given:
            _apart(dX, "dX", inputs)
            if dX_base is not None and not _same(dX, dX_base):
                _apart(dX, "dX", [("dX_base (other than dX_base itself)", dX_base)])
    else:
        dX = None
    ap = wp2 = None
    if need_weights:
        ns = A.shape[0]
        given = [(t, name) for t, name in ((dA, "dA"), (dB, "dB")) if t is not None]
        dA = _output(dA, (ns, r, c1), torch.float32, dev, stream)
        dB = _output(dB, (ns, c2, r), torch.float32, dev, stream)
        ap = _flat(dA, "dA", (ns, r, c1), torch.float32, dev)
        wp2 = _flat(dB, "dB", (ns, c2, r), torch.float32, dev)
        for t, name in given:
            _apart(t, name, inputs + [("dX_base", dX_base), ("dX", dX)])
        if len(given) == 2:
            _apart(dA, "dA", [("dB", dB)])
    else:
        dA = dB = None
    wp, wn, workspace = _workspace(workspace, ad, n, nb, dt, 1, dev, stream)
    D._check("dyra_adapter_backward",
             D.lib().dyra_adapter_backward(ad, xp, ldx, gp, ldg, hp, bp, ldb, op, ldo, ap, wp2, n, nb, off, ids, dt,
                                           wp, wn, handle))
    return dX, dA, dB
