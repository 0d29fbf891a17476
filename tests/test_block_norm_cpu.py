"""Host checks of the block-norm entry points, and the oracle's gradients
against differences of its forward pass."""
import ctypes

import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import block_norm_oracle as O

BF16, F32 = synth.DT_BF16, synth.DT_F32
P = 1 << 12   # fake, never dereferenced, aligned address: every call must be rejected on the host


def _norm(c=64, pre=1, post=0, gate_kind=0, eps=1e-6, scale=1.0, pw=None, pb=None, qw=None, qb=None, gate=None):
    return D.BlockNorm(c, pre, post, gate_kind, eps, scale, pw, pb, qw, qb, gate)


def _forward(x=P, y=P, x_new=P, z=P, n=10, B=0, off=None, dtype=BF16, **kw):
    return D.lib().dyra_block_norm_forward(_norm(**kw), x, y, x_new, z, n, B, off, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(z=None), -1), (dict(x_new=None), -1), (dict(x=P + 8), -1),
    (dict(dtype=4), -1), (dict(pre=0), -1), (dict(pre=3), -1), (dict(post=3), -1), (dict(gate_kind=3, gate=P), -1),
    (dict(gate_kind=1), -1), (dict(gate=P), -1), (dict(qw=P), -1), (dict(qb=P), -1), (dict(pw=P + 2), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(gate_kind=2, gate=P, B=2), -1),                       # no offsets
    (dict(gate_kind=2, gate=P, B=0, off=P), -2),                # rows of no request
    (dict(c=60), -2), (dict(c=0), -2), (dict(c=16392), -2), (dict(n=-1), -2), (dict(n=1 << 31), -2), (dict(B=-1), -2),
])
def test_forward_rejects_before_any_hip_call(kw, code):
    assert _forward(**kw) == code


def test_forward_of_no_rows_is_done_on_the_host():
    assert _forward(n=0, x=None, y=None, x_new=None, z=None) == 0


def _backward(x_new=P, y=P, dz=P, dx_new=None, dx=P, dy=P, n=10, B=0, off=None, dtype=BF16, ws=P, ws_bytes=1 << 40,
              grads=(P, None, None, None, None), **kw):
    return D.lib().dyra_block_norm_backward(_norm(**kw), x_new, y, dz, dx_new, dx, dy, D.BlockNormGrads(*grads), n, B,
                                            off, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x_new=None), -1), (dict(dz=None), -1), (dict(dx=None), -1), (dict(dy=None), -1), (dict(ws=None), -1),
    (dict(dx_new=P + 4), -1), (dict(grads=(P + 4, None, None, None, None)), -1),
    (dict(grads=(None, P, None, None, None)), -1),              # no such bias
    (dict(grads=(None, None, P, None, None)), -1),              # no post norm
    (dict(grads=(None, None, None, None, P)), -1),              # no gate
    (dict(gate_kind=2, gate=P, B=2, off=P), -1),                # a gate per request, its gradient not given
    (dict(c=4), -2), (dict(ws_bytes=16), -3),
])
def test_backward_rejects_before_any_hip_call(kw, code):
    assert _backward(**kw) == code


@pytest.mark.parametrize("kw", [dict(), dict(gate_kind=1, gate=P), dict(gate_kind=2, off=P),
                                dict(gate_kind=2, gate=P, off=P), dict(gate_kind=2)])
def test_backward_of_no_rows_launches_no_row_kernel(kw):
    """Without rows only the join of wanted gradients is launched (a gate per
    request may then have no row to load); with none wanted, nothing is, and
    the call succeeds where there is no GPU."""
    assert _backward(n=0, x_new=None, y=None, dz=None, dx=None, dy=None, grads=(None,) * 5, **kw) == 0


def test_backward_of_too_many_requests_is_rejected_before_any_hip_call():
    """2^32 threads or more in the join of a gate's gradients."""
    for c, B in ((16384, 32768), (4096, 131072), (40, (1 << 23) + 1)):
        kw = dict(c=c, gate_kind=2, gate=P, off=P, grads=(P, None, None, None, P), ws_bytes=1 << 62)
        assert _backward(n=100, B=B, **kw) == -2


def test_workspace_size():
    need = [ctypes.c_size_t() for _ in range(3)]
    L = D.lib()
    assert L.dyra_block_norm_workspace_size(_norm(), 1000, 0, BF16, need[0]) == 0
    assert L.dyra_block_norm_workspace_size(_norm(post=1), 1000, 0, BF16, need[1]) == 0
    assert L.dyra_block_norm_workspace_size(_norm(post=1, gate_kind=2, gate=P), 1000, 3, BF16, need[2]) == 0
    assert 0 < need[0].value < need[1].value < need[2].value
    assert L.dyra_block_norm_workspace_size(_norm(c=12), 1000, 0, BF16, need[0]) == -2
    assert L.dyra_block_norm_workspace_size(_norm(), 1000, 0, BF16, None) == -1


@pytest.mark.parametrize("change,msg", [
    (dict(x="x"), "x must be a 2-D tensor"), (dict(), "must be a GPU tensor"),
    (dict(dtype="float64"), "torch.bfloat16 or torch.float32"),
])
def test_binding_rejects_before_the_library(change, msg):
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    x = torch.zeros((4, 64), dtype=getattr(torch, change.get("dtype", "bfloat16")))
    with pytest.raises(ValueError, match=msg):
        BN.block_norm_forward(change.get("x", x), x)


@pytest.mark.parametrize("pre,post,gate", [("rms", "layer", "request"), ("layer", "rms", "channel"),
                                           ("layer", "none", "none")])
def test_oracle_gradients_match_differences(pre, post, gate):
    """Every gradient of the oracle along random directions, against fourth
    order differences: agreement to 1e-8 of sum |gradient direction|, h = 1e-3
    (truncation h^4 times the fifth derivative, rounding 2^-52 / h of the loss)."""
    g = np.random.default_rng(1)
    n, c, off = 7, 40, np.array([0, 3, 3, 7])
    x, y, dz, dxn = (g.standard_normal((n, c)) for _ in range(4))
    par = dict(pre_weight=1 + 0.2 * g.standard_normal(c), pre_bias=g.standard_normal(c), post_weight=None,
               post_bias=None, gate=None)
    if post != "none":
        par.update(post_weight=1 + 0.2 * g.standard_normal(c), post_bias=g.standard_normal(c))
    if gate != "none":
        par["gate"] = g.standard_normal(c) if gate == "channel" else g.standard_normal((3, c))
    kw = dict(offsets=off, alpha=0.7, eps=1e-3)

    def loss(v):
        a, z = O.forward(v["x"], v["y"], pre, post, {k: v[k] for k in par}, **kw)
        return (a * dxn).sum() + (z * dz).sum()

    at = dict(par, x=x, y=y)
    got = O.backward(O.forward(x, y, pre, post, par, **kw)[0], y, dz, dxn, pre, post, par, **kw)
    for k, v in at.items():
        if v is None:
            continue
        step, h = g.standard_normal(v.shape), 1e-3
        f = lambda t: loss(dict(at, **{k: v + t * step}))  # noqa: E731
        slope = (8 * (f(h) - f(-h)) - (f(2 * h) - f(-2 * h))) / (12 * h)
        grad = got["d" + k if k in ("x", "y") else "d_" + k]
        assert abs(slope - (grad * step).sum()) <= 1e-8 * max(1.0, np.abs(grad * step).sum()), k
