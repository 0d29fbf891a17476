"""Host checks of the vocabulary loss: the library rejects bad arguments with
the documented codes, the binding with ValueError, before any HIP call; the
oracle against differences and a worked example."""
import ctypes

import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import vocab_loss_oracle as O

BF16, F32 = synth.DT_BF16, synth.DT_F32
P = 1 << 12   # a fake, never dereferenced, aligned address


def _size(n=100, C=64, V=1000, dtype=BF16, backward=0, dh=1, dw=1):
    need = ctypes.c_size_t()
    return D.lib().dyra_vocab_loss_workspace_size(n, C, V, dtype, backward, dh, dw, ctypes.byref(need)), need.value


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(dtype=F32), 0), (dict(backward=1), 0), (dict(backward=1, dw=0), 0), (dict(n=0), 0), (dict(V=1), 0),
    (dict(dtype=2), -1), (dict(backward=2), -1),
    (dict(n=-1), -2), (dict(n=(1 << 20) + 1), -2), (dict(C=60), -2), (dict(C=0), -2), (dict(C=(1 << 17) + 8), -2),
    (dict(V=0), -2), (dict(V=(1 << 24) + 1), -2), (dict(n=1 << 20, C=1 << 13), -2), (dict(n=1 << 14, V=1 << 23), -2),
])
def test_workspace_size(kw, code):
    rc, need = _size(**kw)
    assert rc == code
    assert (need > 0) == (code == 0 and kw.get("n", 100) > 0)


def test_workspace_does_not_grow_with_the_logits():
    """Sixteen times the vocabulary: the forward pass keeps eight bytes for 64
    logits, the backward pass a piece of bounded size."""
    small, large = (_size(n=4096, C=1024, V=V)[1] for V in (1 << 16, 1 << 20))
    assert large < 4096 * (1 << 20) * 2 / 8
    small, large = (_size(n=4096, C=1024, V=V, backward=1)[1] for V in (1 << 16, 1 << 20))
    assert large <= 1.1 * small


def _forward(H=P, ldh=64, W=P, targets=P, scale=1.0, loss=P, lse=P, n=10, C=64, V=1000, dtype=BF16, ws=P,
             ws_bytes=1 << 40):
    return D.lib().dyra_vocab_loss_forward(H, ldh, W, targets, scale, loss, lse, n, C, V, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=None), -1), (dict(W=None), -1), (dict(targets=None), -1), (dict(loss=None), -1), (dict(lse=None), -1),
    (dict(ws=None), -1), (dict(H=P + 2), -1), (dict(W=P + 8), -1), (dict(targets=P + 2), -1), (dict(loss=P + 1), -1),
    (dict(ws=P + 8), -1), (dict(dtype=5), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=2.0 ** 127), -1),
    (dict(ldh=56), -2), (dict(ldh=68), -2), (dict(ldh=(1 << 20) + 8), -2), (dict(C=12), -2), (dict(V=0), -2),
    (dict(n=-2), -2), (dict(ws_bytes=64), -3),
])
def test_forward_rejects_before_any_hip_call(kw, code):
    assert _forward(**kw) == code


def _backward(H=P, ldh=64, W=P, targets=P, lse=P, dloss=P, scale=1.0, dH=P, lddh=64, dW=P, n=10, C=64, V=1000,
              dtype=BF16, ws=P, ws_bytes=1 << 40):
    return D.lib().dyra_vocab_loss_backward(H, ldh, W, targets, lse, dloss, scale, dH, lddh, dW, n, C, V, dtype, ws,
                                            ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=None), -1), (dict(W=None), -1), (dict(targets=None), -1), (dict(lse=None), -1), (dict(dloss=None), -1),
    (dict(dH=None, dW=None), -1), (dict(ws=None), -1), (dict(dH=P + 2), -1), (dict(dW=P + 4), -1),
    (dict(lse=P + 2), -1), (dict(scale=0.0), -1), (dict(scale=2.0 ** 127), -1), (dict(dtype=3), -1),
    (dict(lddh=60), -2), (dict(ldh=60), -2), (dict(V=-1), -2), (dict(ws_bytes=1 << 8), -3),
])
def test_backward_rejects_before_any_hip_call(kw, code):
    assert _backward(**kw) == code


def test_a_call_of_no_rows_is_done_on_the_host():
    assert _forward(n=0, H=None, W=None, targets=None, loss=None, lse=None, ws=None, ws_bytes=0) == 0
    assert _backward(n=0, dW=None, H=None, W=None, targets=None, lse=None, dloss=None, ws=None, ws_bytes=0) == 0


def _tensors(n=10, c=64, v=30):
    import torch
    return dict(H=torch.zeros((n, c), dtype=torch.bfloat16), W=torch.zeros((v, c), dtype=torch.bfloat16),
                targets=torch.zeros(n, dtype=torch.int32))


@pytest.mark.parametrize("change,msg", [
    (lambda t: t.update(H=t["H"].double()), "H must be torch.bfloat16 or torch.float32"),
    (lambda t: t.update(H=t["H"][0]), "H must be a 2-D tensor"),
    (lambda t: t.update(targets=None), "targets must be a 1-D tensor"),
    (lambda t: None, "H must be a GPU tensor"),
])
def test_binding_rejects_before_the_library(change, msg):
    from input_adaptive_rank_amd import vocab_loss as L
    t = _tensors()
    change(t)
    with pytest.raises(ValueError, match=msg):
        L.vocab_loss_forward(t["H"], t["W"], t["targets"])
    with pytest.raises(ValueError, match=msg):
        L.vocab_loss_backward(t["H"], t["W"], t["targets"], None, None)


def test_workspace_size_refuses_other_types():
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    assert L.vocab_loss_workspace_size(100, 64, 1000, torch.bfloat16) == _size()[1]
    with pytest.raises(ValueError, match="dtype"):
        L.vocab_loss_workspace_size(100, 64, 1000, torch.float16)


def test_oracle_worked_example():
    """Two words, logits (0, log 3): probabilities 1/4 and 3/4."""
    H, W = np.array([[1.0, 0.0]]), np.array([[0.0, 5.0], [np.log(3.0), 7.0]])
    loss, lse, _ = O.forward(H, W, np.array([0]))
    assert np.allclose([loss[0], lse[0]], np.log(4.0))
    dH, dW, d, _ = O.backward(H, W, np.array([0]), lse, np.array([2.0]))
    assert np.allclose(d, [[-1.5, 1.5]])
    assert np.allclose(dH, [[1.5 * np.log(3.0), 3.0]]) and np.allclose(dW, [[-1.5, 0.0], [1.5, 0.0]])


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(3)
    H, W = rng.standard_normal((5, 8)), rng.standard_normal((11, 8))
    t, g = np.array([3, -1, 10, 11, 0]), rng.standard_normal(5)
    lse = O.forward(H, W, t, 0.7)[1]
    dH, dW, _, _ = O.backward(H, W, t, lse, g, 0.7)
    assert not dH[1].any() and not dH[3].any()
    total = lambda h, w: (O.forward(h, w, t, 0.7)[0] * g).sum()  # noqa: E731
    for x, dx, f in ((H, dH, lambda s: total(s, W)), (W, dW, lambda s: total(H, s))):
        step = rng.standard_normal(x.shape)
        h = 1e-4
        slope = (f(x + h * step) - f(x - h * step)) / (2 * h)
        assert abs(slope - (dx * step).sum()) <= 1e-6 * np.abs(dx * step).sum()
