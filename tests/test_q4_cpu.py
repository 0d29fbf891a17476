"""Host checks of the 4-bit projection: the library rejects bad arguments with
the documented codes, the binding with ValueError, before any HIP call."""
import ctypes

import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import q4_oracle as O

BF16, F32 = synth.DT_BF16, synth.DT_F32
P = 1 << 12   # a fake, never dereferenced, aligned address


def _packed(c1, c2, group):
    need = ctypes.c_size_t()
    return D.lib().dyra_q4_packed_size(c1, c2, group, ctypes.byref(need)), need.value


@pytest.mark.parametrize("args,code", [
    ((4096, 4096, 128), 0), ((8, 8, 32), 0), ((1 << 20, 1 << 14, 64), 0),
    ((64, 64, 16), -1), ((64, 64, 0), -1), ((64, 64, 256), -1),
    ((60, 64, 32), -2), ((64, 4, 32), -2), ((0, 64, 32), -2), ((64, -8, 32), -2), (((1 << 20) + 8, 8, 32), -2),
    ((1 << 20, 1 << 15, 32), -2),
])
def test_packed_size(args, code):
    rc, size = _packed(*args)
    assert rc == code
    if code == 0:
        c1, c2, group = args
        blocks = -(-c2 // 16) * -(-c1 // 128)
        assert size == blocks * (1024 + 128 // group * 64)


def _size(c1=4096, c2=4096, n=2000, dtype=BF16, backward=0):
    need = ctypes.c_size_t()
    return D.lib().dyra_q4_workspace_size(c1, c2, n, dtype, backward, ctypes.byref(need)), need.value


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(dtype=F32), 0), (dict(backward=1), 0), (dict(n=0), 0), (dict(n=1), 0), (dict(n=1, backward=1), 0),
    (dict(dtype=2), -1), (dict(backward=2), -1), (dict(c1=60), -2), (dict(n=-1), -2), (dict(n=(1 << 24) + 1), -2),
    (dict(n=1 << 21), -2),
])
def test_workspace_size(kw, code):
    rc, need = _size(**kw)
    assert rc == code
    if code == 0:
        few = kw.get("n", 2000) <= 1 and not (kw.get("backward") and kw.get("n"))
        assert (need == 0) == few


def test_few_rows_need_no_workspace_and_many_hold_the_weight():
    for dtype, size in ((BF16, 2), (F32, 4)):
        for n in (1, 16, 48, 64):
            assert _size(n=n, dtype=dtype) == (0, 0)
        assert _size(n=4096, dtype=dtype)[1] >= size * 4096 * 4096


def _forward(c1=64, c2=96, group=32, packed=P, X=P, ldx=64, bias=None, Y=P, ldy=96, n=5, dtype=BF16, ws=P,
             ws_bytes=1 << 40):
    return D.lib().dyra_q4_forward(D.Q4(c1, c2, group, packed), X, ldx, bias, Y, ldy, n, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(packed=None), -1), (dict(packed=P + 8), -1), (dict(group=48), -1), (dict(X=None), -1), (dict(X=P + 2), -1),
    (dict(Y=None), -1), (dict(Y=P + 8), -1), (dict(bias=P + 4), -1), (dict(dtype=9), -1), (dict(ws=P + 4), -1),
    (dict(c1=60), -2), (dict(c2=0), -2), (dict(n=-1), -2), (dict(ldx=56), -2), (dict(ldx=68), -2), (dict(ldy=90), -2),
    (dict(ldx=(1 << 20) + 8), -2), (dict(dtype=F32, ldx=66), -2),
    (dict(c1=4096, c2=4096, ldx=4096, ldy=4096, n=4096, ws=None), -1),
    (dict(c1=4096, c2=4096, ldx=4096, ldy=4096, n=4096, ws_bytes=1 << 20), -3),
])
def test_forward_rejects_before_any_hip_call(kw, code):
    assert _forward(**kw) == code


def test_a_call_of_no_rows_is_done_on_the_host():
    assert _forward(n=0, X=None, Y=None, ws=None, ws_bytes=0) == 0
    w = D.Q4(64, 96, 32, P)
    assert D.lib().dyra_q4_backward(w, None, 96, None, 64, 0, BF16, None, 0, None) == 0
    assert D.lib().dyra_q4_forward(None, P, 64, None, P, 96, 5, BF16, P, 1 << 30, None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), -1), (dict(dX=None), -1), (dict(dX=P + 2), -1), (dict(ws=None), -1), (dict(dtype=5), -1),
    (dict(lddy=88), -2), (dict(lddx=60), -2), (dict(n=-4), -2), (dict(ws_bytes=16), -3),
])
def test_backward_rejects_before_any_hip_call(kw, code):
    a = dict(dict(dY=P, lddy=96, dX=P, lddx=64, n=5, dtype=BF16, ws=P, ws_bytes=1 << 40), **kw)
    w = D.Q4(64, 96, 32, P)
    assert D.lib().dyra_q4_backward(w, a["dY"], a["lddy"], a["dX"], a["lddx"], a["n"], a["dtype"], a["ws"],
                                    a["ws_bytes"], None) == code


def test_pack_quantise_and_dense_reject_before_any_hip_call():
    L = D.lib()
    assert L.dyra_q4_pack(64, 96, 32, None, P, None, P, None) == -1
    assert L.dyra_q4_pack(64, 96, 32, P + 2, P, None, P, None) == -1
    assert L.dyra_q4_pack(64, 96, 32, P, P + 1, None, P, None) == -1
    assert L.dyra_q4_pack(64, 96, 32, P, P, None, P + 4, None) == -1
    assert L.dyra_q4_pack(64, 96, 33, P, P, None, P, None) == -1
    assert L.dyra_q4_pack(62, 96, 32, P, P, None, P, None) == -2
    assert L.dyra_q4_quantise(None, 64, 96, 32, BF16, P, P, None, None) == -1
    assert L.dyra_q4_quantise(P, 64, 96, 32, 3, P, P, None, None) == -1
    assert L.dyra_q4_quantise(P + 4, 64, 96, 32, BF16, P, P, None, None) == -1
    assert L.dyra_q4_quantise(P, 64, 0, 32, BF16, P, P, None, None) == -2
    w = D.Q4(64, 96, 32, P)
    assert L.dyra_q4_dense(w, None, BF16, None) == -1
    assert L.dyra_q4_dense(w, P + 8, BF16, None) == -1
    assert L.dyra_q4_dense(w, P, 7, None) == -1
    assert L.dyra_q4_dense(D.Q4(64, 96, 32, None), P, BF16, None) == -1


def test_binding_rejects_before_the_library():
    import torch
    from input_adaptive_rank_amd import q4 as Q
    codes = torch.zeros((96, 32), dtype=torch.uint8)
    for call, msg in [
        (lambda: Q.q4_pack(codes, None), "codes must be a GPU tensor"),
        (lambda: Q.q4_pack(codes[0], None), "2-D"),
        (lambda: Q.q4_quantise(torch.zeros((96, 64))), "W must be a GPU tensor"),
        (lambda: Q.q4_quantise(torch.zeros((96, 64), dtype=torch.float16)), "bfloat16 or torch.float32"),
        (lambda: Q.q4_quantise("W"), "2-D tensor"),
        (lambda: Q.Q4Weight(64, 96, 48, codes), "group must be one of"),
        (lambda: Q.Q4Weight(62, 96, 32, codes), "multiples of 8"),
        (lambda: Q.Q4Weight(64, 96, 32, codes), "GPU tensor"),
        (lambda: Q.q4_forward(torch.zeros((2, 64)), codes), "Q4Weight"),
        (lambda: Q.q4_backward(torch.zeros((2, 64)), None), "Q4Weight"),
        (lambda: Q.q4_dense(codes), "Q4Weight"),
        (lambda: Q.q4_workspace_size(64, 64, 5, torch.float16), "dtype"),
    ]:
        with pytest.raises(ValueError, match=msg):
            call()


def test_oracle_codes_are_the_nearest():
    """No other code of a value lies nearer to it (but for clamped ends), and
    the worked example: scale 1, codes 8 + value."""
    codes, scale, zero = O.quantise(np.array([[-7.0, 0.0, 0.5, 1.5, 2.5, 7.0, 3.0, -1.0]]), 32, False)
    assert scale.tolist() == [[1.0]] and zero is None
    assert codes.tolist() == [[1, 8, 8, 10, 10, 15, 11, 7]]   # halves go to the even code
    rng = np.random.default_rng(0)
    W = synth.round_bf16(rng.standard_normal((5, 72)))
    for zp in (False, True):
        codes, scale, zero = O.quantise(W, 32, zp)
        got = O.weight(codes, scale, zero, 32)
        step = np.repeat(scale, 32, axis=1)[:, :72]
        inner = (codes > 0) & (codes < 15)
        assert np.all(np.abs(got - W)[inner] <= 0.5 * step[inner] * (1 + 1e-6))
        assert np.all((codes >= 0) & (codes <= 15))
