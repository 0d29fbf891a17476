"""Host checks of the adapter entry points: the library rejects bad arguments
with the documented codes, the binding with ValueError, before any HIP call."""
import ctypes

import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth

BF16, F32 = synth.DT_BF16, synth.DT_F32


def _size(slots=4, r=16, c1=64, c2=96, n=100, B=7, dtype=BF16, backward=0):
    need = ctypes.c_size_t()
    return D.lib().dyra_adapter_workspace_size(slots, r, c1, c2, n, B, dtype, backward, ctypes.byref(need)), need.value


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(dtype=F32), 0), (dict(n=0, B=0), 0), (dict(r=128), 0), (dict(slots=2048), 0),
    (dict(dtype=2), -1), (dict(backward=2), -1),
    (dict(slots=0), -2), (dict(slots=2049), -2), (dict(r=0), -2), (dict(r=12), -2), (dict(r=136), -2),
    (dict(c1=60), -2), (dict(c2=0), -2), (dict(c1=1 << 25), -2), (dict(n=-1), -2), (dict(n=1 << 30), -2),
    (dict(B=-1), -2),
])
def test_workspace_size(kw, code):
    """(A few rows need no workspace; the thousand here do.)"""
    rc, need = _size(**dict(dict(n=1000), **kw))
    assert rc == code
    assert (need > 0) == (code == 0 and kw.get("n", 1000) > 0)


def test_workspace_grows_with_the_backward_pass():
    assert _size()[1] < _size(backward=1)[1]
    assert _size(n=1000)[1] < _size(n=2000)[1]


@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_follows_the_slots_that_can_be_used(backward):
    """Eight requests use at most eight slots of a pool of any size: but for
    a word a slot, the same bytes."""
    kw = dict(r=64, c1=4096, c2=4096, n=5003, B=8, backward=backward)
    small, large, largest = (_size(slots=slots, **kw)[1] for slots in (8, 512, 2048))
    assert small <= large <= largest <= small + 4 * 2048 + 256


# fake, never dereferenced, aligned addresses: every call must be rejected on the host
P = 1 << 12


def _forward(slots=4, r=16, c1=64, c2=96, A=P, B=P, rank=None, scale=None, X=P, ldx=64, base=None, ldb=0, Y=P, ldy=96,
             H=None, n=1000, nb=7, off=P, ids=P, dtype=BF16, ws=P, ws_bytes=1 << 40):
    ad = D.Adapters(slots, r, c1, c2, A, B, rank, scale)
    return D.lib().dyra_adapter_forward(ad, X, ldx, base, ldb, Y, ldy, H, n, nb, off, ids, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), -1), (dict(B=None), -1), (dict(X=None), -1), (dict(Y=None), -1), (dict(ws=None), -1),
    (dict(off=None), -1), (dict(ids=None), -1), (dict(dtype=7), -1),
    (dict(A=P + 8), -1), (dict(X=P + 2), -1), (dict(Y=P + 4), -1), (dict(base=P + 8, ldb=96), -1), (dict(H=P + 4), -1),
    (dict(rank=P + 2), -1), (dict(scale=P + 1), -1), (dict(off=P + 2), -1), (dict(ws=P + 8), -1),
    (dict(ldx=56), -2), (dict(ldx=68), -2), (dict(ldy=90), -2), (dict(base=P, ldb=0), -2),
    (dict(r=9), -2), (dict(slots=-1), -2), (dict(n=-3), -2),
    (dict(ws_bytes=64), -3),
])
def test_forward_rejects_before_any_hip_call(kw, code):
    assert _forward(**kw) == code


def test_forward_of_no_rows_is_done_on_the_host():
    assert _forward(n=0, X=None, Y=None, ws=None, off=None, ids=None, nb=0) == 0
    assert _forward(n=0, r=9) == -2


def _backward(slots=4, r=16, c1=64, c2=96, A=P, B=P, X=P, ldx=64, dY=P, ldy=96, H=P, dXb=None, ldb=0, dX=P, ldo=64,
              dA=P, dB=P, n=100, nb=7, off=P, ids=P, dtype=BF16, ws=P, ws_bytes=1 << 40):
    ad = D.Adapters(slots, r, c1, c2, A, B, None, None)
    return D.lib().dyra_adapter_backward(ad, X, ldx, dY, ldy, H, dXb, ldb, dX, ldo, dA, dB, n, nb, off, ids, dtype, ws,
                                         ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), -1), (dict(X=None), -1), (dict(dY=None), -1), (dict(H=None), -1), (dict(dA=None), -1),
    (dict(dB=None), -1), (dict(dX=None, dA=None, dB=None), -1), (dict(dA=P + 8), -1), (dict(dX=P + 2), -1),
    (dict(off=None), -1), (dict(ws=None), -1),
    (dict(ldo=60), -2), (dict(ldy=88), -2), (dict(dXb=P, ldb=8), -2), (dict(c1=12), -2),
    (dict(ws_bytes=1 << 8), -3),
])
def test_backward_rejects_before_any_hip_call(kw, code):
    assert _backward(**kw) == code


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_launches_of_too_many_threads_are_rejected_before_any_hip_call(dtype):
    """2^32 threads or more: the tiles of 2^28 rows, the packing of a pool,
    the join of a pool's gradients."""
    kw = dict(dtype=dtype, ws_bytes=1 << 62)
    assert _forward(n=1 << 28, c1=8, c2=8, ldx=8, ldy=8, r=8, **kw) == -2
    assert _backward(n=1 << 28, c1=8, c2=8, ldx=8, ldy=8, ldo=8, r=8, **kw) == -2
    wide = 1 << 20
    assert _backward(n=10, nb=2048, slots=2048, c1=wide, c2=wide, ldx=wide, ldy=wide, ldo=wide, r=128, **kw) == -2


def _tensors(n=10, c1=64, c2=96, r=16, slots=3, nb=2):
    import torch
    bf = torch.bfloat16
    return dict(X=torch.zeros((n, c1), dtype=bf), A=torch.zeros((slots, r, c1), dtype=bf),
                B=torch.zeros((slots, c2, r), dtype=bf), offsets=torch.zeros(nb + 1, dtype=torch.int32),
                slots=torch.zeros(nb, dtype=torch.int32))


@pytest.mark.parametrize("change,msg", [
    (lambda t: t.update(X=t["X"].double()), "X must be torch.bfloat16 or torch.float32"),
    (lambda t: t.update(X=t["X"][0]), "X must be a 2-D tensor"),
    (lambda t: t.update(offsets=None), "offsets must be a 1-D tensor"),
    (lambda t: None, "X must be a GPU tensor"),
])
def test_binding_rejects_before_the_library(change, msg):
    from input_adaptive_rank_amd import adapters as AD
    t = _tensors()
    change(t)
    with pytest.raises(ValueError, match=msg):
        AD.adapter_forward(t["X"], t["A"], t["B"], t["offsets"], t["slots"])


def test_binding_operand_checks():
    """The checks behind the entry points, on host tensors."""
    import torch
    from input_adaptive_rank_amd import adapters as AD
    cpu, bf = torch.device("cpu"), torch.bfloat16
    t = torch.zeros((10, 64), dtype=bf)
    assert AD._rows(t, "t", 10, 64, bf, cpu) == (t.data_ptr(), 64)
    wide = torch.zeros((10, 96), dtype=bf)
    assert AD._rows(wide[:, 8:72], "t", 10, 64, bf, cpu) == (wide.data_ptr() + 16, 96)
    for bad in (wide[:, 4:68], wide[:, ::2][:, :40], torch.zeros((64, 10), dtype=bf).t(),
                torch.zeros((1, 64), dtype=bf).expand(10, 64), t.float(), t[:9], "x"):
        with pytest.raises(ValueError):
            AD._rows(bad, "t", 10, 64, bf, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        AD._flat(wide[:, :64], "t", (10, 64), bf, cpu)
    with pytest.raises(ValueError, match="overlap"):
        AD._apart(wide[:5], "out", [("X", wide[4:])])
    AD._apart(wide[:5], "out", [("X", wide[5:]), ("base", None)])
    assert AD._same(wide[:, :64], wide[:, :64]) and not AD._same(wide[:, :64], wide[:, 8:72])


def test_results_and_workspace_are_allocated_on_the_given_stream(monkeypatch):
    """A block of the current stream's pool could be handed out with work on it
    still pending there; only a result is for the current stream to use too."""
    import contextlib

    import torch
    from input_adaptive_rank_amd import adapters as AD
    current, other = object(), object()
    at, made = [current], []

    class Block:
        def __init__(self, shape, dtype, device):
            self.stream, self.recorded = at[-1], []
            made.append(self)

        def record_stream(self, stream):
            self.recorded.append(stream)

        def data_ptr(self):
            return P

        def numel(self):
            return 1

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    monkeypatch.setattr(torch, "empty", Block)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    ad = D.Adapters(4, 16, 64, 96, P, P, None, None)
    for stream in (None, other):
        out = AD._output(None, (1000, 96), torch.bfloat16, "cuda:0", stream)
        assert AD._workspace(None, ad, 1000, 7, BF16, 1, "cuda:0", stream)[2] is made[-1]
        assert out.recorded == ([] if stream is None else [current]) and made[-1].recorded == []
    assert [b.stream for b in made] == [current, current, other, other]


def test_column_ranges_of_one_matrix_do_not_overlap():
    """Against the bytes themselves: every pair of column and row ranges."""
    import itertools

    import torch
    from input_adaptive_rank_amd import adapters as AD
    base = torch.zeros(6 * 5, dtype=torch.bfloat16)
    wide = base.view(6, 5)
    views = [wide[r0:r1, c0:c1] for r0, r1 in ((0, 6), (0, 2), (2, 6), (3, 4), (1, 1))
             for c0, c1 in ((0, 5), (0, 2), (2, 5), (1, 4), (4, 5))]
    views += [base[3:15].view(4, 3), base[7:9].view(1, 2), base[7:9].view(2, 1), base[4:22].view(3, 3, 2)]
    where = torch.arange(30)
    bytes_of = [set(where.as_strided(v.shape, v.stride(), v.storage_offset()).flatten().tolist()) for v in views]
    for (a, x), (b, y) in itertools.product(zip(views, bytes_of), repeat=2):
        one_grid = a.dim() == b.dim() == 2 and (a.shape[0] < 2 or b.shape[0] < 2 or a.stride(0) == b.stride(0))
        if one_grid or x & y:
            assert AD._overlap(a, b) == bool(x & y), (a.shape, a.storage_offset(), b.shape, b.storage_offset())


def test_a_single_row_is_the_same_memory_whatever_its_stride():
    import torch
    from input_adaptive_rank_amd import adapters as AD
    wide = torch.zeros((3, 96), dtype=torch.bfloat16)
    row = wide[0, 8:72]
    assert AD._same(wide[:1, 8:72], row[None]) and not AD._same(wide[:1, 8:72], wide[:1, 16:80])
    assert not AD._same(wide[:2, :32], wide.view(9, 32)[:2])


def test_workspace_size_refuses_other_types():
    import torch
    from input_adaptive_rank_amd import adapters as AD
    sizes = (4, 16, 64, 96, 1000, 7)
    assert AD.adapter_workspace_size(*sizes, torch.bfloat16) == AD.adapter_workspace_size(*sizes, BF16) == _size(n=1000)[1]
    for dtype in (torch.float16, 7, "bf16"):
        with pytest.raises(ValueError, match="dtype"):
            AD.adapter_workspace_size(*sizes, dtype)
