"""Gradients of the vocabulary loss where the vocabulary is taken in several
pieces, and what they may write.  References in float64 on the device; bounds as in
test_gpu_vocab_loss."""
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth

from gpu_cases import log

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U, HALF = 2.0 ** -24, {F32: 2.0 ** -24, BF16: 2.0 ** -8}
IDS = {F32: "fp32", BF16: "bf16"}
GUARD = 1 << 23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def up(a, m):
    return -(-a // m) * m


def make(n, c, v, dtype, seed, ignored=0.3):
    """H, W, targets, dloss; the last word and the first are targets too."""
    import torch
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn((v, c), generator=gen, device="cuda") / c ** 0.5).to(td)
    t = torch.randint(0, v, (n,), generator=gen, device="cuda")
    t[n // 2], t[n // 3] = v - 1, 0
    H = (torch.randn((n, c), generator=gen, device="cuda") + 6 * W[t].float()).to(td)
    t[torch.rand(n, generator=gen, device="cuda") < ignored] = -1
    return H, W, t.int(), torch.rand(n, generator=gen, device="cuda") / n


def guarded(size):
    import torch
    return torch.full((size + GUARD,), 90, dtype=torch.uint8, device="cuda")


def check_gradients(H, W, t, g, lse, dH, dW, dtype, pieces):
    """In blocks of words, so that float64 logits of a large vocabulary fit."""
    import torch
    n, c = H.shape
    v = W.shape[0]
    terms = 6 if dtype == F32 else 1
    live = torch.nonzero(t >= 0)[:, 0]
    Hd, at = H[live].double(), t[live].long()
    w, l2 = g[live].double()[:, None], lse[live].double()[:, None]
    dh, eh, mh = (torch.zeros_like(Hd) for _ in range(3))
    block = max(64, (1 << 27) // max(n, c) // 64 * 64)
    for v0 in range(0, v, block):
        Wd = W[v0:v0 + block].double()
        a, mag = Hd @ Wd.t(), Hd.abs() @ Wd.abs().t()
        p = torch.exp(a - l2)
        ea = (terms * (c / 16 + 2) + 67) * U * mag + U * (4 * a.abs() + 4 * l2.abs() + 4)
        d = p.clone()
        here = torch.nonzero((at >= v0) & (at < v0 + block))[:, 0]
        d[here, at[here] - v0] -= 1
        d *= w
        e = w * p * ea + 3 * U * d.abs() + 2.0 ** -126
        if dtype == BF16:
            e += 2.0 ** -8 * (d.abs() + e)
        ad = d.abs() + e
        dh += d @ Wd
        eh += e @ Wd.abs()
        mh += ad @ Wd.abs()
        if dW is not None:
            want, err, mags = d.t() @ Hd, e.t() @ Hd.abs(), ad.t() @ Hd.abs()
            lim = err + (terms * (len(live) / 16 + 6) + 72) * U * mags + HALF[dtype] * (want.abs() * (1 + 2.0 ** -6) + err)
            got = dW[v0:v0 + block].double()
            assert bool(((got - want).abs() <= lim + 2.0 ** -126).all()), f"dW of words from {v0}"
    if dH is not None and len(live):
        lim = eh + (terms * (v / 16 + 6) + 72 + pieces) * U * mh + HALF[dtype] * (dh.abs() * (1 + 2.0 ** -6) + eh)
        got = dH[live].double()
        log(f"    dH: worst error {float(((got - dh).abs() / lim).max()):.3f} of its bound, "
            f"relative {float((got - dh).norm() / dh.norm()):.2e}")
        assert bool(((got - dh).abs() <= lim).all()), "dH"
    assert dH is None or not bool(dH[t < 0].any())


# planes: fp32 weights are written out as planes (else read as they are)
PIECES = [(BF16, 4099, 128, 33000, False, 2), (BF16, 9001, 64, 31000, False, 3), (BF16, 40000, 64, 6000, False, 2),
          (F32, 8, 64, 1049687, False, 2), (F32, 300, 64, 1049687, False, 3), (F32, 400, 8192, 10816, True, 2),
          (F32, 600, 16384, 12000, True, 3), (F32, 9001, 64, 31000, True, 3)]


@pytest.mark.parametrize("dtype,n,c,v,planes,pieces", PIECES,
                         ids=["-".join([IDS[p[0]], *map(str, p[1:4])]) for p in PIECES])
def test_gradients_of_several_pieces(dtype, n, c, v, planes, pieces):
    """The last piece is shorter than the others.  Each gradient alone has the same
    bits, and nothing behind a workspace of exactly the size asked for is written."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    # how many pieces: d of one is at most 2^27 elements, its planes of W 2^28
    most = min(1 << 20, (1 << 27) // n)
    if planes:
        most = min(most, (1 << 28) // (3 * c))
    most = max(256, most // 256 * 256)
    piece = min(up(v, 64), up(-(-v // -(-v // most)), 256))
    assert -(-v // piece) == pieces and v % piece
    # and that the library does the same: its workspace holds those planes, d of such a
    # piece and partial tiles, and not the whole
    kinds = 3 if dtype == F32 else 1
    least = lambda cols: 2 * kinds * (n * c + n * cols + (cols * c if planes else 0)) + 4 * n * c  # noqa: E731
    parts = 135 << 20 if planes or dtype == BF16 else 17 << 20
    size = L.vocab_loss_workspace_size(n, c, v, dtype, True, need_dw=False)
    assert least(piece) <= size <= least(piece) + parts
    assert size < least(up(v, 64))

    H, W, t, g = make(n, c, v, dtype, seed=41)
    lse = L.vocab_loss_forward(H, W, t)[1]
    out = {}
    for need in ((True, True), (True, False), (False, True)):
        size = L.vocab_loss_workspace_size(n, c, v, dtype, True, *need)
        ws = guarded(size)
        out[need] = L.vocab_loss_backward(H, W, t, lse, g, need_dh=need[0], need_dw=need[1], workspace=ws)
        assert bool((ws[size:] == 90).all())
        del ws
    dH, dW = out[True, True]
    assert out[True, False][1] is None and out[False, True][0] is None
    assert torch.equal(out[True, False][0], dH) and torch.equal(out[False, True][1], dW)
    check_gradients(H, W, t, g, lse, dH, dW, dtype, pieces)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("ignored", [0.0, 0.5, 0.9])
@pytest.mark.parametrize("n,c,v", [(3, 264, 1000), (64, 520, 3001), (257, 264, 1024), (700, 1024, 5000), (1500, 512, 600),
                                   (9001, 136, 515)])
def test_nothing_behind_the_workspace_is_written(n, c, v, ignored, dtype):
    """Partial tiles follow from the rows that count, which the device finds."""
    from input_adaptive_rank_amd import vocab_loss as L
    H, W, t, g = make(n, c, v, dtype, seed=42, ignored=ignored)
    size = L.vocab_loss_workspace_size(n, c, v, dtype)
    ws = guarded(size)
    lse = L.vocab_loss_forward(H, W, t, workspace=ws)[1]
    assert bool((ws[size:] == 90).all())
    for need in ((True, True), (True, False), (False, True)):
        size = L.vocab_loss_workspace_size(n, c, v, dtype, True, *need)
        ws = guarded(size)
        dH, dW = L.vocab_loss_backward(H, W, t, lse, g, need_dh=need[0], need_dw=need[1], workspace=ws)
        assert bool((ws[size:] == 90).all())
        check_gradients(H, W, t, g, lse, dH, dW, dtype, 1)
