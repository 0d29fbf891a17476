"""That fp32 products hold 24 bits of both operands: results of a single product
each, within a few roundings (plane_cases derives the bounds and what a missing plane
would do to them)."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import q4_oracle as QO

import plane_cases as P
from gpu_cases import log
from test_gpu_q4 import make, pack, put
from test_gpu_vocab_loss import floats, host, ints

pytestmark = pytest.mark.gpu

F32, U = synth.DT_F32, P.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def check(name, got, want, units):
    """units: of U, relative to the result."""
    off = np.abs(host(got) - want)
    worst = float((off / np.maximum(np.abs(want), 1e-30)).max() / U)
    log(f"    {name}: worst error {worst:.2f} U, bound {np.max(units):.2f}")
    assert np.all(off <= units * U * np.abs(want)), name


# W is read as it is in the first two, and by gradients written out as planes in the
# others, by the loss in the last
SIZES = [(5, 64, 130), (130, 264, 1000), (700, 1024, 5000), (1500, 512, 8000)]


@pytest.mark.parametrize("n,c,v", [(1, 8, 1)] + SIZES)
def test_logits(n, c, v):
    """Rows of one entry and a single word that is not zero: where its logit is
    large enough, lse is that logit."""
    from input_adaptive_rank_amd import vocab_loss as L
    H, x = P.single_entries(n, c, 51)
    W = np.zeros((v, c))
    W[v // 2] = 64 * P.numbers(c, 52)   # logits above 64 x 0.01, others 0
    a = (H * W[v // 2]).sum(1)
    far = a > 60 + np.log(v)            # others add less than e^-60
    assert far.mean() > 0.9
    loss, lse = L.vocab_loss_forward(put(H, F32), put(W, F32), ints(np.full(n, v // 2)))
    check("lse", lse[np.nonzero(far)[0]], a[far], P.THREE_BY_THREE + 1)
    assert not host(loss)[far].any()


@pytest.mark.parametrize("n,c,v", SIZES)
def test_gradients(n, c, v):
    """H = 0 and one word a column: dH is one product.  W = 0 and rows of one
    entry: dW is one product for each of the rows that share a column.  All words
    have the probability 1 / v."""
    from input_adaptive_rank_amd import vocab_loss as L
    rng = np.random.default_rng(53)
    t, g = rng.integers(0, v, n), np.float32(1.0 + rng.random(n)).astype(np.float64)
    units = P.probability_bound(v)
    rows, cols = np.arange(n), np.arange(c)
    # d for the lse that the device gives
    H, W = np.zeros((n, c)), np.zeros((v, c))
    word = cols * 7 % v
    W[word, cols] = w = P.numbers(c, 54)
    lse = L.vocab_loss_forward(put(H, F32), put(W, F32), ints(t))[1]
    d = np.exp(-host(lse))[:, None] * np.ones((n, v))
    d[rows, t] -= 1
    d *= g[:, None]
    dH, _ = L.vocab_loss_backward(put(H, F32), put(W, F32), ints(t), lse, floats(g), need_dw=False)
    check("dH", dH, d[:, word] * w[None, :], units)
    H, x = P.single_entries(n, c, 55)
    W[:] = 0
    _, dW = L.vocab_loss_backward(put(H, F32), put(W, F32), ints(t), lse, floats(g), need_dh=False)
    want, mag = d.T @ H, np.abs(d).T @ np.abs(H)
    off = np.abs(host(dW) - want) / np.maximum(mag, 1e-30) / U
    log(f"    dW: worst error {off.max():.2f} U, bound {units + -(-n // c):.2f}")
    assert off.max() <= units + -(-n // c)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n,c1,c2", [(1, 64, 24), (40, 264, 520), (900, 1024, 4096), (600, 264, 6000)])
def test_projections(n, c1, c2, group):
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, c1, c2, group, True, F32, seed=56)
    w = pack(c)
    X, x = P.single_entries(n, c1, 57)
    few = Q.q4_workspace_size(c1, c2, n, F32) == 0
    assert few == (n < 100)
    # few rows: three exact products, the last of their sums, the scale's product
    check("Y", Q.q4_forward(put(X, F32), w), QO.forward(X, c["W"])[0], 3.2 if few else P.THREE_BY_TWO)
    dY, _ = P.single_entries(n, c2, 58)
    check("dX", Q.q4_backward(put(dY, F32), w), QO.backward(dY, c["W"])[0], P.THREE_BY_TWO)
