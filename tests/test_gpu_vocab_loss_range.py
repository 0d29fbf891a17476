"""The vocabulary loss at the ends of its range: fp32 values next to the largest,
words that are certain, the largest scale, operands past 2^31 bytes.  References in
float64, bounds as in test_gpu_vocab_loss."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import vocab_loss_oracle as O

from gpu_cases import log
from test_gpu_vocab_loss import check_backward, check_forward, floats, host, ints, make, put

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U, HALF = 2.0 ** -24, {F32: 2.0 ** -24, BF16: 2.0 ** -8}
IDS = {F32: "fp32", BF16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


# fp32: the first two round to an infinity in bf16
@pytest.mark.parametrize("dtype,value", [(BF16, -3.3895313892515355e38), (F32, -3.4028234663852886e38),
                                         (F32, -3.3961775292304601e38), (F32, -3.3895313892515355e38), (F32, -1e38)])
@pytest.mark.parametrize("n,c,v", [(3, 72, 300), (70, 64, 300), (600, 1024, 3000)])
def test_words_masked_by_their_weights(n, c, v, dtype, value):
    """Words whose weights are next to the type's lowest value, met by rows of
    positive entries: their logits are -inf or of that size, they have no
    probability and no gradient, and all others are what they are without them."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    case = make(n, c, v, dtype, seed=21)
    case["H"] = np.abs(case["H"])
    gone = np.array([0, 63, 64, 130, v - 1])
    keep = np.setdiff1d(np.arange(v), gone)
    rest = dict(case, W=case["W"][keep])
    # each row that counts keeps its word, or takes another
    t = case["t"]
    rest["t"] = np.where((t < 0) | (t >= v), -1, np.searchsorted(keep, t) % len(keep))
    t = np.where(rest["t"] < 0, -1, keep[rest["t"]])
    W = put(case["W"], dtype)
    W[torch.from_numpy(gone).cuda()] = value
    H = put(case["H"], dtype)
    loss, lse = L.vocab_loss_forward(H, W, ints(t))
    check_forward(rest, dtype, loss, lse)
    dH, dW = L.vocab_loss_backward(H, W, ints(t), lse, floats(rest["dloss"]))
    check_backward(rest, dtype, lse, dH, dW[torch.from_numpy(keep).cuda()])
    assert not bool(dW[torch.from_numpy(gone).cuda()].any())


@pytest.mark.parametrize("n,c,v", [(5, 64, 130), (600, 1024, 3000)])
def test_hidden_values_next_to_the_largest(n, c, v):
    """fp32 rows with entries at the type's ends, whose weights are small enough
    for the logits to be ordinary numbers."""
    from input_adaptive_rank_amd import vocab_loss as L
    case = make(n, c, v, F32, seed=22)
    g = np.random.default_rng(23)
    ends = np.array([3.4028234663852886e38, -3.4028234663852886e38, 3.3961775292304601e38, 3.4e38])
    case["H"][:, 5] = synth.round_f32(g.choice(ends, n))
    case["W"][:, 5] = synth.round_f32(case["W"][:, 5] * 2.0 ** -100)
    case["dloss"][:], case["scale"] = 1.0 / n, 2.0 ** -24
    H, W, t = put(case["H"], F32), put(case["W"], F32), ints(case["t"])
    loss, lse = L.vocab_loss_forward(H, W, t, case["scale"])
    check_forward(case, F32, loss, lse)
    dH, _ = L.vocab_loss_backward(H, W, t, lse, floats(case["dloss"]), case["scale"], need_dw=False)
    check_backward(case, F32, lse, dH, None, need=(True, False))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("scale", [1.0, 0.7, 1 / 3])
@pytest.mark.parametrize("size", [1.0, 10.0, 100.0])
def test_the_loss_of_a_certain_word_is_not_negative(size, scale, dtype):
    """lse is at least every logit, so no loss is below 0: the target's logit and
    the largest one are rounded alike before they are subtracted.  Logits up to 7,
    70 and 700, most targets far above the others."""
    from input_adaptive_rank_amd import vocab_loss as L
    g = np.random.default_rng(24)
    n, c, v = 800, 64, 300
    W = synth.round_storage(g.standard_normal((v, c)) / 8, dtype)
    t = g.integers(0, v, n)
    H = synth.round_storage(size * (1 + 6 * g.random((n, 1))) * W[t], dtype)
    case = dict(H=H, W=W, t=t, scale=scale)
    loss, lse = L.vocab_loss_forward(put(H, dtype), put(W, dtype), ints(t), scale)
    check_forward(case, dtype, loss, lse)
    log(f"    least loss {float(loss.min()):.3e}")
    assert float(loss.min()) >= 0.0
    # a single word: the logit itself, and no loss at all
    for m in (1, 70, 800):
        loss, lse = L.vocab_loss_forward(put(H[:m], dtype), put(W[:1], dtype), ints(np.zeros(m)), scale)
        assert not bool(loss.any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("scale", [1.0, 0.25, 2.0 ** 126])
def test_the_gradient_of_a_single_word_is_zero(scale, dtype):
    """Its probability is exp(a - lse) = 1, whatever its logit."""
    from input_adaptive_rank_amd import vocab_loss as L
    g = np.random.default_rng(25)
    for n in (7, 700):
        W = put(synth.round_storage(g.standard_normal((1, 64)), dtype), dtype)
        H = g.standard_normal((n, 64)) * (10.0 if scale < 2 else 2.0 ** -7)
        H, t = put(synth.round_storage(H, dtype), dtype), ints(np.zeros(n))
        loss, lse = L.vocab_loss_forward(H, W, t, scale)
        assert not bool(loss.any())
        dH, dW = L.vocab_loss_backward(H, W, t, lse, floats(g.standard_normal(n)), scale)
        assert not bool(dH.any()) and not bool(dW.any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
def test_the_largest_scale(dtype):
    """A scale of 2^126: the largest logits are next to the type's end."""
    from input_adaptive_rank_amd import vocab_loss as L
    g = np.random.default_rng(25)
    n, c, v = 40, 64, 130
    W = synth.round_storage(g.standard_normal((v, c)) / 8, dtype)
    H = synth.round_storage(g.standard_normal((n, c)), dtype)
    H /= 2.0 ** np.ceil(np.log2(np.abs(H @ W.T).max(1, keepdims=True)) - 1.9)   # magnitudes up to 1.87 .. 3.74
    t = g.integers(0, v, n)
    loss, lse = L.vocab_loss_forward(put(H, dtype), put(W, dtype), ints(t), 2.0 ** 126)
    # a target far below the largest logit: a loss past fp32's largest number
    past = O.forward(H, W, t, 2.0 ** 126)[0] >= 2.0 ** 128
    assert past.any() and not past.all() and np.array_equal(np.isinf(host(loss)), past)
    at = np.nonzero(~past)[0]
    check_forward(dict(H=H[at], W=W, t=t[at], scale=2.0 ** 126), dtype, loss[at], lse[at])


@pytest.mark.parametrize("n,c,v,ldh", [(2200, 64, 300, 1 << 20), (4, 32768, 33000, 32768), (1100, 64, 300, 1 << 20)])
def test_operands_beyond_two_gibibytes(n, c, v, ldh):
    """Rows, weights and their gradients whose last bytes lie past 2^31 (2200 rows
    2^21 bytes apart: past 2^32)."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    gen = torch.Generator(device="cuda").manual_seed(26)
    W = (torch.randn((v, c), generator=gen, device="cuda") / c ** 0.5).bfloat16()
    t = torch.randint(0, v, (n,), generator=gen, device="cuda")
    t[-1] = v - 1
    H = (torch.randn((n, c), generator=gen, device="cuda") + 3 * W[t].float()).bfloat16()
    wide, dwide = (torch.empty((n, ldh), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h, dh = wide[:, ldh - c:], dwide[:, ldh - c:]
    h.copy_(H)
    loss, lse = L.vocab_loss_forward(h, W, t.int())
    g = torch.full((n,), 1.0 / n, device="cuda")
    dW = L.vocab_loss_backward(h, W, t.int(), lse, g, dH=dh)[1]
    a = H.double() @ W.double().t()
    mag = (H.double().abs() @ W.double().abs().t()).amax(1)
    want = torch.logsumexp(a, 1)
    ea = (c / 16 + 66) * U * mag
    bound = ea + U * (4 * a.abs().amax(1) + 132 + v / 2048 + 4 * want.abs())
    assert bool(((lse - want).abs() <= bound).all())
    rows = torch.arange(n, device="cuda")
    assert bool(((loss - (want - a[rows, t])).abs() <= 2 * bound + U * 4 * a.abs().amax(1)).all())
    p = torch.exp(a - lse.double()[:, None])
    d = p.clone()
    d[rows, t] -= 1
    d /= n
    e = p / n * (ea + U * (4 * a.abs().amax(1) + 4 * lse.double().abs() + 4))[:, None] + 3 * U * d.abs()
    e += 2.0 ** -8 * (d.abs() + e)
    lim = lambda err, mags, want, K: (err + (K / 16 + 70) * U * mags) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()  # noqa: E731
    Wd, Hd = W.double(), H.double()
    dhw, dww = d @ Wd, d.t() @ Hd
    assert bool(((dh.double() - dhw).abs() <= lim(e @ Wd.abs(), (d.abs() + e) @ Wd.abs(), dhw, v)).all())
    assert bool(((dW.double() - dww).abs() <= lim(e.t() @ Hd.abs(), (d.abs() + e).t() @ Hd.abs(), dww, n)).all())
