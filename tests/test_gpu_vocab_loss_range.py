"""The vocabulary loss at the ends of its range: fp32 values next to the largest.
References in float64, bounds as in test_gpu_vocab_loss."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth

from gpu_cases import log
from test_gpu_vocab_loss import check_backward, check_forward, floats, ints, make, put

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
