"""The vocabulary loss (dyra_vocab_loss_*) through the package's entry points,
against the float64 oracle on the same inputs.

Bounds are sums of what each step may lose.  U = 2^-24 is a rounding to fp32,
2^-8 one to bf16.  A logit is a sum of C products on matrix instructions, which
add 16 of them at a time and the results one after the other: at most terms (C / 16 +
2) + 64 roundings of at most the sum of the products' magnitudes, terms = 6
plane pairs in fp32 (those left out are below 3 U of it) and 1 in bf16.  Its
exponential in powers of two has a scaled argument (two roundings of it) and a
result within 2 U; a row's sum adds 32 of them in a lane, then lanes, blocks of 64
columns and lanes again: at most 128 + V / 2048 roundings.  d is rounded to
bf16 for the products of the backward pass in bf16, in fp32 its three terms
hold it.  What is below 2^-126, the smallest normal fp32 number, may become 0
(a word 100 below the largest logit has a probability of e^-100 = 2^-144): each
of p, d and a result may be off by TINY = 2^-126 beside that."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import vocab_loss_oracle as O

from gpu_cases import log

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U, HALF, TINY = 2.0 ** -24, {F32: 2.0 ** -24, BF16: 2.0 ** -8}, 2.0 ** -126
IDS = {F32: "fp32", BF16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def put(a, dtype):
    return D.to_device(a, dtype).reshape(a.shape).contiguous()


def ints(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def floats(a):
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).cuda()


def make(n, c, v, dtype, seed, ignored=0.2, scale=1.0, size=1.0):
    """Rows some of which lean towards their targets; now and then the same
    target twice, the first and the last word, and targets outside."""
    g = np.random.default_rng(seed)
    W = synth.round_storage(g.standard_normal((v, c)) * size / np.sqrt(c), dtype)
    t = g.integers(0, v, n)
    t[g.random(n) < 0.1] = v - 1
    t[g.random(n) < 0.1] = 0
    H = synth.round_storage(g.standard_normal((n, c)) + 6 * g.random((n, 1)) * W[t] / max(size, 1e-9), dtype)
    out = g.random(n) < ignored
    t[out] = g.choice([-1, -100, v, v + 7, -2 ** 31, 2 ** 31 - 1], out.sum())
    dloss = np.float32(g.standard_normal(n) / n).astype(np.float64)
    return dict(H=H, W=W, t=t, dloss=dloss, scale=scale)


def logit_error(c, dtype):
    C = c["H"].shape[1]
    mag = c["scale"] * (np.abs(c["H"]) @ np.abs(c["W"]).T)
    terms = 6 if dtype == F32 else 1
    return (terms * (C / 16 + 2) + 64 + (3 if dtype == F32 else 0)) * U * mag


def check(name, got, want, bound):
    got = host(got)
    err = np.abs(got - want)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    log(f"    {name}: worst error {worst:.3f} of its bound, "
        f"relative {np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300):.2e}")
    assert np.isfinite(got).all() and worst <= 1.0, name


def check_forward(c, dtype, loss, lse):
    V = c["W"].shape[0]
    wl, we, a = O.forward(c["H"], c["W"], c["t"], c["scale"])
    top = np.abs(a).max(1)
    # every logit's error, the exponentials' arguments and results, their sum, its logarithm and place
    bound = logit_error(c, dtype).max(1) + U * (4 * top + 128 + V / 2048 + 4 + 4 * np.abs(we))
    check("lse", lse, we, bound)
    check("loss", loss, wl, 2 * bound + U * 4 * top)
    assert not host(loss)[(c["t"] < 0) | (c["t"] >= V)].any()


def check_backward(c, dtype, lse, dH, dW, need=(True, True)):
    """lse: the device's own."""
    n, V, C = c["H"].shape[0], c["W"].shape[0], c["H"].shape[1]
    lse = host(lse)
    wh, ww, d, p = O.backward(c["H"], c["W"], c["t"], lse, c["dloss"], c["scale"])
    a = c["scale"] * (c["H"] @ c["W"].T)
    w = np.abs(c["scale"] * c["dloss"])[:, None]
    # p: the logit, its argument, the exponential; then one subtraction, one product
    live = np.zeros((n, 1))
    live[O.live_rows(c["t"], V)] = 1
    e = w * p * (logit_error(c, dtype) + U * (4 * np.abs(a) + 4 * np.abs(lse)[:, None] + 4)) + 3 * U * np.abs(d)
    e = e + (w + 1) * TINY
    if dtype == BF16:
        e = e + 2.0 ** -8 * (np.abs(d) + e)
    e = e * live
    terms = 6 if dtype == F32 else 1
    pieces = 8
    if need[0]:
        aW, ad = np.abs(c["W"]), np.abs(d) + e
        bound = e @ aW + (terms * (V / 16 + 2) + 64 + pieces) * U * (ad @ aW) + HALF[dtype] * np.abs(wh) * (1 + 2.0 ** -6)
        check("dH", dH, wh, bound + HALF[dtype] * (e @ aW) + TINY)
        assert not host(dH)[live[:, 0] == 0].any()
    if need[1]:
        aH, ad = np.abs(c["H"]), np.abs(d) + e
        bound = e.T @ aH + (terms * (n / 16 + 6) + 64) * U * (ad.T @ aH) + HALF[dtype] * np.abs(ww) * (1 + 2.0 ** -6)
        check("dW", dW, ww, bound + HALF[dtype] * (e.T @ aH) + TINY)


def run(c, dtype, **kw):
    from input_adaptive_rank_amd import vocab_loss as L
    H, W, t = put(c["H"], dtype), put(c["W"], dtype), ints(c["t"])
    loss, lse = L.vocab_loss_forward(H, W, t, c["scale"])
    dH, dW = L.vocab_loss_backward(H, W, t, lse, floats(c["dloss"]), c["scale"], **kw)
    return loss, lse, dH, dW


SIZES = [(4, 1032, 5003), (40, 520, 3001), (100, 264, 2053), (1, 8, 1), (1, 64, 130), (2, 8, 63), (3, 72, 64), (17, 264, 65), (63, 128, 1000), (64, 64, 257), (65, 136, 129),
         (128, 520, 300), (129, 64, 5003), (257, 264, 1024), (700, 72, 515), (1031, 128, 2053)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n,c,v", SIZES, ids=lambda x: str(x))
def test_forward_and_backward_match_the_oracle(n, c, v, dtype):
    case = make(n, c, v, dtype, seed=n + c + v, scale=0.5 if n % 2 else 1.0)
    log(f"  {n} rows of {c}, vocabulary {v}")
    loss, lse, dH, dW = run(case, dtype)
    check_forward(case, dtype, loss, lse)
    check_backward(case, dtype, lse, dH, dW)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n,v", [(640, 32000), (620, 31000), (1270, 9001)])
def test_forward_of_many_columns(n, v, dtype):
    case = make(n, 136, v, dtype, seed=n)
    from input_adaptive_rank_amd import vocab_loss as L
    loss, lse = L.vocab_loss_forward(put(case["H"], dtype), put(case["W"], dtype), ints(case["t"]))
    check_forward(case, dtype, loss, lse)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
def test_large_and_small_logits(dtype):
    """Logits in the thousands (the exponentials of most underflow) and none
    above 1e-6: the maximum is taken off, the loss keeps its digits."""
    for size, seed in ((1000.0, 1), (1e-6, 2)):
        case = make(70, 64, 515, dtype, seed=seed, size=size)
        loss, lse, dH, dW = run(case, dtype)
        check_forward(case, dtype, loss, lse)
        check_backward(case, dtype, lse, dH, dW)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n,v", [(300, 1100), (1031, 700), (2500, 130), (9001, 65)])
@pytest.mark.parametrize("ignored", [0.0, 0.4, 0.7, 0.9, 0.99])
def test_any_number_of_rows_that_count(ignored, n, v, dtype):
    """How tiles are split is worked out from the rows found on the device."""
    case = make(n, 520, v, dtype, seed=int(100 * ignored), ignored=ignored)
    loss, lse, dH, dW = run(case, dtype)
    check_backward(case, dtype, lse, dH, dW)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n", [9, 300])
def test_ignored_rows_count_for_nothing(n, dtype):
    """Whatever an ignored row's H, lse and dloss hold, every other result has
    the same bits as without it."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(n, 72, 515, dtype, seed=3, ignored=0.4)
    out = torch.from_numpy((c["t"] < 0) | (c["t"] >= 515)).cuda()
    assert bool(out.any()) and not bool(out.all())
    H, W, t, g = put(c["H"], dtype), put(c["W"], dtype), ints(c["t"]), floats(c["dloss"])
    loss, lse = L.vocab_loss_forward(H, W, t)
    want = L.vocab_loss_backward(H, W, t, lse, g)
    for value in (float("nan"), float("inf")):
        H2, lse2, g2 = H.clone(), lse.clone(), g.clone()
        H2[out, 5], lse2[out], g2[out] = value, value, value
        loss2, _ = L.vocab_loss_forward(H2, W, t)
        assert torch.equal(loss2, loss) and not bool(loss2[out].any())
        got = L.vocab_loss_backward(H2, W, t, lse2, g2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not bool(got[0][out].any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
def test_no_row_that_counts(dtype):
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(130, 72, 515, dtype, seed=4)
    H, W = put(c["H"], dtype), put(c["W"], dtype)
    t, g = ints(np.full(130, -1)), floats(np.full(130, np.nan))
    loss, lse = L.vocab_loss_forward(H, W, t)
    assert not bool(loss.any()) and bool(torch.isfinite(lse).all())
    dH, dW = torch.full_like(H, 7), torch.full_like(W, 7)
    L.vocab_loss_backward(H, W, t, lse, g, dH=dH, dW=dW)
    assert not bool(dH.any()) and not bool(dW.any())
    # and none at all
    none = H[:0]
    assert [x.shape for x in L.vocab_loss_forward(none, W, t[:0])] == [(0,), (0,)]
    dW.fill_(7)
    dH, dW = L.vocab_loss_backward(none, W, t[:0], lse[:0], g[:0], dW=dW)
    assert dH.shape == (0, 72) and not bool(dW.any())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
def test_bad_rows_stay_in_their_row(dtype):
    """A NaN or an infinity in a row that counts: its own results alone are not
    finite, but for dW, whose sum it enters; other rows keep their bits."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(300, 72, 515, dtype, seed=5, ignored=0.0)
    H, W, t, g = put(c["H"], dtype), put(c["W"], dtype), ints(c["t"]), floats(c["dloss"])
    loss, lse = L.vocab_loss_forward(H, W, t)
    want = L.vocab_loss_backward(H, W, t, lse, g, need_dw=False)[0]
    keep = torch.arange(300, device="cuda") != 150
    for value in (float("nan"), float("inf")):
        H2 = H.clone()
        H2[150, 3] = value
        loss2, lse2 = L.vocab_loss_forward(H2, W, t)
        assert torch.equal(loss2[keep], loss[keep]) and torch.equal(lse2[keep], lse[keep])
        assert not bool(torch.isfinite(loss2[150]))
        got = L.vocab_loss_backward(H2, W, t, lse2, g, need_dw=False)[0]
        assert torch.equal(got[keep], want[keep]) and not bool(torch.isfinite(got[150]).all())


@pytest.mark.parametrize("n,c,v", [(8, 8192, 10816), (65, 8192, 10816), (130, 8192, 10816), (400, 32768, 2624),
                                   (520, 32768, 2624)])
def test_a_last_piece_stays_within_the_workspace(n, c, v):
    """fp32 weights are taken in pieces; of these two the last has fewer tiles, split
    into more parts than the first's."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    gen = torch.Generator(device="cuda").manual_seed(n)
    H, W = (torch.randn(s, generator=gen, device="cuda") / c ** 0.5 for s in ((n, c), (v, c)))
    t = torch.randint(0, v, (n,), generator=gen, device="cuda", dtype=torch.int32)
    size = L.vocab_loss_workspace_size(n, c, v, F32)
    ws = torch.full((size + (1 << 23),), 90, dtype=torch.uint8, device="cuda")
    loss, lse = L.vocab_loss_forward(H, W, t, workspace=ws)
    assert bool((ws[size:] == 90).all())
    a = H.double() @ W.double().t()
    want = torch.logsumexp(a, 1)
    # logits of c products in six terms; the bounds of check_forward
    mag = (H.double().abs() @ W.double().abs().t()).amax(1)
    bound = (6 * (c / 16 + 2) + 67) * U * mag + U * (4 * a.abs().amax(1) + 132 + v / 2048 + 4 * want.abs())
    assert bool(((lse - want).abs() <= bound).all())
    assert bool(((loss - (want - a.gather(1, t.long()[:, None])[:, 0])).abs() <= 2 * bound + U * 4 * a.abs().amax(1)).all())


@pytest.mark.parametrize("weight", [1.0, 1 + 2.0 ** -8, 1 / 3279, 3e-5])
def test_equal_weights_cost_no_rounding(weight):
    """Two words and rows of zeros: every probability is 1/2 and d an exact half
    of the weight, so that a gradient is rounded once, as it is stored.  Rounded
    with its weight, d would be off by as much again, in every row alike."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    n, c = 96, 72
    gen = torch.Generator(device="cuda").manual_seed(20)
    W = torch.randn((2, c), generator=gen, device="cuda").bfloat16()
    t = (torch.arange(n, device="cuda") % 3 - 1).int()   # none, the first, the second
    H, g = torch.zeros((n, c), dtype=torch.bfloat16, device="cuda"), torch.full((n,), weight, device="cuda")
    lse = L.vocab_loss_forward(H, W, t)[1]
    dH, dW = L.vocab_loss_backward(H, W, t, lse, g)
    half = 0.5 * g.double()[0] * (W[1] - W[0].double())
    want = torch.stack([half * 0, half, -half])[(t.long() + 1)]
    assert bool(((dH.double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -12) * want.abs()).all())
    assert not bool(dW.any())


def test_a_word_that_is_masked_by_its_weights():
    """Rows of W of the type's lowest value give logits of -inf or of its
    size: such words have no probability, and the others keep theirs."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(70, 64, 300, F32, seed=6, ignored=0.0)
    H, W = torch.from_numpy(np.abs(c["H"])).float().cuda().bfloat16(), put(c["W"], BF16)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[0, 63, 64, 130, 299]] = False
    t = torch.nonzero(keep)[:70, 0].int()
    loss, lse = L.vocab_loss_forward(H, W[keep].contiguous(), torch.arange(70, device="cuda", dtype=torch.int32))
    W2 = W.clone()
    W2[~keep] = torch.finfo(torch.bfloat16).min
    loss2, lse2 = L.vocab_loss_forward(H, W2, t)
    # the same sums in another order
    assert float((lse2 - lse).abs().max()) <= 300 * U * float(lse.abs().max() + 1)
    assert float((loss2 - loss).abs().max()) <= 300 * U * float(lse.abs().max() + 10)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n", [1, 40, 400])
def test_column_ranges_and_what_lies_beside_them(n, dtype):
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(n, 72, 515, dtype, seed=7)
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    H, W, t, g = put(c["H"], dtype), put(c["W"], dtype), ints(c["t"]), floats(c["dloss"])
    loss, lse = L.vocab_loss_forward(H, W, t)
    want = L.vocab_loss_backward(H, W, t, lse, g)
    wide = torch.full((n + 2, 200), 3.0, dtype=td, device="cuda")
    h, dh = wide[1:n + 1, 16:88], wide[1:n + 1, 96:168]
    h.copy_(H)
    got = L.vocab_loss_forward(h, W, t)
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
    got = L.vocab_loss_backward(h, W, t, lse, g, dH=dh)
    assert got[0].data_ptr() == dh.data_ptr() and torch.equal(dh, want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(h, H)
    h.fill_(3.0)
    dh.fill_(3.0)
    assert bool((wide == 3.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
def test_one_gradient_alone_has_the_same_bits(dtype):
    import torch
    c = make(300, 136, 1500, dtype, seed=8)
    both, dh, dw = run(c, dtype)[2:], run(c, dtype, need_dw=False)[2:], run(c, dtype, need_dh=False)[2:]
    assert dh[1] is None and dw[0] is None
    assert torch.equal(dh[0], both[0]) and torch.equal(dw[1], both[1])


@pytest.mark.parametrize("dtype,n,c,v", [(BF16, 4099, 128, 33000), (BF16, 2048, 64, 50257), (F32, 1500, 64, 48000),
                                         (BF16, 8, 512, 32000)])
def test_a_large_vocabulary_in_pieces(dtype, n, c, v):
    """Against float64 on the device: several pieces, tiles of a last round
    split along the reduction, rows left out."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(9)
    W = (torch.randn((v, c), generator=gen, device="cuda") / c ** 0.5).to(td)
    t = torch.randint(0, v, (n,), generator=gen, device="cuda")
    H = (torch.randn((n, c), generator=gen, device="cuda") + 6 * W[t].float()).to(td)
    t[torch.rand(n, generator=gen, device="cuda") < 0.3] = -1
    g = (torch.rand(n, generator=gen, device="cuda") / n)
    loss, lse = L.vocab_loss_forward(H, W, t.int())
    dH, dW = L.vocab_loss_backward(H, W, t.int(), lse, g)
    live = torch.nonzero(t >= 0)[:, 0]
    Hd, Wd = H.double(), W.double()
    a = Hd @ Wd.t()
    mag = Hd.abs() @ Wd.abs().t()
    terms = 6 if dtype == F32 else 1
    ea = (terms * (c / 16 + 2) + 67) * U * mag.amax(1)
    we = torch.logsumexp(a, 1)
    bound = ea + U * (4 * a.abs().amax(1) + 132 + v / 2048 + 4 * we.abs())
    assert bool(((lse.double() - we).abs() <= bound).all())
    wl = torch.zeros_like(we)
    wl[live] = we[live] - a[live, t[live]]
    assert bool(((loss.double() - wl).abs() <= 2 * bound + U * 4 * a.abs().amax(1)).all())
    p = torch.exp(a[live] - lse[live].double()[:, None])
    d = p.clone()
    d[torch.arange(len(live), device="cuda"), t[live]] -= 1
    d *= g[live].double()[:, None]
    e = g[live].double()[:, None] * p * (ea[live] + U * (4 * a[live].abs().amax(1) + 4 * lse[live].abs().double() + 4))[:, None]
    e += 3 * U * d.abs()
    if dtype == BF16:
        e += 2.0 ** -8 * (d.abs() + e)
    ad = d.abs() + e
    for name, got, want, err, mags, K in (
            ("dH", dH[live], d @ Wd, e @ Wd.abs(), ad @ Wd.abs(), v),
            ("dW", dW, d.t() @ Hd[live], e.t() @ Hd[live].abs(), ad.t() @ Hd[live].abs(), len(live))):
        lim = err + (terms * (K / 16 + 6) + 72) * U * mags + HALF[dtype] * (want.abs() * (1 + 2.0 ** -6) + err)
        worst = float(((got.double() - want).abs() / lim.clamp(min=1e-300)).max())
        rel = float((got.double() - want).norm() / want.norm())
        log(f"    {name}: worst error {worst:.3f} of its bound, relative {rel:.2e}")
        assert worst <= 1.0, name
    assert not bool(dH[t < 0].any())


def test_gradients_match_differences():
    """The device's fp32 gradients along random directions against fourth
    order differences of the float64 forward.  By the tests above an element is
    off by some hundred U of the magnitudes that it is a sum of: along a direction at
    most 2^-14 of sum |gradient direction|."""
    c = make(23, 72, 130, F32, seed=12, scale=0.7)
    _, lse, dH, dW = run(c, F32)
    rng = np.random.default_rng(13)
    for k, dev in (("H", host(dH)), ("W", host(dW))):
        step = rng.standard_normal(c[k].shape)

        def at(x):
            m = dict(c, **{k: c[k] + x * step})
            return (O.forward(m["H"], m["W"], c["t"], c["scale"])[0] * c["dloss"]).sum()

        h = 1e-3
        slope = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
        log(f"    d{k}: difference {slope:.8f}, gradient {(dev * step).sum():.8f}")
        assert abs(slope - (dev * step).sum()) <= 2.0 ** -14 * np.abs(dev * step).sum()


@pytest.mark.parametrize("dtype,n,c,v", [(BF16, 300, 136, 3000), (BF16, 9001, 72, 515), (F32, 40, 136, 3000),
                                         (F32, 900, 520, 1500)])
def test_same_bits_on_every_call_and_in_graph_replays(dtype, n, c, v):
    """Two captured graphs with their own workspaces; targets and rows change
    between replays, and with them how many rows count."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    c = make(n, c, v, dtype, seed=14)
    H, W, t, g, keep = put(c["H"], dtype), put(c["W"], dtype), ints(c["t"]), floats(c["dloss"]), {}

    def step():
        keep["f"] = L.vocab_loss_forward(H, W, t)
        keep["b"] = L.vocab_loss_backward(H, W, t, keep["f"][1], g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((graph, dict(keep)))
    for rep in range(4):
        H.mul_(0.75)
        t.copy_(torch.randint(-1 - v // 3 * rep, v, (n,), device="cuda", dtype=torch.int32))
        f = L.vocab_loss_forward(H, W, t)
        want = f + L.vocab_loss_backward(H, W, t, f[1], g)
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, held in graphs:
            assert all(torch.equal(p, q) for p, q in zip(want, held["f"] + held["b"])), rep


def test_another_stream_leaves_memory_that_is_still_in_use():
    """Blocks of the sizes that a call allocates, just freed on the current
    stream with their readers still to run there, are not written by a call on
    another stream."""
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    n, c, v = 512, 256, 4000
    case = make(n, c, v, BF16, seed=15)
    H, W, t, g = put(case["H"], BF16), put(case["W"], BF16), ints(case["t"]), floats(case["dloss"])
    loss, lse = L.vocab_loss_forward(H, W, t)
    want = L.vocab_loss_backward(H, W, t, lse, g)
    s, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    sizes = (4 * n, 4 * n, 2 * n * c, 2 * v * c, L.vocab_loss_workspace_size(n, c, v, BF16),
             L.vocab_loss_workspace_size(n, c, v, BF16, True))
    old = [torch.full((size,), 3, dtype=torch.uint8, device="cuda") for size in sizes]
    kept = [torch.empty_like(x) for x in old]
    torch.cuda.synchronize()
    for _ in range(50):   # some 70 ms on the current stream, then the readers
        torch.mm(a, a, out=b)
    for x, k in zip(old, kept):
        torch.add(x, 1, out=k)
    del x, old
    got_loss, got_lse = L.vocab_loss_forward(H, W, t, stream=s)
    got = L.vocab_loss_backward(H, W, t, got_lse, g, stream=s)
    torch.cuda.synchronize()
    assert all(bool((k == 4).all()) for k in kept)
    assert torch.equal(got_loss, loss) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def refusals():
    import torch
    from input_adaptive_rank_amd import vocab_loss as L
    bf = torch.bfloat16
    H, W = torch.zeros((6, 64), dtype=bf, device="cuda"), torch.zeros((30, 64), dtype=bf, device="cuda")
    t, f = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(6, device="cuda")
    small = torch.zeros(16, dtype=torch.uint8, device="cuda")
    fwd = lambda H=H, W=W, t=t, **kw: L.vocab_loss_forward(H, W, t, **kw)  # noqa: E731
    bwd = lambda lse=f, g=f, **kw: L.vocab_loss_backward(H, W, t, lse, g, **kw)  # noqa: E731
    return {
        "width": (lambda: fwd(W=torch.zeros((30, 72), dtype=bf, device="cuda")), "W must have shape"),
        "odd width": (lambda: fwd(H=H[:, :60], W=W[:, :60].contiguous()), "multiple of 8"),
        "no words": (lambda: fwd(W=W[:0]), "vocabulary not empty"),
        "weight type": (lambda: fwd(W=W.float()), "W must be torch.bfloat16"),
        "strided weights": (lambda: fwd(W=torch.zeros((30, 72), dtype=bf, device="cuda")[:, :64]), "contiguous"),
        "host weights": (lambda: fwd(W=W.cpu()), "W is on cpu"),
        "long targets": (lambda: fwd(t=t.long()), "targets must be torch.int32"),
        "few targets": (lambda: fwd(t=t[:5]), "targets must have shape"),
        "scale zero": (lambda: fwd(logit_scale=0.0), "positive and finite"),
        "scale infinite": (lambda: fwd(logit_scale=float("inf")), "positive and finite"),
        "scale NaN": (lambda: fwd(logit_scale=float("nan")), "positive and finite"),
        "broadcast rows": (lambda: fwd(H=H[:1].expand(6, 64)), "rows must be dense"),
        "loss shape": (lambda: fwd(loss=f[:5]), "loss must have shape"),
        "loss is lse": (lambda: fwd(loss=f, lse=f), "overlap"),
        "loss type": (lambda: fwd(loss=f.bfloat16()), "loss must be torch.float32"),
        "small workspace": (lambda: fwd(workspace=small), "needs"),
        "nothing wanted": (lambda: bwd(need_dh=False, need_dw=False), "nothing is asked for"),
        "no lse": (lambda: bwd(lse=None), "must be tensors"),
        "dloss shape": (lambda: bwd(g=f[:3]), "dloss must have shape"),
        "dH is H": (lambda: bwd(dH=H), "overlap"),
        "dW is W": (lambda: bwd(dW=W), "overlap"),
        "dW shape": (lambda: bwd(dW=W[:29]), "dW must have shape"),
        "dH type": (lambda: bwd(dH=H.float()), "dH must be torch.bfloat16"),
        "small backward workspace": (lambda: bwd(workspace=small), "needs"),
    }


REFUSALS = ["width", "odd width", "no words", "weight type", "strided weights", "host weights", "long targets", "few targets",
            "scale zero", "scale infinite", "scale NaN", "broadcast rows", "loss shape", "loss is lse", "loss type",
            "small workspace", "nothing wanted", "no lse", "dloss shape", "dH is H", "dW is W", "dW shape", "dH type",
            "small backward workspace"]


@pytest.mark.parametrize("name", REFUSALS)
def test_refuses(name):
    call, msg = refusals()[name]
    with pytest.raises(ValueError, match=msg):
        call()
