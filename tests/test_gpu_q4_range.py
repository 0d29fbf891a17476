"""The 4-bit projection at the ends of its range: loud columns, fp32 values next to
the largest, weights and rows past 2^31 bytes.  References in float64."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import q4_oracle as O

from test_gpu_q4 import check, forward_case, host, make, pack, put, sums

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U, HALF = 2.0 ** -24, {F32: 2.0 ** -24, BF16: 2.0 ** -8}
IDS = {F32: "fp32", BF16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,c1,c2", [(1, 264, 72), (5, 2056, 136), (48, 520, 264), (197, 1024, 520)])
def test_a_loud_column_of_no_weight_drowns_nothing(n, c1, c2, group, dtype):
    """A column of 2^19 that every weight meets with 0, beside small whole numbers.
    A few bf16 rows add x (16 + code) and take (16 + zero) sum x off: all of it whole
    numbers up to 31 x 2^19 + 31 x 8 x 127 < 2^24, so nothing is rounded before the
    result is stored.  The scale is 1, a group's sum at most 15 x 8 x 127."""
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, c1, c2, group, True, dtype, seed=31)
    g = np.random.default_rng(32)
    c["scale"] = np.ones_like(c["scale"])
    c["X"] = g.integers(-8, 9, (n, c1)).astype(np.float64)
    for k in range(3, c1, group):   # one in each group
        c["X"][:, k] = 2.0 ** 19 * g.choice([-1, 1], n)
        c["codes"][:, k] = c["zero"][:, k // group]
    W = O.weight(c["codes"], c["scale"], c["zero"], group)
    want = c["X"] @ W.T
    assert np.abs(want).max() < 2 ** 24 and Q.q4_workspace_size(c1, c2, n, dtype) == 0
    assert np.array_equal(host(Q.q4_forward(put(c["X"], dtype), pack(c))), synth.round_storage(want, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n,c1,c2", [(1, 264, 72), (48, 520, 264), (197, 1024, 520)])
def test_few_rows_of_the_largest_values(n, c1, c2, group, dtype):
    """Whole numbers up to 8 times 2^111: a group's sums of x (16 + code) reach 31 x 8 x
    128 x 2^111 < 2^126, without a rounding; the scale brings them back."""
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, c1, c2, group, True, dtype, seed=39)
    c["scale"][:] = 2.0 ** -40
    c["X"] = np.random.default_rng(40).integers(-8, 9, (n, c1)) * 2.0 ** 111
    c["X"][0] = 2.0 ** 114
    want = c["X"] @ O.weight(c["codes"], c["scale"], c["zero"], group).T
    assert Q.q4_workspace_size(c1, c2, n, dtype) == 0
    assert np.array_equal(host(Q.q4_forward(put(c["X"], dtype), pack(c))), synth.round_storage(want, dtype))


@pytest.mark.parametrize("n,c1,c2", [(900, 1024, 4096), (600, 264, 6000)])
def test_values_next_to_the_largest(n, c1, c2):
    """Many fp32 rows with entries at the type's ends by small weights: the results
    are numbers, forward and backward."""
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, c1, c2, 64, True, F32, seed=33, spread=2.0 ** -20)
    assert Q.q4_workspace_size(c1, c2, n, F32) > 0
    ends = np.array([3.4028234663852886e38, -3.4028234663852886e38, 3.3961775292304601e38, 3.4e38])
    g = np.random.default_rng(34)
    c["X"][:, 9] = synth.round_f32(g.choice(ends, n))
    c["dY"][:, 17] = synth.round_f32(g.choice(ends, n))
    forward_case(c, F32)
    dX = Q.q4_backward(put(c["dY"], F32), pack(c))
    want, mag = O.backward(c["dY"], c["W"])
    check("dX", dX, want, (sums(c2, 5) + 3) * U * mag + HALF[F32] * np.abs(want) * (1 + 2.0 ** -7))


def test_weights_next_to_the_largest():
    """Scales of 73 x 2^119, whose sevenfold is 511 x 2^119: a number in fp32, an
    infinity if it is rounded to bf16."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(900, 1024, 4096, 64, False, F32, seed=35)
    c["codes"] = np.clip(c["codes"], 1, 15)
    c["scale"] = np.full_like(c["scale"], 73 * 2.0 ** 119)
    c["X"], c["dY"] = (synth.round_f32(c[k] * 2.0 ** -100) for k in ("X", "dY"))
    c["W"] = O.weight(c["codes"], c["scale"], None, 64)
    assert np.array_equal(Q.q4_dense(pack(c), torch.float32).double().cpu().numpy(), c["W"])
    assert Q.q4_workspace_size(1024, 4096, 900, F32) > 0
    forward_case(c, F32, bias=False)
    want, mag = O.backward(c["dY"], c["W"])
    check("dX", Q.q4_backward(put(c["dY"], F32), pack(c)), want,
          (sums(4096, 5) + 3) * U * mag + HALF[F32] * np.abs(want) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("n,c1,c2,ld", [(2200, 72, 264, 1 << 20), (40, 72, 264, 1 << 20), (1 << 18, 64, 4104, 4104)])
def test_rows_beyond_two_gibibytes(n, c1, c2, ld):
    """Rows and results whose last bytes lie past 2^31 (2200 rows of 2^21 bytes: past
    2^32), in bf16."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(1, c1, c2, 64, True, BF16, seed=36)
    w, W = pack(c), torch.from_numpy(synth.round_bf16(c["W"])).cuda()
    few = Q.q4_workspace_size(c1, c2, n, BF16) == 0
    gen = torch.Generator(device="cuda").manual_seed(37)
    wide, out = (torch.empty((n, ld), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step = torch.from_numpy(np.repeat(c["scale"], 64, axis=1)[:, :c1]).cuda()
    exact = torch.from_numpy(c["W"]).cuda()
    for back in (False, True):
        cin, cout = (c2, c1) if back else (c1, c2)
        x, y = wide[:, ld - cin:], out[:, ld - cout:]
        x.copy_(torch.randn((n, cin), generator=gen, device="cuda"))
        if back:
            Q.q4_backward(x, w, dX=y)
        else:
            Q.q4_forward(x, w, out=y)
        m = W if back else (exact if few else W).t().contiguous()
        terms = 0.0 if back or not few else 62.0 * step.t()
        for at in range(0, n, 1 << 16):
            rows = slice(at, at + (1 << 16))
            want, mag = x[rows].double() @ m, x[rows].double().abs() @ (m.abs() + terms)
            bound = (sums(cin, 1) + 3) * U * mag + HALF[BF16] * want.abs() * (1 + 2.0 ** -7)
            assert bool(((y[rows].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("n", [3, 1500])
def test_weights_beyond_two_gibibytes(n):
    """A weight of 65544 x 65536: its codes pass 2^31 bytes, its bf16 form 2^33.
    Compared at the last columns and some others."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c1, c2, group = 65544, 65536, 128
    groups = -(-c1 // group)
    gen = torch.Generator(device="cuda").manual_seed(38)
    codes = torch.randint(0, 256, (c2, c1 // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scale = (0.5 + torch.rand((c2, groups), generator=gen, device="cuda")).bfloat16()
    w = Q.q4_pack(codes, scale, group=group)
    X = torch.randn((n, c1), generator=gen, device="cuda").bfloat16()
    at = torch.cat([torch.arange(c2 - 40, c2, device="cuda"), torch.randint(0, c2, (200,), generator=gen, device="cuda")])

    def rows(at):
        q = codes[at]
        v = torch.stack([q & 15, q >> 4], 2).flatten(1).double() - 8
        s = scale[at].double().repeat_interleave(group, 1)[:, :c1]
        return v * s, s

    few = Q.q4_workspace_size(c1, c2, n, BF16) == 0
    assert few == (n == 3)
    W, s = rows(at)
    if not few:
        W = W.bfloat16().double()
    want, mag = X.double() @ W.t().contiguous(), X.double().abs() @ (W.abs() + (62.0 * s if few else 0.0)).t().contiguous()
    bound = (sums(c1, 1) + 3) * U * mag + HALF[BF16] * want.abs() * (1 + 2.0 ** -7)
    got = Q.q4_forward(X, w)[:, at].double()
    assert bool(((got - want).abs() <= bound).all())
    if few:
        return
    # the gradient of rows that are zero but at those columns
    dY = torch.zeros((n, c2), dtype=torch.bfloat16, device="cuda")
    at = torch.unique(at)
    dY[:, at] = torch.randn((n, len(at)), generator=gen, device="cuda").bfloat16()
    W = rows(at)[0].bfloat16().double()
    g = dY[:, at].double()
    want, mag = g @ W, g.abs() @ W.abs()
    bound = (sums(c2, 1) + 3) * U * mag + HALF[BF16] * want.abs() * (1 + 2.0 ** -7)
    assert bool(((Q.q4_backward(dY, w).double() - want).abs() <= bound).all())
