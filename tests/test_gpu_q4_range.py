"""The 4-bit projection at the ends of its range: loud columns, fp32 values next to
the largest.  References in float64."""
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
