"""The 4-bit projection (dyra_q4_*) through the package's entry points, against
the float64 oracle on the same codes.

Bounds are sums of what each step may lose.  U = 2^-24 is a rounding to fp32,
2^-8 one to bf16.  A sum of K products on matrix instructions adds them 16 or 32
at a time and the results one after the other, at most K / 16 + 32 roundings of at most the
sum of the terms' magnitudes; a few hundred partial sums are joined with one
rounding each.  A few rows multiply (128 + code) and take (128 + zero) times the
plain sum off again: their terms are up to 136 + 136 instead of |code - zero|.
fp32 operands are three bf16 terms (exact), of whose products with the weight's
two those below 2^-24 are left out.  Where the library keeps the weight in
bf16 (documented: many rows, bf16) the oracle's is rounded too."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import q4_oracle as O

from gpu_cases import log

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U, HALF = 2.0 ** -24, {F32: 2.0 ** -24, BF16: 2.0 ** -8}
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


def rounded(a, dtype):
    return synth.round_storage(a, dtype)


def make(n, c1, c2, group, zero, dtype, seed, spread=1.0):
    """Codes over their whole range and operands with a few loud columns."""
    g = np.random.default_rng(seed)
    groups = -(-c1 // group)
    c = dict(codes=g.integers(0, 16, (c2, c1)).astype(np.float64), group=group,
             scale=synth.round_bf16((0.5 + g.random((c2, groups))) * 0.1 * spread),
             zero=g.integers(0, 16, (c2, groups)).astype(np.float64) if zero else None)
    loud = np.where(g.random(c1) < 0.02, 8.0, 1.0)
    c["X"] = rounded(g.standard_normal((n, c1)) * loud, dtype)
    c["dY"] = rounded(g.standard_normal((n, c2)), dtype)
    c["bias"] = rounded(g.standard_normal(c2), dtype)
    c["W"] = O.weight(c["codes"], c["scale"], c["zero"], group)
    return c


def pack(c, stream=None):
    import torch
    from input_adaptive_rank_amd import q4 as Q
    codes = c["codes"].astype(np.uint8)
    u8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return Q.q4_pack(u8(codes[:, 0::2] | codes[:, 1::2] << 4), put(c["scale"], BF16),
                     None if c["zero"] is None else u8(c["zero"].astype(np.uint8)), group=c["group"], stream=stream)


def sums(K, terms):
    """Roundings of a sum of K products in `terms` plane pairs, and of its join."""
    return terms * (K / 16 + 2) + 64


def check(name, got, want, bound):
    err = np.abs(host(got) - want)
    worst = float((err / bound).max())
    log(f"    {name}: worst error {worst:.3f} of its bound, "
        f"relative {np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300):.2e}")
    assert np.isfinite(host(got)).all() and worst <= 1.0, name


def forward_case(c, dtype, bias=True, X=None, out=None):
    from input_adaptive_rank_amd import q4 as Q
    w = pack(c)
    n, c1 = c["X"].shape
    x = put(c["X"], dtype) if X is None else X
    b = put(c["bias"], dtype) if bias else None
    Y = Q.q4_forward(x, w, bias=b, out=out)
    few = Q.q4_workspace_size(c1, c["W"].shape[0], n, dtype) == 0
    W = c["W"] if few or dtype == F32 else synth.round_bf16(c["W"])
    want, mag = O.forward(c["X"], W, c["bias"] if bias else None)
    if few and dtype == BF16:
        # the terms as they are added
        step = np.repeat(c["scale"], c["group"], axis=1)[:, :c1]
        mag = mag + np.abs(c["X"]) @ (272.0 * step).T
    bound = sums(c1, 1 if dtype == BF16 else 5) * U * mag + HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7)
    if dtype == F32:
        bound = bound + 3 * U * mag   # plane pairs left out
    check(f"Y ({'few' if few else 'many'} rows)", Y, want, bound)
    return Y


SIZES = [(1, 8, 8), (1, 4096, 520), (2, 72, 24), (7, 136, 16), (15, 264, 200), (16, 128, 128), (17, 520, 1032),
         (33, 1032, 72), (47, 392, 4104), (49, 264, 520), (64, 1024, 264), (65, 200, 8), (97, 2056, 776),
         (130, 264, 136), (300, 1024, 1024), (700, 520, 2048)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,c1,c2", SIZES, ids=lambda v: str(v))
def test_forward_and_backward_match_the_oracle(n, c1, c2, group, dtype):
    from input_adaptive_rank_amd import q4 as Q
    zero = bool((n + group // 32) & 1)
    c = make(n, c1, c2, group, zero, dtype, seed=n + c1 + c2 + group)
    log(f"  {n} rows, {c1} -> {c2}, group {group}, zero points {zero}")
    forward_case(c, dtype, bias=not zero)
    dX = Q.q4_backward(put(c["dY"], dtype), pack(c))
    want, mag = O.backward(c["dY"], c["W"] if dtype == F32 else synth.round_bf16(c["W"]))
    check("dX", dX, want, (sums(c2, 1 if dtype == BF16 else 5) + (3 if dtype == F32 else 0)) * U * mag +
          HALF[dtype] * np.abs(want) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("n,c1,c2,dtype", [(5003, 512, 1024, BF16), (2048, 4096, 1024, BF16), (4099, 1024, 4096, BF16),
                                           (2100, 1024, 1024, F32), (600, 12288, 256, BF16), (5003, 264, 4096, BF16),
                                           (5003, 4096, 264, BF16), (2900, 264, 6000, F32)])
def test_many_rows_whose_last_round_is_split(n, c1, c2, dtype):
    """Against float64 products on the device, forward and backward."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(1, c1, c2, 128, True, dtype, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    X = torch.randn((n, c1), generator=gen, device="cuda").to(td)
    dY = torch.randn((n, c2), generator=gen, device="cuda").to(td)
    w = pack(c)
    exact = torch.from_numpy(c["W"]).cuda()
    kept = exact if dtype == F32 else torch.from_numpy(synth.round_bf16(c["W"])).cuda()
    few = Q.q4_workspace_size(c1, c2, n, dtype) == 0
    step = torch.from_numpy(np.repeat(c["scale"], 128, axis=1)[:, :c1]).cuda()
    fW = exact if few else kept
    for got, x, m, K, terms in ((Q.q4_forward(X, w), X, fW.t().contiguous(), c1, 272.0 * step.t() if few else 0.0),
                                (Q.q4_backward(dY, w), dY, kept, c2, 0.0)):
        want, mag = x.double() @ m, x.double().abs() @ (m.abs() + terms)
        bound = (sums(K, 1 if dtype == BF16 else 5) + 3) * U * mag + HALF[dtype] * want.abs() * (1 + 2.0 ** -7)
        worst = float(((got.double() - want).abs() / bound).max())
        log(f"    worst error {worst:.3f} of its bound")
        assert worst <= 1.0


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("zero", [False, True], ids=["symmetric", "zero_points"])
@pytest.mark.parametrize("group,c1,c2", [(32, 8, 8), (32, 72, 24), (64, 264, 40), (128, 264, 520), (128, 1024, 8)])
def test_codes_scales_and_dense_forms(group, c1, c2, zero, dtype):
    """Codes, scales and zero points equal the oracle's; the dense form is the
    formula's, exact in fp32 and rounded once in bf16.  Among the rows: zeros,
    one sign only, ties between two codes, tiny and large values."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    g = np.random.default_rng(c1 + c2)
    W = g.standard_normal((c2, c1))
    W[0] = 0.0
    W[1] = np.abs(W[1])
    W[2] = -np.abs(W[2])
    W[3] = np.clip(np.rint(W[3] * 4), -14, 14) / 2 + 0.0   # scale 1 where 7 occurs: halves are ties
    W[3, ::group] = 7.0
    W[4] *= 1e-30
    W[5] *= 1e30
    W = rounded(W, dtype)
    codes, scale, zp = Q.q4_quantise(put(W, dtype), group, zero_points=zero)
    want = O.quantise(W, group, zero)
    assert np.array_equal(host(scale), want[1])
    assert (zp is None) == (not zero) and (zp is None or np.array_equal(host(zp), want[2]))
    assert np.array_equal(O.unpack(codes.cpu().numpy()), want[0])
    w = Q.q4_pack(codes, scale, zp, group)
    assert w.shape == (c2, c1)
    dense = O.weight(want[0], want[1], want[2], group)
    assert np.array_equal(Q.q4_dense(w, torch.float32).double().cpu().numpy(), dense)
    assert np.array_equal(host(Q.q4_dense(w)), synth.round_bf16(dense))


def test_no_rows():
    import torch
    from input_adaptive_rank_amd import q4 as Q
    w = pack(make(1, 72, 24, 32, False, BF16, seed=0))
    assert Q.q4_forward(torch.empty((0, 72), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 24)
    assert Q.q4_backward(torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 72)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n", [1, 5, 40, 900])
def test_column_ranges_and_what_lies_beside_them(n, dtype):
    """Operands and results as column ranges of wider matrices: the same bits,
    and nothing beside the result is written."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c1, c2 = 264, 520
    c = make(n, c1, c2, 64, True, dtype, seed=7)
    w, td = pack(c), torch.bfloat16 if dtype == BF16 else torch.float32
    X, dY = put(c["X"], dtype), put(c["dY"], dtype)
    want, gwant = Q.q4_forward(X, w), Q.q4_backward(dY, w)
    wide = torch.full((n + 2, c1 + c2 + 64), 3.0, dtype=td, device="cuda")
    x, y = wide[1:n + 1, 16:16 + c1], wide[1:n + 1, 24 + c1:24 + c1 + c2]
    x.copy_(X)
    assert Q.q4_forward(x, w, out=y).data_ptr() == y.data_ptr()
    assert torch.equal(y, want) and torch.equal(x, X)
    wide[1:n + 1, 16:16 + c1] = 3.0
    wide[1:n + 1, 24 + c1:24 + c1 + c2] = 3.0
    assert bool((wide == 3.0).all())
    y.copy_(dY)
    Q.q4_backward(y, w, dX=x)
    assert torch.equal(x, gwant) and torch.equal(y, dY)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n", [3, 40, 1000])
def test_bad_rows_stay_in_their_row(n, dtype):
    """A NaN or an infinity in a row of X or dY reaches that row's results alone."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, 264, 136, 32, True, dtype, seed=8)
    w, X, dY = pack(c), put(c["X"], dtype), put(c["dY"], dtype)
    want, gwant = Q.q4_forward(X, w), Q.q4_backward(dY, w)
    bad = n // 2
    for value in (float("nan"), float("inf")):
        X2, dY2 = X.clone(), dY.clone()
        X2[bad, 9], dY2[bad, 100] = value, value
        keep = torch.arange(n, device="cuda") != bad
        assert torch.equal(Q.q4_forward(X2, w)[keep], want[keep])
        assert torch.equal(Q.q4_backward(dY2, w)[keep], gwant[keep])
        assert not torch.isfinite(Q.q4_forward(X2, w)[bad]).any()


def test_gradient_matches_differences():
    """fp32: along random directions, the forward pass's own differences (it
    is linear, so a whole step does)."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(37, 264, 136, 64, True, F32, seed=9)
    w, X, G = pack(c), put(c["X"], F32), put(c["dY"], F32)
    dX = Q.q4_backward(G, w).double()
    gen = torch.Generator(device="cuda").manual_seed(1)
    step = torch.randn(X.shape, generator=gen, device="cuda")
    a, b = Q.q4_forward(X + step, w).double(), Q.q4_forward(X, w).double()
    slope, want = float(((a - b) * G.double()).sum()), float((dX * ((X + step).double() - X.double())).sum())
    mag = float((a.abs() * G.double().abs()).sum() + (b.abs() * G.double().abs()).sum())
    assert abs(slope - want) <= 400 * U * 16 * mag   # sums() U of terms that cancel up to 16 fold


def test_same_bits_on_every_call_and_in_graph_replays():
    """Two captured graphs with their own workspaces, replayed with other rows."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(700, 520, 264, 64, True, BF16, seed=10)
    w, X, G, keep = pack(c), put(c["X"], BF16), put(c["dY"], BF16), {}
    few = X[:20].clone()

    def step():
        keep["Y"], keep["dX"], keep["few"] = Q.q4_forward(X, w), Q.q4_backward(G, w), Q.q4_forward(few, w)

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
        X.add_(0.25)
        few.mul_(0.5)
        want = (Q.q4_forward(X, w), Q.q4_backward(G, w), Q.q4_forward(few, w))
        torch.cuda.synchronize()
        for graph, held in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, held in graphs:
            assert all(torch.equal(held[k], t) for k, t in zip(("Y", "dX", "few"), want)), rep


def test_another_stream_leaves_memory_that_is_still_in_use():
    """Blocks of the sizes that a call allocates, just freed on the current
    stream with their readers still to run there, are not written by a call on
    another stream."""
    import torch
    from input_adaptive_rank_amd import q4 as Q
    n, c1, c2 = 2000, 512, 1024
    c = make(n, c1, c2, 128, False, BF16, seed=11)
    w, X, G = pack(c), put(c["X"], BF16), put(c["dY"], BF16)
    want, gwant = Q.q4_forward(X, w), Q.q4_backward(G, w)
    s, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    sizes = (2 * n * c2, 2 * n * c1, Q.q4_workspace_size(c1, c2, n, BF16), Q.q4_workspace_size(c1, c2, n, BF16, True))
    old = [torch.full((size,), 3, dtype=torch.uint8, device="cuda") for size in sizes]
    kept = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    for _ in range(50):   # some 70 ms on the current stream, then the readers
        torch.mm(a, a, out=b)
    for t, k in zip(old, kept):
        torch.add(t, 1, out=k)
    del t, old
    got, g = Q.q4_forward(X, w, stream=s), Q.q4_backward(G, w, stream=s)
    torch.cuda.synchronize()
    assert all(bool((k == 4).all()) for k in kept)
    assert torch.equal(got, want) and torch.equal(g, gwant)


def refusals():
    import torch
    from input_adaptive_rank_amd import q4 as Q
    bf = torch.bfloat16
    w = pack(make(1, 64, 96, 32, False, BF16, seed=0))
    X, dY = torch.zeros((5, 64), dtype=bf, device="cuda"), torch.zeros((5, 96), dtype=bf, device="cuda")
    codes = torch.zeros((96, 32), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((96, 2), dtype=bf, device="cuda")
    odd = torch.zeros(5 * 64 + 4, dtype=bf, device="cuda")[4:].view(5, 64)
    return {
        "columns": (lambda: Q.q4_forward(dY, w), "must have 64 columns"),
        "type": (lambda: Q.q4_forward(X.half(), w), "bfloat16 or torch.float32"),
        "host rows": (lambda: Q.q4_forward(X.cpu(), w), "X is on cpu"),
        "no rows": (lambda: Q.q4_forward(None, w), "2-D tensor"),
        "bias type": (lambda: Q.q4_forward(X, w, bias=torch.zeros(96, device="cuda")), "bias must be"),
        "bias shape": (lambda: Q.q4_forward(X, w, bias=dY[0, :88]), "bias must have shape"),
        "out shape": (lambda: Q.q4_forward(X, w, out=dY[:4]), "out must have shape"),
        "out overlaps": (lambda: Q.q4_backward(dY, w, dX=dY[:, :64]), "overlap"),
        "odd address": (lambda: Q.q4_forward(odd, w), "16-byte aligned"),
        "transposed rows": (lambda: Q.q4_forward(torch.zeros((64, 5), dtype=bf, device="cuda").t(), w), "rows must be dense"),
        "broadcast rows": (lambda: Q.q4_forward(X[:1].expand(5, 64), w), "rows must be dense"),
        "small workspace": (lambda: Q.q4_backward(dY, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                            "needs"),
        "codes type": (lambda: Q.q4_pack(codes.int(), scale, group=32), "codes must be"),
        "scale type": (lambda: Q.q4_pack(codes, scale.float(), group=32), "scale must be"),
        "scale shape": (lambda: Q.q4_pack(codes, scale, group=64), "scale must have shape"),
        "no scale": (lambda: Q.q4_pack(codes, None, group=32), "scale must be a tensor"),
        "zero shape": (lambda: Q.q4_pack(codes, scale, scale[:, :1].byte(), group=32), "zero must have shape"),
        "group": (lambda: Q.q4_pack(codes, scale, group=16), "group must be one of"),
        "strided codes": (lambda: Q.q4_pack(torch.zeros((96, 64), dtype=torch.uint8, device="cuda")[:, ::2], scale, group=32),
                          "contiguous"),
        "packed bytes": (lambda: Q.Q4Weight(64, 96, 32, w.packed[:100]), "needs"),
        "strided W": (lambda: Q.q4_quantise(torch.zeros((96, 128), dtype=bf, device="cuda")[:, ::2]), "contiguous"),
        "dense type": (lambda: Q.q4_dense(w, torch.float16), "dtype must be"),
    }


REFUSALS = ["columns", "type", "host rows", "no rows", "bias type", "bias shape", "out shape", "out overlaps", "odd address",
            "transposed rows", "broadcast rows", "small workspace", "codes type", "scale type", "scale shape", "no scale",
            "zero shape", "group", "strided codes", "packed bytes", "strided W", "dense type"]


@pytest.mark.parametrize("name", REFUSALS)
def test_refuses(name):
    call, msg = refusals()[name]
    with pytest.raises(ValueError, match=msg):
        call()
