"""Low-rank adapters of many requests (dyra_adapter_forward / _backward)
through the package's entry points, against the float64 oracle on the same
inputs.

Bounds, elementwise, derived from the number formats: a sum of N products
accumulated in fp32 in any order is off by at most N 2^-23 (a factor of two
over N 2^-24 for the order-dependent second-order terms) times the sum of the
products' magnitudes; H or G entering a bf16 product as two bf16 terms adds
2^-16 of the magnitudes, as three 2^-24; an output rounded to bf16 adds 2^-8
of itself (half a unit is 2^-9), to fp32 2^-23.
"""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import adapter_oracle as O

from gpu_cases import log

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
OUT = {F32: 2.0 ** -23, BF16: 2.0 ** -8}
MID = {F32: 0.0, BF16: 2.0 ** -16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def make(lens, ids, c1, c2, r, slots, dtype, seed, ranks=None):
    """Host float64 inputs already representable in the storage type.  Past
    an adapter's rank the pool holds NaN: it must not be used."""
    g = np.random.default_rng(seed)
    rnd = lambda a: synth.round_storage(a, dtype)  # noqa: E731
    n = int(sum(lens))
    case = dict(X=rnd(g.standard_normal((n, c1))), base=rnd(g.standard_normal((n, c2))),
                dY=rnd(g.standard_normal((n, c2))), dX_base=rnd(g.standard_normal((n, c1))),
                A=rnd(g.standard_normal((slots, r, c1)) / np.sqrt(c1)), B=rnd(g.standard_normal((slots, c2, r))),
                offsets=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), slots=np.array(ids, np.int32),
                scale=g.uniform(0.5, 2.0, slots).astype(np.float32),
                rank=None if ranks is None else np.array(ranks, np.int32))
    for a in range(slots if ranks is not None else 0):
        case["A"][a, ranks[a]:] = np.nan
        case["B"][a, :, ranks[a]:] = np.nan
    return case


def put(case, dtype):
    import torch
    d = {}
    for k, v in case.items():
        if v is None:
            d[k] = None
        elif v.dtype == np.float64:
            d[k] = D.to_device(v, dtype)
        else:
            d[k] = torch.from_numpy(v).cuda()
    return d


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def within(name, got, want, bound):
    err = np.abs(got - want)
    worst = float(np.max(err / np.maximum(bound, 1e-300))) if err.size else 0.0
    log(f"    {name}: largest error / bound {worst:.3f}")
    assert np.all(np.isfinite(got)), name
    assert np.all(err <= bound), (name, worst)


def check_forward(case, dtype, Y, H, base):
    want, wh, ay, ah = O.forward(case["X"], case["A"], case["B"], case["offsets"], case["slots"], base=base,
                                 rank=case["rank"], scale=case["scale"])
    c1, r = case["X"].shape[1], case["A"].shape[1]
    within("Y", host(Y), want, OUT[dtype] * np.abs(want) + (MID[dtype] + (c1 + r + 16) * 2.0 ** -23) * ay)
    if H is not None:
        within("H", host(H), wh, (c1 + 16) * 2.0 ** -23 * ah)
    return wh


def check_backward(case, dtype, grads, dX_base, H):
    """H: what the device was given, as float64."""
    dX, dA, dB, aX, aA, aB = O.backward(case["X"], case["dY"], H, case["A"], case["B"], case["offsets"],
                                        case["slots"], dX_base=dX_base, rank=case["rank"], scale=case["scale"])
    n, c2, r = case["X"].shape[0], case["dY"].shape[1], case["A"].shape[1]
    if grads[0] is not None:
        within("dX", host(grads[0]), dX, OUT[dtype] * np.abs(dX) + (MID[dtype] + (c2 + r + 16) * 2.0 ** -23) * aX)
    if grads[1] is not None:
        within("dA", host(grads[1]), dA, (n + c2 + 64) * 2.0 ** -23 * aA)
        within("dB", host(grads[2]), dB, (n + 64) * 2.0 ** -23 * aB)


def run_forward(d, **kw):
    from input_adaptive_rank_amd import adapters as AD
    return AD.adapter_forward(d["X"], d["A"], d["B"], d["offsets"], d["slots"], rank=d["rank"], scale=d["scale"], **kw)


def run_backward(d, H, **kw):
    from input_adaptive_rank_amd import adapters as AD
    return AD.adapter_backward(d["X"], d["dY"], H, d["A"], d["B"], d["offsets"], d["slots"], rank=d["rank"],
                               scale=d["scale"], **kw)


# name: (lengths, slots of the requests, c1, c2, r, pool size, ranks)
CASES = {
    "one_token": ([1], [0], 64, 72, 8, 1, None),
    "one_bare_token": ([1], [-1], 64, 72, 8, 1, None),
    "singles_shared_slots": ([1] * 37, [i * 7 % 5 - 1 for i in range(37)], 264, 520, 24, 4, [24, 9, 16, 1]),
    "empty_requests": ([0, 5, 0, 0, 33, 0], [1, 0, 2, -1, 2, 1], 128, 256, 16, 3, None),
    "ragged": ([65, 1, 130, 7, 64, 3, 200], [0, 2, 0, -1, 1, 2, 1], 520, 776, 40, 3, [40, 33, 8]),
    "long_tiles": ([600, 1, 299, 64], [1, 0, 1, -1], 256, 320, 64, 2, [64, 17]),
    "narrow": ([513, 100], [0, 1], 8, 8, 8, 2, None),
    "rank_zero": ([40, 50], [0, 1], 72, 136, 16, 2, [0, 16]),
    "rank_128": ([100, 420, 77], [2, 0, 2], 384, 264, 128, 3, [128, 100, 127]),
    "slot_out_of_pool": ([20, 30, 10], [3, 1, 1 << 30], 64, 64, 8, 3, None),
    "wide": ([9, 2], [0, 1], 4104, 12296, 16, 2, None),
}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("name", CASES)
def test_forward_and_backward_match_the_oracle(name, dtype):
    import torch
    lens, ids, c1, c2, r, slots, ranks = CASES[name]
    log(f"  {name} {'bf16' if dtype == BF16 else 'fp32'}")
    case = make(lens, ids, c1, c2, r, slots, dtype, seed=len(name), ranks=ranks)
    d = put(case, dtype)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    torch.cuda.synchronize()
    check_forward(case, dtype, Y, H, case["base"])
    check_forward(case, dtype, run_forward(d), None, None)
    grads = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    check_backward(case, dtype, grads, case["dX_base"], host(H))
    dX, none_a, none_b = run_backward(d, None, need_weights=False)
    assert none_a is None and none_b is None
    check_backward(case, dtype, (dX, None, None), None, host(H))
    none_x, dA, dB = run_backward(d, H, need_dx=False)
    assert none_x is None and torch.equal(dA, grads[1]) and torch.equal(dB, grads[2])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("r", [16, 72])
def test_gradients_of_slots_with_one_run_of_rows_and_with_many(r, dtype):
    """Slots of a few rows beside slots of many, ranks that end inside a
    block of 16 or of 4, into memory that held NaN."""
    import torch
    ranks = [r, 0, r - 3, r, 5, r - 8, r]
    lens, ids = [3, 700, 64, 1, 20, 500, 9, 65], [0, 1, 2, 4, 1, 3, 5, 2]   # slot 6 has no row
    case = make(lens, ids, 264, 520, r, 7, dtype, seed=r, ranks=ranks)
    d = put(case, dtype)
    _, H = run_forward(d, save_h=True)
    dA = torch.full(d["A"].shape, float("nan"), dtype=torch.float32, device="cuda")
    dB = torch.full(d["B"].shape, float("nan"), dtype=torch.float32, device="cuda")
    grads = run_backward(d, H, dX_base=d["dX_base"], dA=dA, dB=dB)
    torch.cuda.synchronize()
    check_backward(case, dtype, grads, case["dX_base"], host(H))


def test_many_requests_and_slots():
    """More requests than a workgroup sorts at once, more slots than rows of a tile."""
    import torch
    g = np.random.default_rng(5)
    lens = g.integers(0, 3, 2500).tolist()
    ids = g.integers(-1, 200, 2500).tolist()
    case = make(lens, ids, 64, 64, 8, 200, BF16, seed=6)
    d = put(case, BF16)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    check_forward(case, BF16, Y, H, case["base"])
    check_backward(case, BF16, grads, case["dX_base"], host(H))


def test_no_rows_and_no_requests():
    import torch
    case = make([0, 0], [0, 1], 64, 72, 8, 2, BF16, seed=1)
    d = put(case, BF16)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    assert Y.shape == (0, 72) and H.shape == (0, 8)
    dX, dA, dB = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    d = put(make([70], [0], 64, 72, 8, 2, BF16, seed=2), BF16)
    d["offsets"], d["slots"] = d["offsets"][:1].contiguous(), d["slots"][:0].contiguous()   # rows of no request
    assert torch.equal(run_forward(d, base=d["base"]), d["base"])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_rows_without_an_adapter_ignore_their_inputs(dtype):
    """NaN and Inf in bare rows reach neither their outputs nor any gradient."""
    import torch
    case = make([30, 40, 50], [1, -1, 0], 136, 200, 16, 2, dtype, seed=3)
    d = put(case, dtype)
    for t in (d["X"], d["dY"]):
        t[30:50] = float("nan")
        t[50:70] = float("inf")
    Y, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    assert torch.equal(Y[30:70], d["base"][30:70]) and not H[30:70].any()
    check_forward(case, dtype, Y, H, case["base"])
    check_backward(case, dtype, grads, case["dX_base"], host(H))


def test_bad_rows_stay_in_their_request():
    """A NaN row spoils its own Y and its adapter's gradients, nothing else."""
    import torch
    case = make([90, 90], [0, 1], 136, 200, 16, 2, BF16, seed=4)
    d = put(case, BF16)
    clean = run_forward(d, base=d["base"])
    Y0, H0 = run_forward(d, base=d["base"], save_h=True)
    clean_grads = run_backward(d, H0)
    d["X"][7] = float("nan")
    Y, H = run_forward(d, base=d["base"], save_h=True)
    dX, dA, dB = run_backward(d, H)
    torch.cuda.synchronize()
    keep = torch.arange(180, device="cuda") != 7
    assert torch.equal(Y[keep], clean[keep]) and torch.isnan(Y[7]).all()
    assert torch.equal(dA[1], clean_grads[1][1]) and torch.equal(dB[1], clean_grads[2][1])
    assert torch.isnan(dA[0]).all() and torch.isnan(dB[0]).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_column_ranges_of_wider_matrices_and_in_place(dtype):
    """X, base, Y, dY, dX as column ranges; Y into base and dX into dX_base."""
    import torch
    case = make([70, 3, 90], [1, 0, 1], 264, 136, 24, 2, dtype, seed=8)
    d = put(case, dtype)
    plain = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, plain[1], dX_base=d["dX_base"])

    def widen(t, before, after):
        w = torch.full((t.shape[0], before + t.shape[1] + after), float("nan"), dtype=t.dtype, device=t.device)
        v = w[:, before:before + t.shape[1]]
        v.copy_(t)
        return w, v

    views = {}
    for k, (a, z) in dict(X=(8, 16), base=(16, 8), dY=(24, 8), dX_base=(8, 8)).items():
        views[k], d[k] = widen(d[k], a, z)
    assert run_forward(d, base=d["base"], out=d["base"]) is d["base"]
    dX, dA, dB = run_backward(d, plain[1], dX_base=d["dX_base"], dX=d["dX_base"])
    torch.cuda.synchronize()
    assert dX is d["dX_base"]
    assert torch.equal(d["base"], plain[0]) and torch.equal(dX, grads[0])
    assert torch.equal(dA, grads[1]) and torch.equal(dB, grads[2])
    assert torch.isnan(views["base"][:, :16]).all() and torch.isnan(views["base"][:, 152:]).all()
    assert torch.isnan(views["dX_base"][:, :8]).all() and torch.isnan(views["dX_base"][:, 272:]).all()


def test_gradients_match_differences():
    """Y is linear in each of X, A and B, so a difference of the forward pass
    over any step equals the gradient along it up to rounding."""
    import torch
    case = make([50, 1, 33, 20], [0, 1, 0, -1], 72, 88, 16, 2, F32, seed=9)
    d = put(case, F32)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    grads = dict(zip("XAB", run_backward(d, H)))
    dY = case["dY"]
    for k in "XAB":
        step = D.to_device(np.random.default_rng(10).standard_normal(case[k].shape), F32)
        moved = dict(d)
        moved[k] = d[k] + step
        delta = float((dY * (host(run_forward(moved, base=d["base"])) - host(Y))).sum())
        slope = float((host(grads[k]) * (host(moved[k]) - case[k])).sum())
        # each Y element is off by at most (c1 + r + 16) 2^-23 of its terms' magnitudes, on both sides
        both = dict(case, X=host(moved["X"]), A=host(moved["A"]), B=host(moved["B"]))
        terms = [O.forward(c["X"], c["A"], c["B"], c["offsets"], c["slots"], base=c["base"], scale=c["scale"])
                 for c in (case, both)]
        size = sum((np.abs(dY) * (np.abs(t[0]) + t[2])).sum() for t in terms)
        log(f"    {k}: difference {delta:.6f}, gradient {slope:.6f}")
        assert abs(delta - slope) <= 2 * (72 + 16 + 16) * 2.0 ** -23 * size


def test_same_bits_on_every_call_and_in_graph_replays():
    import torch
    g = np.random.default_rng(11)
    lens = g.integers(1, 90, 40).tolist()
    case = make(lens, g.integers(-1, 6, 40).tolist(), 512, 776, 32, 6, BF16, seed=12)
    d = put(case, BF16)
    from input_adaptive_rank_amd import adapters as AD
    n = d["X"].shape[0]
    ws = [torch.empty(AD.adapter_workspace_size(6, 32, 512, 776, n, 40, torch.bfloat16, back), dtype=torch.uint8,
                      device="cuda") for back in (False, True)]
    out = dict(Y=torch.empty_like(d["base"]), H=torch.empty((n, 32), device="cuda"), dX=torch.empty_like(d["X"]),
               dA=torch.empty((6, 32, 512), device="cuda"), dB=torch.empty((6, 776, 32), device="cuda"))

    def step():
        run_forward(d, base=d["base"], out=out["Y"], H=out["H"], workspace=ws[0])
        run_backward(d, out["H"], dX_base=d["dX_base"], dX=out["dX"], dA=out["dA"], dB=out["dB"], workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        d["slots"].copy_(torch.from_numpy(g.integers(-1, 6, 40).astype(np.int32)))   # other requests each time
        Y, H = run_forward(d, base=d["base"], save_h=True)
        want = dict(zip(("dX", "dA", "dB"), run_backward(d, H, dX_base=d["dX_base"])), Y=Y, H=H)
        torch.cuda.synchronize()
        for t in out.values():
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for k, t in out.items():
            assert torch.equal(t, want[k]), (rep, k)


def test_another_stream():
    import torch
    case = make([300, 500], [0, 1], 256, 256, 16, 2, BF16, seed=13)
    d = put(case, BF16)
    want, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = run_forward(d, base=d["base"], stream=s)
    other = run_backward(d, H, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(other, grads))


def test_another_stream_leaves_memory_that_is_still_in_use():
    """Blocks of the sizes that a call allocates, just freed on the current
    stream with their readers still to run there, are not written by a call on
    another stream."""
    import torch
    from input_adaptive_rank_amd import adapters as AD
    n, c, r = 4096, 1024, 16
    case = make([3000, n - 3000], [0, 1], c, c, r, 2, BF16, seed=14)
    d = put(case, BF16)
    want, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H)
    s, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    sizes = [2 * n * c, 4 * n * r] + [AD.adapter_workspace_size(2, r, c, c, n, 2, BF16, back) for back in (0, 1)]
    old = [torch.full((size,), 3, dtype=torch.uint8, device="cuda") for size in sizes]
    kept = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    for _ in range(50):   # some 70 ms on the current stream, then the readers
        torch.mm(a, a, out=b)
    for t, k in zip(old, kept):
        torch.add(t, 1, out=k)
    del t, old
    got, h = run_forward(d, base=d["base"], save_h=True, stream=s)
    other = run_backward(d, h, stream=s)
    torch.cuda.synchronize()
    assert all(bool((k == 4).all()) for k in kept)
    assert torch.equal(got, want) and torch.equal(h, H)
    assert all(torch.equal(p, q) for p, q in zip(other, grads))


@pytest.mark.parametrize("n", [5, 700])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_operands_and_results_side_by_side_in_one_matrix(n, dtype):
    """X, base (written in place) and dX as column ranges of one wide matrix."""
    import torch
    c1, c2 = 136, 72
    case = make([n - 2, 2], [1, 0], c1, c2, 24, 2, dtype, seed=15)
    d = put(case, dtype)
    want, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H)
    wide = torch.full((n, 2 * c1 + c2), float("nan"), dtype=d["X"].dtype, device="cuda")
    X, Y, dX = wide[:, :c1], wide[:, c1:c1 + c2], wide[:, c1 + c2:]
    X.copy_(d["X"])
    Y.copy_(d["base"])
    d["X"] = X
    run_forward(d, base=Y, out=Y)
    run_backward(d, H, dX=dX)
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and torch.equal(dX, grads[0])
    with pytest.raises(ValueError, match="overlap"):
        run_forward(d, out=wide[:, c1 - 8:c1 + c2 - 8])


def test_one_row_in_place_by_another_view():
    """base and out as two views of one row, which have different strides."""
    import torch
    d = put(make([1], [0], 64, 72, 8, 1, BF16, seed=16), BF16)
    want = run_forward(d, base=d["base"])
    wide = torch.zeros((2, 80), dtype=torch.bfloat16, device="cuda")
    wide[:1, 8:].copy_(d["base"])
    run_forward(d, base=wide[:1, 8:], out=wide[0, 8:][None])
    assert torch.equal(wide[:1, 8:], want)


FORWARD_REFUSALS = {
    "out_not_a_tensor": dict(out="out"), "out_shape": dict(out=(10, 80)), "out_type": dict(out=(10, 72, "float32")),
    "h_not_a_tensor": dict(H=3.0), "h_shape": dict(H=(10, 16, "float32")), "h_type": dict(H=(10, 8)),
    "base_rows": dict(base=(9, 72)), "base_not_a_tensor": dict(base=[1]), "rank_type": dict(rank=(2, "float32")),
    "scale_shape": dict(scale=(3, "float32")), "workspace_type": dict(workspace=(1 << 20, "float32")),
    "offsets_short": dict(offsets=(2, "int32")),
}


def made(v):
    """A tensor of the shape, and type if it ends in one, that a tuple names."""
    import torch
    if not isinstance(v, tuple):
        return v
    dtype = getattr(torch, v[-1]) if isinstance(v[-1], str) else torch.bfloat16
    return torch.zeros(tuple(k for k in v if not isinstance(k, str)), dtype=dtype, device="cuda")


@pytest.mark.parametrize("name", FORWARD_REFUSALS)
def test_forward_refuses(name):
    from input_adaptive_rank_amd import adapters as AD
    d = put(make([4, 6], [0, 1], 64, 72, 8, 2, BF16, seed=17), BF16)
    kw = dict(base=d["base"], rank=d["rank"], scale=d["scale"], offsets=d["offsets"], slots=d["slots"])
    kw.update({k: made(v) for k, v in FORWARD_REFUSALS[name].items()})
    with pytest.raises(ValueError, match=next(iter(FORWARD_REFUSALS[name]))):
        AD.adapter_forward(d["X"], d["A"], d["B"], **kw)


BACKWARD_REFUSALS = {
    "dx_not_a_tensor": dict(dX="dX"), "dx_shape": dict(dX=(10, 72)), "da_not_a_tensor": dict(dA=0),
    "da_type": dict(dA=(2, 8, 64)), "db_shape": dict(dB=(2, 8, 72, "float32")), "db_not_a_tensor": dict(dB="dB"),
    "dx_base_shape": dict(dX_base=(10, 72)), "h_missing": dict(H=None),
}


@pytest.mark.parametrize("name", BACKWARD_REFUSALS)
def test_backward_refuses(name):
    from input_adaptive_rank_amd import adapters as AD
    d = put(make([4, 6], [0, 1], 64, 72, 8, 2, BF16, seed=18), BF16)
    kw = dict(H=made((10, 8, "float32")), offsets=d["offsets"], slots=d["slots"])
    kw.update({k: made(v) for k, v in BACKWARD_REFUSALS[name].items()})
    with pytest.raises(ValueError, match=next(iter(BACKWARD_REFUSALS[name]))):
        AD.adapter_backward(d["X"], d["dY"], A=d["A"], B=d["B"], **kw)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("r", [16, 40])
def test_a_large_pool_few_of_whose_slots_are_used(r, dtype):
    """More slots than requests: repeated slots, an empty request before the
    first one with rows of its slot, bare ones; slots far apart and the last."""
    import torch
    slots = 300
    lens = [0, 700, 64, 0, 130, 1, 65, 300, 200]
    ids = [299, 17, -1, 17, 299, 0, 17, 300, 299]
    ranks = [r - s % 9 for s in range(slots)]
    case = make(lens, ids, 264, 136, r, slots, dtype, seed=19, ranks=ranks)
    d = put(case, dtype)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    grads = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    check_forward(case, dtype, Y, H, case["base"])
    check_backward(case, dtype, grads, case["dX_base"], host(H))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("r", [40, 64, 72, 128])
def test_a_few_rows_at_high_ranks(r, dtype):
    """One launch, whose waves split 64 or 128 rank columns."""
    import torch
    from input_adaptive_rank_amd import adapters as AD
    lens, ids, ranks = [1, 2, 0, 1, 1], [2, 0, 1, -1, 1], [r, r - 3, 17]
    case = make(lens, ids, 520, 776, r, 3, dtype, seed=r, ranks=ranks)
    d = put(case, dtype)
    assert AD.adapter_workspace_size(3, r, 520, 776, 5, 5, dtype) == 0
    Y, H = run_forward(d, base=d["base"], save_h=True)
    torch.cuda.synchronize()
    check_forward(case, dtype, Y, H, case["base"])


def chunk_count(slots, r, c1, c2, n, requests, dtype):
    """Chunks of rows that a backward pass has partial gradients for, from
    what its workspace gains with c1 (their sums, and A's packed operands)."""
    from input_adaptive_rank_amd import adapters as AD
    wide, narrow = (AD.adapter_workspace_size(slots, r, c, c2, n, requests, dtype, True) for c in (240, 16))
    packed = min(slots, requests) * 14 * -(-r // (32 if dtype == BF16 else 16)) * 1024
    return round((wide - narrow - packed) / (4 * r * 224))


def make_whole(lens, ids, c1, c2, r, slots, dtype, seed, ranks):
    """Small whole numbers: every product and sum is exact in fp32, in whatever
    order, so results equal the oracle's, rounded once."""
    g = np.random.default_rng(seed)
    n = int(sum(lens))
    ints = lambda *shape: g.integers(-1, 2, shape).astype(np.float64)  # noqa: E731
    return dict(X=ints(n, c1), base=ints(n, c2), dY=ints(n, c2), dX_base=ints(n, c1), A=ints(slots, r, c1),
                B=ints(slots, c2, r), offsets=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32),
                slots=np.array(ids, np.int32), scale=g.choice([0.5, 1.0, 2.0], slots).astype(np.float32),
                rank=np.array(ranks, np.int32))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("r,n", [(8, 33000), (32, 33000), (40, 33000), (72, 33000), (128, 33000), (40, 530000)])
def test_many_rows_bit_by_bit(r, n, dtype):
    """Chunks of several tiles (of the most there are at 530000 rows), several
    chunks a slot, runs that end inside a tile and inside its halves, two row
    blocks a workgroup in the product with c1 or c2; small odd widths."""
    import torch
    c1, c2, slots = 136, 72, 3
    lens = [n // 3 + 17, 1, 4000, 40, n // 2 - 5000, 0]
    lens.append(n - sum(lens))
    ids = [0, 1, 2, 1, 0, 2, -1]
    case = make_whole(lens, ids, c1, c2, r, slots, dtype, seed=r, ranks=[r, r - 1, r - 5])
    tiles, chunks = n // 64, chunk_count(slots, r, c1, c2, n, len(lens), dtype)
    log(f"  {tiles} tiles, {chunks} chunks")
    assert chunks <= (tiles // 32 + slots + 1 if n == 530000 else tiles // 2)
    d = put(case, dtype)
    Y, H = run_forward(d, base=d["base"], save_h=True)
    dX, dA, dB = run_backward(d, H, dX_base=d["dX_base"])
    torch.cuda.synchronize()
    y, h, _, _ = O.forward(case["X"], case["A"], case["B"], case["offsets"], ids, base=case["base"], rank=case["rank"],
                           scale=case["scale"])
    dx, da, db, _, size_a, size_b = O.backward(case["X"], case["dY"], h, case["A"], case["B"], case["offsets"], ids,
                                               dX_base=case["dX_base"], rank=case["rank"], scale=case["scale"])
    assert max(size_a.max(), size_b.max()) < 2.0 ** 23   # halves of whole numbers
    for name, got, want in (("Y", Y, synth.round_storage(y, dtype)), ("H", H, h),
                            ("dX", dX, synth.round_storage(dx, dtype)), ("dA", dA, da), ("dB", dB, db)):
        wrong = int((host(got) != want).sum())
        assert wrong == 0, (name, wrong)
