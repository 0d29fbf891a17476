"""Norms around a block (dyra_block_norm_forward / _backward) through the
package's entry points, against the float64 oracle on the same inputs.

Bounds come from a running error analysis: the formulas are evaluated once
more on (value, error) pairs, where every operation adds its own fp32 rounding
(U = 2^-23 of its result, twice the half unit, which leaves room for an order
of operations that differs) to what it passes on from its operands.  A sum of
N terms adds min(N, 64) U of the terms' magnitudes along a row (a tree: 16
terms a lane, 6 levels of lanes, up to 16 waves) and (N + 64) U down a column.
Storing a result in bf16 adds 2^-8 of it, twice the half unit of its 8 bits.
"""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth
from oracle import block_norm_oracle as O

from gpu_cases import log

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
U = 2.0 ** -23
OUT = {F32: U, BF16: 2.0 ** -8}
PARAMS = ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


class V:
    """A value with a bound on its error."""

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)

    def _of(self, v, e):
        return V(v, e + U * (np.abs(v) + e))

    def __add__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._of(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        return self + V(-o.v, o.e)

    def __mul__(self, o):
        o = o if isinstance(o, V) else V(o)
        return self._of(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    def row_mean(self):
        n = self.v.shape[1]
        return self._of(self.v.mean(1, keepdims=True),
                        (self.e + min(n, 64) * U * np.abs(self.v)).mean(1, keepdims=True))

    def col_sum(self):
        n = self.v.shape[0]
        return self._of(self.v.sum(0), (self.e + (n + 64) * U * np.abs(self.v)).sum(0))

    def rsqrt(self):
        r = 1 / np.sqrt(self.v)
        low = np.maximum(self.v - self.e, 1e-300)
        return V(r, 1 / np.sqrt(low) - r + 4 * U * r)


def hat(v, kind, eps):
    if kind == "layer":
        v = v - v.row_mean()
    inv = ((v * v).row_mean() + eps).rsqrt()
    return v * inv, inv


def affine(v, w, b):
    v = v if w is None else v * w
    return v if b is None else v + b


def hat_grad(d, h, inv, kind):
    t = d - h * (d * h).row_mean()
    if kind == "layer":
        t = t - d.row_mean()
    return t * inv


def bounds(c, forward):
    par, n = c["par"], c["y"].shape[0]
    y = V(c["y"])
    g = O.gate_rows(par["gate"], c["offsets"], n)
    if c["post"] == "none":
        u = y
    else:
        hy, iy = hat(y, c["post"], c["eps"])
        u = affine(hy, par["post_weight"], par["post_bias"])
    if forward:
        xn = V(c["x"]) * c["alpha"] + u * g
        return {"x_new": xn, "z": affine(hat(xn, c["pre"], c["eps"])[0], par["pre_weight"], par["pre_bias"])}
    dz = V(c["dz"])
    h, inv = hat(V(c["x_new"]), c["pre"], c["eps"])
    t = dz if par["pre_weight"] is None else dz * par["pre_weight"]
    d = hat_grad(t, h, inv, c["pre"])
    if c["dx_new"] is not None:
        d = d + c["dx_new"]
    out = {"dx": d * c["alpha"], "d_pre_weight": (dz * h).col_sum(), "d_pre_bias": dz.col_sum()}
    du, dg = d * g, d * u
    if par["gate"] is not None and par["gate"].ndim == 1:
        out["d_gate"] = dg.col_sum()
    elif par["gate"] is not None:
        off = c["offsets"]
        parts = [V(dg.v[a:z], dg.e[a:z]).col_sum() for a, z in zip(off[:-1], off[1:])]
        out["d_gate"] = V(np.stack([p.v for p in parts]), np.stack([p.e for p in parts]))
    if c["post"] != "none":
        out["d_post_weight"], out["d_post_bias"] = (du * hy).col_sum(), du.col_sum()
        du = hat_grad(du if par["post_weight"] is None else du * par["post_weight"], hy, iy, c["post"])
    out["dy"] = du
    return out


def make(lens, c, pre, post, gate, dtype, seed, weights=True, biases=False, alpha=1.0, eps=1e-6, mean=0.0,
         with_dx=True):
    g = np.random.default_rng(seed)
    rnd = lambda a: synth.round_storage(a, dtype)  # noqa: E731
    n, nb = int(sum(lens)), len(lens)
    row = lambda m=0.0: rnd(g.standard_normal((n, c)) + m)  # noqa: E731
    vec = lambda m: rnd(m + 0.3 * g.standard_normal(c))  # noqa: E731
    par = dict.fromkeys(PARAMS)
    if weights:
        par["pre_weight"] = vec(1.0)
        par["post_weight"] = vec(1.0) if post != "none" else None
    if biases:
        par["pre_bias"] = vec(0.0)
        par["post_bias"] = vec(0.0) if post != "none" else None
    if gate == "channel":
        par["gate"] = vec(0.5)
    elif gate == "request":
        par["gate"] = rnd(0.5 + 0.3 * g.standard_normal((nb, c)))
    return dict(x=row(mean), y=row(mean), x_new=row(mean), dz=row(), dx_new=row() if with_dx else None, par=par,
                offsets=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), pre=pre, post=post, alpha=alpha,
                eps=eps)


def put(c, dtype):
    import torch
    d = {k: None if c[k] is None else D.to_device(c[k], dtype).reshape(c[k].shape).contiguous()
         for k in ("x", "y", "x_new", "dz", "dx_new")}
    kw = {k: None if v is None else D.to_device(v, dtype) for k, v in c["par"].items()}
    kw.update(pre=c["pre"], post=c["post"], residual_scale=c["alpha"], eps=c["eps"])
    if c["par"]["gate"] is not None and c["par"]["gate"].ndim == 2:
        kw["offsets"] = torch.from_numpy(c["offsets"]).cuda()
    return d, kw


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(c, dtype, got, forward):
    keys = ("pre", "post")
    args = [c[k] for k in keys] + [c["par"]]
    tail = dict(offsets=c["offsets"], alpha=c["alpha"], eps=c["eps"])
    if forward:
        want = dict(zip(("x_new", "z"), O.forward(c["x"], c["y"], *args, **tail)))
    else:
        want = O.backward(c["x_new"], c["y"], c["dz"], c["dx_new"], *args, **tail)
    lim = bounds(c, forward)
    for k, t in got.items():
        if t is None:
            assert k.startswith("d_") and c["par"][k[2:]] is None, k
            continue
        v = host(t)
        unit = OUT[dtype] if k in ("x_new", "z", "dx", "dy") else U
        tol = lim[k].e + unit * (np.abs(want[k]) + lim[k].e)
        err = np.abs(v - want[k])
        worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
        log(f"    {k}: largest error / bound {worst:.3f}")
        assert np.all(np.isfinite(v)), k
        assert np.all(err <= tol), (k, worst)


def run(c, dtype):
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    d, kw = put(c, dtype)
    x_new, z = BN.block_norm_forward(d["x"], d["y"], **kw)
    grads = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], **kw)
    torch.cuda.synchronize()
    check(c, dtype, {"x_new": x_new, "z": z}, True)
    check(c, dtype, grads, False)


KINDS = [(pre, post, gate, biases) for pre in ("rms", "layer") for post in ("none", "rms", "layer")
         for gate in ("none", "channel", "request") for biases in (False, True)]


@pytest.mark.parametrize("pre,post,gate,biases", KINDS)
def test_every_kind_matches_the_oracle(pre, post, gate, biases):
    """Both types at a width whose last chunk of lanes is partly idle, ragged requests, an empty one among them."""
    for dtype in (BF16, F32):
        log(f"  {'bf16' if dtype == BF16 else 'fp32'}")
        run(make([3, 0, 17, 1, 12], 328, pre, post, gate, dtype, seed=1, biases=biases, alpha=0.5), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("c", [8, 64, 512, 520, 1024, 1032, 2048, 2056, 2600, 4096, 4104, 4232, 5640,
                               7000, 8192, 8200, 16384])
def test_every_width_class(c, dtype):
    run(make([5, 4], c, "layer", "rms", "request", dtype, seed=c, biases=True), dtype)
    run(make([1], c, "rms", "none", "none", dtype, seed=c + 1, weights=False), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[1], [2], [7], [4099], [1, 2000, 0, 3, 700, 1395], [33] * 129, [1] * 700,
                                  [9000, 1, 1, 1, 8998]], ids=str)
def test_rows_and_requests(lens, dtype):
    """Requests that lie in a run of rows, span several, start and end with one."""
    run(make(lens, 72, "rms", "layer", "request", dtype, seed=len(lens), alpha=1.5), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_large_mean(dtype):
    """A layer norm of rows whose mean is far above their deviation."""
    run(make([40], 1024, "layer", "layer", "channel", dtype, seed=3, mean=100.0), dtype)


def test_no_direct_gradient_and_zero_rows():
    run(make([50], 264, "layer", "rms", "channel", BF16, seed=4, with_dx=False), BF16)
    c = make([6], 264, "rms", "rms", "none", F32, seed=5, eps=1e-5)
    c["y"][2] = 0
    c["x"][3] = 0
    c["x_new"][4] = 0
    run(c, F32)


def test_no_rows():
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    for gate in ("none", "channel", "request"):
        d, kw = put(make([0, 0], 64, "rms", "rms", gate, BF16, seed=1, biases=True), BF16)
        x_new, z = BN.block_norm_forward(d["x"], d["y"], **kw)
        assert x_new.shape == z.shape == (0, 64)
        g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], **kw)
        torch.cuda.synchronize()
        assert all(t is None or not t.any() for t in g.values())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("post", ["none", "rms"])
def test_no_requests(post, dtype):
    """A gate per request of no requests: no rows, a gate without rows, and
    parameter gradients that are zero whatever the memory held."""
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    d, kw = put(make([0], 64, "rms", post, "request", dtype, seed=1, biases=True), dtype)
    kw.update(gate=kw["gate"][:0].contiguous(), offsets=kw["offsets"][:1].contiguous())
    assert all(t.shape == (0, 64) for t in BN.block_norm_forward(d["x"], d["y"], **kw))
    g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], **kw)
    torch.cuda.synchronize()
    assert g["d_gate"].shape == g["dx"].shape == g["dy"].shape == (0, 64)
    for k in PARAMS[:4]:
        assert (g["d_" + k] is None) == (kw[k] is None) and (kw[k] is None or not g["d_" + k].any())


def test_a_bad_row_spoils_only_itself():
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    c = make([30, 40], 520, "layer", "rms", "request", BF16, seed=6)
    d, kw = put(c, BF16)
    clean = BN.block_norm_forward(d["x"], d["y"], **kw)
    g0 = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], **kw)
    d["y"][11, 3] = float("inf")
    d["dz"][12] = float("nan")
    out = BN.block_norm_forward(d["x"], d["y"], **kw)
    g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], **kw)
    torch.cuda.synchronize()
    rows = torch.arange(70, device="cuda")
    for a, b in zip(clean, out):
        assert torch.equal(a[rows != 11], b[rows != 11]) and not torch.isfinite(b[11]).all()
    keep = (rows != 11) & (rows != 12)
    for k in ("dx", "dy"):
        assert torch.equal(g[k][keep], g0[k][keep])
    assert torch.equal(g["d_gate"][1], g0["d_gate"][1]) and not torch.isfinite(g["d_gate"][0]).any()


def test_in_place():
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    for c in (520, 4096):
        d, kw = put(make([70], c, "rms", "layer", "channel", BF16, seed=7), BF16)
        want = BN.block_norm_forward(d["x"], d["y"], **kw)
        g0 = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], **kw)
        x, y = d["x"].clone(), d["y"].clone()
        a, b = BN.block_norm_forward(x, y, x_new=x, z=y, **kw)
        assert a is x and b is y and torch.equal(x, want[0]) and torch.equal(y, want[1])
        y, dxn = d["y"].clone(), d["dx_new"].clone()
        g = BN.block_norm_backward(d["x_new"], y, d["dz"], dxn, dx=dxn, dy=y, **kw)
        torch.cuda.synchronize()
        assert g["dx"] is dxn and torch.equal(dxn, g0["dx"]) and torch.equal(y, g0["dy"])
        with pytest.raises(ValueError, match="overlap"):
            BN.block_norm_forward(x, y, x_new=x, z=x, **kw)


def test_gradients_match_differences():
    """The device's fp32 gradients along random directions against fourth
    order differences of the float64 forward.  Each gradient element is off by
    some tens of U of the magnitudes it is a sum of (measured against the
    oracle's by the tests above); along a direction that is at most 2^-13 of
    sum |gradient direction|, and the differences' own error (h^4, and 2^-52
    of the loss over h) is far below."""
    from input_adaptive_rank_amd import block_norm as BN
    c = make([9, 14], 136, "layer", "rms", "request", F32, seed=8, biases=True, alpha=0.5)
    args, tail = (c["pre"], c["post"]), dict(offsets=c["offsets"], alpha=c["alpha"], eps=c["eps"])
    x_new = synth.round_storage(O.forward(c["x"], c["y"], *args, c["par"], **tail)[0], F32)
    c["x_new"] = x_new
    d, kw = put(c, F32)
    g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], **kw)
    rng = np.random.default_rng(9)

    def loss(x, y, par):
        a, z = O.forward(x, y, *args, par, **tail)
        return (a * c["dx_new"]).sum() + (z * c["dz"]).sum()

    for k in ("x", "y") + PARAMS:
        base = c[k] if k in ("x", "y") else c["par"][k]
        step = rng.standard_normal(base.shape)

        def at(t):
            moved = base + t * step
            x, y, par = c["x"], c["y"], dict(c["par"])
            if k == "x":
                x = moved
            elif k == "y":
                y = moved
            else:
                par[k] = moved
            return loss(x, y, par)

        h = 1e-3
        slope = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
        dev = host(g["d" + k if k in ("x", "y") else "d_" + k])
        log(f"    {k}: difference {slope:.6f}, gradient {(dev * step).sum():.6f}")
        assert abs(slope - (dev * step).sum()) <= 2.0 ** -13 * np.abs(dev * step).sum()


def test_same_bits_on_every_call_and_in_graph_replays():
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    d, kw = put(make([700, 1, 0, 300], 1032, "layer", "rms", "request", BF16, seed=10, biases=True), BF16)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    keep = {}

    def step():
        keep["f"] = BN.block_norm_forward(d["x"], d["y"], **kw)
        keep["b"] = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], workspace=ws, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = dict(keep)
    for rep in range(4):
        d["y"].add_(0.25)
        kw["offsets"].copy_(torch.tensor([0, 100 + rep, 100 + rep, 900, 1001], dtype=torch.int32))
        f = BN.block_norm_forward(d["x"], d["y"], **kw)
        b = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], d["dx_new"], **kw)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(f, held["f"])), rep
        for k, t in b.items():
            assert torch.equal(t, held["b"][k]), (rep, k)


def test_another_stream():
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    d, kw = put(make([500], 1024, "rms", "rms", "channel", BF16, seed=11), BF16)
    want = BN.block_norm_forward(d["x"], d["y"], **kw)
    g0 = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = BN.block_norm_forward(d["x"], d["y"], stream=s, **kw)
    g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], stream=s, **kw)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(g[k] is None or torch.equal(g[k], g0[k]) for k in g)


def test_another_stream_leaves_memory_that_is_still_in_use():
    """Blocks of the sizes that a call allocates, just freed on the current
    stream with their readers still to run there, are not written by a call on
    another stream."""
    import torch
    from input_adaptive_rank_amd import block_norm as BN
    n, c = 4096, 1024
    d, kw = put(make([n], c, "rms", "rms", "channel", BF16, seed=12), BF16)
    want = BN.block_norm_forward(d["x"], d["y"], **kw)
    g0 = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], **kw)
    s, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    b = torch.empty_like(a)
    old = [torch.full((size,), 3, dtype=torch.uint8, device="cuda") for size in (2 * n * c, 2 * n * c, 3 * 4 * c, 4 << 20)]
    kept = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    for _ in range(50):   # some 70 ms on the current stream, then the readers
        torch.mm(a, a, out=b)
    for t, k in zip(old, kept):
        torch.add(t, 1, out=k)
    del t, old
    got = BN.block_norm_forward(d["x"], d["y"], stream=s, **kw)
    g = BN.block_norm_backward(d["x_new"], d["y"], d["dz"], stream=s, **kw)
    torch.cuda.synchronize()
    assert all(bool((k == 4).all()) for k in kept)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(g[k] is None or torch.equal(g[k], g0[k]) for k in g)
