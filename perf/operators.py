"""The measured cases of the adapter and block-norm operators.

adapter_forward    Y = base + scale_a (X A_a^T) B_a^T, the low-rank adapter a
                   of each request beside a shared projection's output `base`
adapter_backward   its gradients: dX, dA, dB
norm_forward       x' = alpha x + gate * postnorm(y),  z = prenorm(x')
norm_backward      its gradients: dx, dy, weights, biases, gate

`run` computes a pass in elementary torch operations in 32 bits, rounded once
at the end, or (own = True) by the package's entry points.  Tokens of all
requests are concatenated: request b is rows offsets[b] .. offsets[b + 1] - 1.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _adapter(name, op, tokens, requests, c1, c2, r, slots, dtype="bf16", mixed=False, bare=0, save_h=False):
    """mixed: ranks r, r/2, r/4 (at least 1) in turn instead of r everywhere;
    bare: requests without an adapter; save_h: the pass keeps H = X A^T for a
    backward pass."""
    return {"name": name, "op": op, "tokens": tokens, "requests": requests, "c1": c1, "c2": c2, "r": r,
            "slots": slots, "dtype": dtype, "mixed": mixed, "bare": bare, "save_h": save_h}


def _norm(name, op, tokens, requests, c, pre, post, gate, dtype="bf16", bias=False, alpha=1.0):
    """pre / post: "rms", "layer" ("none" too for post); gate: "none",
    "channel" (one row) or "request" (one row per request)."""
    return {"name": name, "op": op, "tokens": tokens, "requests": requests, "c": c, "pre": pre, "post": post,
            "gate": gate, "dtype": dtype, "bias": bias, "alpha": alpha}


def listed():
    return [
        # the smallest serving step: four requests, one new token each
        _adapter("decode_few", "adapter_forward", 4, 4, 4096, 4096, 16, 8),
        # a full serving step: one token of each of 192 requests, a large pool with ranks 64, 32 and 16
        _adapter("decode_many", "adapter_forward", 192, 192, 4096, 12288, 64, 64, mixed=True, bare=12),
        # a step that mixes prompts with single tokens: ragged requests, some without an adapter
        _adapter("prefill_mixed", "adapter_forward", 5003, 24, 4096, 4096, 32, 16, mixed=True, bare=3),
        # training forward over the patches of 32 images, H kept for the backward pass
        _adapter("vision_forward", "adapter_forward", 32928, 32, 1024, 4096, 16, 8, save_h=True),
        # fp32 weights, odd sizes, a rank that is no power of two
        _adapter("forward_fp32_odd", "adapter_forward", 211, 6, 264, 520, 24, 5, dtype="fp32", mixed=True, save_h=True),
        # fine-tuning three adapters at once on ragged text
        _adapter("finetune_text", "adapter_backward", 4099, 11, 4096, 4096, 16, 3),
        # fine-tuning on image patches at a high rank
        _adapter("finetune_vision", "adapter_backward", 32928, 32, 1024, 4096, 64, 4),
        # fp32 training at a small rank
        _adapter("finetune_fp32", "adapter_backward", 1031, 9, 1024, 1024, 8, 4, dtype="fp32", mixed=True, bare=1),
        # a serving step between two blocks: norms on both sides of the residual
        _norm("norm_decode", "norm_forward", 8, 8, 4096, "rms", "rms", "none"),
        # a vision block: per-channel gate on the residual branch, layer norm before the next block
        _norm("norm_vision", "norm_forward", 32928, 32, 1024, "layer", "none", "channel", bias=True),
        # training a block with norms on both sides and a gate per request
        _norm("norm_grad_text", "norm_backward", 4099, 7, 4096, "rms", "rms", "request", alpha=0.5),
        # training the vision block
        _norm("norm_grad_vision", "norm_backward", 32928, 32, 1024, "layer", "none", "channel", bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width spread over its logarithm, a multiple of 8 as the layers need."""
    return max(8, 8 * (_log_int(rng, lo, hi) // 8))


def draw(rng):
    op = rng.choice(["adapter_forward", "adapter_forward", "adapter_backward", "norm_forward", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    size = 2 if dtype == "bf16" else 4
    if op.startswith("adapter"):
        c1, c2 = _width(rng, 64, 12288), _width(rng, 64, 12288)
        r, slots = 8 * _log_int(rng, 1, 8), _log_int(rng, 1, 64)
        serving = op == "adapter_forward" and rng.random() < 0.4
        most = min(32928, int(400e6 / size / (2 * (c1 + c2))), int(1.6e11 / (2.0 * slots * r * (2 * c1 + 2 * c2))))
        if serving:
            tokens = requests = _log_int(rng, 1, max(1, min(512, most)))
        else:
            tokens = _log_int(rng, 1, max(1, most))
            requests = _log_int(rng, 1, min(64, tokens))
        bare = rng.randint(0, requests // 4)
        return _draw_only(_adapter("", op, tokens, requests, c1, c2, r, slots, dtype, rng.random() < 0.5, bare,
                                   op == "adapter_forward" and not serving and rng.random() < 0.5))
    c = _width(rng, 64, 8192)
    tokens = _log_int(rng, 1, min(32928, int(400e6 / size / (6 * c))))
    post = rng.choice(["none", "rms", "layer"])
    return _draw_only(_norm("", op, tokens, _log_int(rng, 1, min(64, tokens)), c, rng.choice(["rms", "layer"]), post,
                            rng.choice(["none", "channel", "request"]), dtype, rng.random() < 0.5,
                            rng.choice([1.0, 0.5])))


def _draw_only(case):
    case.pop("name")
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ranks(case):
    r = case["r"]
    return [max(1, r >> (s % 3)) if case["mixed"] else r for s in range(case["slots"])]


def _used_slots(case):
    """How many slots the requests use: they are dealt out in turn."""
    return min(case["slots"], case["requests"] - case["bare"])


def _offsets(gen, tokens, requests):
    """Row offsets of the requests: one token each where that is the count,
    else lengths of random cuts (short, long and now and then empty)."""
    if tokens == requests:
        off = torch.arange(requests + 1)
    else:
        cuts = torch.sort(torch.randint(0, tokens + 1, (requests - 1,), generator=gen)).values
        off = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.full((1,), tokens)])
    return off.to(torch.int32).to(DEV)


def _activations(gen, n, c, dtype):
    """Rows with a few loud channels, as hidden states have."""
    loud = torch.ones(c, device=DEV)
    loud[torch.randint(0, c, (max(1, c // 256),), generator=gen, device=DEV)] = 8.0
    return (torch.randn((n, c), generator=gen, device=DEV) * loud).to(dtype)


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    gen = torch.Generator(device=DEV).manual_seed(int(seed) + 1)
    n, requests, dt = case["tokens"], case["requests"], DT[case["dtype"]]
    randn = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    st = {"op": case["op"], "offsets": _offsets(host, n, requests)}
    if case["op"].startswith("adapter"):
        c1, c2, r, slots = case["c1"], case["c2"], case["r"], case["slots"]
        # requests are dealt to slots in turn; the order is shuffled, `bare` of them have none
        order = torch.randperm(requests, generator=host)
        ids = torch.randperm(slots, generator=host)[torch.arange(requests) % slots].to(torch.int32)
        ids[case["requests"] - case["bare"]:] = -1
        st["slots"] = ids[order].to(DEV)
        st["rank"] = torch.tensor(_ranks(case), dtype=torch.int32, device=DEV)
        st["scale"] = torch.rand(slots, generator=gen, device=DEV) + 0.5
        st["A"] = (randn(slots, r, c1) / math.sqrt(c1)).to(dt)
        st["B"] = (randn(slots, c2, r) * 0.25).to(dt)
        st["X"] = _activations(gen, n, c1, dt)
        if case["op"] == "adapter_forward":
            st["base"] = randn(n, c2).to(dt)
            st["save_h"] = case["save_h"]
        else:
            st["dY"] = (randn(n, c2) * 0.1).to(dt)
            st["dX_base"] = (randn(n, c1) * 0.1).to(dt)
            # what the forward pass kept: X A^T of each row's own adapter
            own_slot, keep = _rows(st, n), _kept(st)
            every = st["X"].float() @ st["A"].float().reshape(slots * r, c1).t()
            mine = every.reshape(n, slots, r).gather(1, own_slot.clamp(min=0)[:, None, None].expand(n, 1, r))[:, 0]
            live = keep[own_slot.clamp(min=0)] & (own_slot >= 0)[:, None]
            st["H"] = torch.where(live, mine, torch.zeros_like(mine))
        return st
    c = case["c"]
    st.update(pre=case["pre"], post=case["post"], alpha=case["alpha"], eps=1e-6)
    weight = lambda: (1 + 0.1 * randn(c)).to(dt)  # noqa: E731
    st["pre_weight"], st["pre_bias"] = weight(), (0.1 * randn(c)).to(dt) if case["bias"] else None
    st["post_weight"] = weight() if case["post"] != "none" else None
    st["post_bias"] = (0.1 * randn(c)).to(dt) if case["bias"] and case["post"] != "none" else None
    rows = {"none": 0, "channel": 1, "request": requests}[case["gate"]]
    gate = (0.5 + 0.2 * randn(rows, c)).to(dt) if rows else None
    st["gate"] = gate[0] if case["gate"] == "channel" else gate
    if case["gate"] != "request":
        st["offsets"] = None
    st["y"] = _activations(gen, n, c, dt)
    if case["op"] == "norm_forward":
        st["x"] = _activations(gen, n, c, dt)
    else:
        st["x_new"] = _activations(gen, n, c, dt)
        st["dz"], st["dx_new"] = (0.1 * randn(n, c)).to(dt), (0.1 * randn(n, c)).to(dt)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _segments(offsets, n):
    """The request of each row."""
    return torch.bucketize(torch.arange(n, device=offsets.device, dtype=torch.int32), offsets[1:], right=True)


def _rows(st, n):
    """The slot of each row, -1 for none."""
    return st["slots"].long()[_segments(st["offsets"], n)]


def _kept(st):
    """[slots][r]: whether a slot's rank reaches this row of A / column of B."""
    return torch.arange(st["A"].shape[1], device=DEV)[None, :] < st["rank"][:, None]


def _pool(st):
    """The whole pool as one pair of fp32 matrices [slots r][c1], [slots r][c2]
    (zero past a slot's rank), and the weight of each row for each of their
    rows: the slot's scale where the slot is the row's own, else zero."""
    A, B, keep = st["A"].float(), st["B"].float().transpose(1, 2), _kept(st)
    slots, r, c1 = A.shape
    A = torch.where(keep[:, :, None], A, torch.zeros_like(A)).reshape(slots * r, c1)
    B = torch.where(keep[:, :, None], B, torch.zeros_like(B)).reshape(slots * r, B.shape[2])
    mine = _rows(st, st["X"].shape[0])[:, None] == torch.arange(slots, device=DEV)[None, :]
    return A, B, mine, (mine * st["scale"][None, :])


def _plain_adapter_forward(st):
    A, B, mine, weight = _pool(st)
    n, (slots, r, _) = st["X"].shape[0], st["A"].shape
    H = (st["X"].float() @ A.t()).reshape(n, slots, r)
    Y = st["base"].float() + (H * weight[:, :, None]).reshape(n, slots * r) @ B
    out = {"Y": Y.to(st["base"].dtype)}
    if st["save_h"]:
        out["H"] = (H * mine[:, :, None]).sum(1)
    return out


def _plain_adapter_backward(st):
    A, B, _, weight = _pool(st)
    n, (slots, r, c1) = st["X"].shape[0], st["A"].shape
    dY = st["dY"].float()
    G = ((dY @ B.t()).reshape(n, slots, r) * weight[:, :, None]).reshape(n, slots * r)
    H = (st["H"][:, None, :] * weight[:, :, None]).reshape(n, slots * r)
    dX = st["dX_base"].float() + G @ A
    dA = G.t() @ st["X"].float()
    dB = dY.t() @ H
    return {"dX": dX.to(st["X"].dtype), "dA": dA.reshape(slots, r, c1),
            "dB": dB.reshape(-1, slots, r).transpose(0, 1).contiguous()}


def _normalised(v, kind, eps):
    """(v - mean) / deviation, and 1 / deviation (mean 0 for "rms")."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    inv = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return v * inv, inv


def _affine(v, weight, bias):
    v = v if weight is None else v * weight.float()
    return v if bias is None else v + bias.float()


def _gate_rows(st, n):
    g = st["gate"]
    if g is None:
        return None
    return g.float()[_segments(st["offsets"], n)] if g.dim() == 2 else g.float()[None, :]


def _branch(st, y):
    """The residual branch before its gate, and the normalised y."""
    if st["post"] == "none":
        return y, None, None
    hat, inv = _normalised(y, st["post"], st["eps"])
    return _affine(hat, st["post_weight"], st["post_bias"]), hat, inv


def _plain_norm_forward(st):
    u, _, _ = _branch(st, st["y"].float())
    g = _gate_rows(st, u.shape[0])
    x_new = st["alpha"] * st["x"].float() + (u if g is None else g * u)
    z = _affine(_normalised(x_new, st["pre"], st["eps"])[0], st["pre_weight"], st["pre_bias"])
    return {"x_new": x_new.to(st["x"].dtype), "z": z.to(st["x"].dtype)}


def _norm_input_grad(d, hat, inv, kind):
    """The gradient of v through hat = normalised(v)."""
    d = d - hat * (d * hat).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if kind == "layer" else 0)
    return d * inv


def _plain_norm_backward(st):
    x, y, dz, dt = st["x_new"].float(), st["y"].float(), st["dz"].float(), st["y"].dtype
    n = x.shape[0]
    hat, inv = _normalised(x, st["pre"], st["eps"])
    out = {"d_pre_weight": (dz * hat).sum(0)}
    if st["pre_bias"] is not None:
        out["d_pre_bias"] = dz.sum(0)
    d = st["dx_new"].float() + _norm_input_grad(dz * st["pre_weight"].float(), hat, inv, st["pre"])
    out["dx"] = (st["alpha"] * d).to(dt)
    u, y_hat, y_inv = _branch(st, y)
    g = _gate_rows(st, n)
    du = d if g is None else d * g
    if g is not None:
        dg = d * u
        if st["gate"].dim() == 2:
            seg = _segments(st["offsets"], n)
            hot = torch.arange(st["gate"].shape[0], device=DEV)[:, None] == seg[None, :]
            out["d_gate"] = hot.float() @ dg
        else:
            out["d_gate"] = dg.sum(0)
    if st["post"] != "none":
        out["d_post_weight"] = (du * y_hat).sum(0)
        if st["post_bias"] is not None:
            out["d_post_bias"] = du.sum(0)
        du = _norm_input_grad(du * st["post_weight"].float(), y_hat, y_inv, st["post"])
    out["dy"] = du.to(dt)
    return out


# ---------------------------------------------------------------------------
# the package's entry points
# ---------------------------------------------------------------------------

def _own_adapter_forward(st):
    from input_adaptive_rank_amd import adapters
    if st["save_h"]:
        Y, H = adapters.adapter_forward(st["X"], st["A"], st["B"], st["offsets"], st["slots"], base=st["base"],
                                        rank=st["rank"], scale=st["scale"], save_h=True)
        return {"Y": Y, "H": H}
    return {"Y": adapters.adapter_forward(st["X"], st["A"], st["B"], st["offsets"], st["slots"], base=st["base"],
                                          rank=st["rank"], scale=st["scale"])}


def _own_adapter_backward(st):
    from input_adaptive_rank_amd import adapters
    dX, dA, dB = adapters.adapter_backward(st["X"], st["dY"], st["H"], st["A"], st["B"], st["offsets"], st["slots"],
                                           dX_base=st["dX_base"], rank=st["rank"], scale=st["scale"])
    return {"dX": dX, "dA": dA, "dB": dB}


def _own_norm_forward(st):
    from input_adaptive_rank_amd import block_norm
    x_new, z = block_norm.block_norm_forward(
        st["x"], st["y"], pre=st["pre"], post=st["post"], pre_weight=st["pre_weight"], pre_bias=st["pre_bias"],
        post_weight=st["post_weight"], post_bias=st["post_bias"], gate=st["gate"], offsets=st["offsets"],
        residual_scale=st["alpha"], eps=st["eps"])
    return {"x_new": x_new, "z": z}


def _own_norm_backward(st):
    from input_adaptive_rank_amd import block_norm
    g = block_norm.block_norm_backward(
        st["x_new"], st["y"], st["dz"], st["dx_new"], pre=st["pre"], post=st["post"], pre_weight=st["pre_weight"],
        pre_bias=st["pre_bias"], post_weight=st["post_weight"], post_bias=st["post_bias"], gate=st["gate"],
        offsets=st["offsets"], residual_scale=st["alpha"], eps=st["eps"])
    return {k: v for k, v in g.items() if v is not None}


_PLAIN = {"adapter_forward": _plain_adapter_forward, "adapter_backward": _plain_adapter_backward,
          "norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward}
_OWN = {"adapter_forward": _own_adapter_forward, "adapter_backward": _own_adapter_backward,
        "norm_forward": _own_norm_forward, "norm_backward": _own_norm_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size, n = (2 if case["dtype"] == "bf16" else 4), case["tokens"]
    if case["op"].startswith("adapter"):
        c1, c2, r = case["c1"], case["c2"], case["r"]
        adapted = n * (case["requests"] - case["bare"]) // case["requests"]
        ranks = _ranks(case)
        rank = sum(ranks) / len(ranks)
        pool = _used_slots(case) * rank * (c1 + c2)
        if case["op"] == "adapter_forward":
            moved = size * (adapted * c1 + 2 * n * c2 + pool) + (4 * n * r if case["save_h"] else 0)
            return {"bytes": moved, "flops": 2.0 * adapted * rank * (c1 + c2) + n * c2}
        moved = size * (adapted * (c1 + c2) + 2 * n * c1 + pool) + 4 * adapted * rank + 4 * case["slots"] * r * (c1 + c2)
        return {"bytes": moved, "flops": 4.0 * adapted * rank * (c1 + c2) + n * c1}
    c = case["c"]
    vectors = 1 + case["bias"] + (case["post"] != "none") * (1 + case["bias"])
    gate = {"none": 0, "channel": 1, "request": case["requests"]}[case["gate"]]
    if case["op"] == "norm_forward":
        return {"bytes": size * (4 * n * c + (vectors + gate) * c), "flops": 12.0 * n * c}
    return {"bytes": size * (6 * n * c + (vectors + gate) * c) + 4 * (vectors + gate) * c, "flops": 30.0 * n * c}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_adapter(st):
    f64 = torch.float64
    off, ids = st["offsets"].tolist(), st["slots"].tolist()
    rank, scale = st["rank"].tolist(), st["scale"].to(f64).tolist()
    forward = st["op"] == "adapter_forward"
    X, r = st["X"], st["A"].shape[1]
    if forward:
        Y, H = st["base"].to(f64), torch.zeros((X.shape[0], r), dtype=f64, device=DEV)
    else:
        dX = st["dX_base"].to(f64)
        dA, dB = torch.zeros(st["A"].shape, dtype=f64, device=DEV), torch.zeros(st["B"].shape, dtype=f64, device=DEV)
    for b, s in enumerate(ids):
        lo, hi = off[b], off[b + 1]
        if s < 0 or lo == hi:
            continue
        k = rank[s]
        A, B, x = st["A"][s, :k].to(f64), st["B"][s, :, :k].to(f64), X[lo:hi].to(f64)
        if forward:
            H[lo:hi, :k] = x @ A.t()
            Y[lo:hi] += scale[s] * (H[lo:hi, :k] @ B.t())
        else:
            dy = st["dY"][lo:hi].to(f64)
            g = scale[s] * (dy @ B)
            dX[lo:hi] += g @ A
            dA[s, :k] += g.t() @ x
            dB[s, :, :k] += scale[s] * (dy.t() @ st["H"][lo:hi, :k].to(f64))
    if forward:
        return {"Y": Y, "H": H} if st["save_h"] else {"Y": Y}
    return {"dX": dX, "dA": dA, "dB": dB}


def _exact_norm(st):
    """Forward from the definition; backward as the derivative, by automatic
    differentiation in 64 bits, of the part of the definition it inverts."""
    f64 = torch.float64
    n = st["y"].shape[0]
    up = lambda k: None if st[k] is None else st[k].to(f64).requires_grad_(True)  # noqa: E731
    par = {k: up(k) for k in ("pre_weight", "pre_bias", "post_weight", "post_bias", "gate")}

    def norm(v, kind, weight, bias):
        centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
        v = (v - centre) / torch.sqrt(((v - centre) ** 2).mean(1, keepdim=True) + st["eps"])
        v = v if weight is None else v * weight
        return v if bias is None else v + bias

    def branch(y):
        u = y if st["post"] == "none" else norm(y, st["post"], par["post_weight"], par["post_bias"])
        if par["gate"] is None:
            return u
        if par["gate"].dim() == 1:
            return u * par["gate"]
        off = st["offsets"].long()
        return u * torch.repeat_interleave(par["gate"], off[1:] - off[:-1], dim=0, output_size=n)

    y = st["y"].to(f64).requires_grad_(True)
    if st["op"] == "norm_forward":
        with torch.no_grad():
            x_new = st["alpha"] * st["x"].to(f64) + branch(y)
            return {"x_new": x_new, "z": norm(x_new, st["pre"], par["pre_weight"], par["pre_bias"])}
    x_new = st["x_new"].to(f64).requires_grad_(True)
    norm(x_new, st["pre"], par["pre_weight"], par["pre_bias"]).backward(st["dz"].to(f64))
    d = x_new.grad + st["dx_new"].to(f64)
    branch(y).backward(d)
    out = {"dx": st["alpha"] * d, "dy": y.grad}
    out.update({"d_" + k: v.grad for k, v in par.items() if v is not None})
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_adapter(st) if st["op"].startswith("adapter") else _exact_norm(st)
