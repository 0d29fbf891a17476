"""A block around a DyRA layer as a server or a trainer would run it: the
shared layer, each request's adapter beside it, and the norms, gate and
residual around both.

  Y  = dyra_forward_varlen(z)          the shared approximated projection, or
       q4_forward(z)                   one with 4-bit weights
  Y += scale (z A^T) B^T               each request's adapter (in place)
  x' = residual_scale x + gate * post(Y),  z' = pre(x')

forward() serves prompts and single tokens alike; backward() gives the
adapters' and norms' gradients for fine-tuning beside the frozen layer.  The
frozen layer passes gradients to its input as the dense weight it stands for,
dz = dY W^T (dyra_dense_ref), which the DyRA output approximates; a 4-bit
projection as itself (q4_backward).  Usage:

    python -m input_adaptive_rank_amd.adapted_block --steps 30 [--base q4] [--loss text]

fine-tunes two adapters on synthetic rows, one bare request among them, towards
a teacher's output, or (text) towards next tokens by the cross entropy of a
frozen head over z' (vocab_loss), and then serves one new token of each request;
prints one JSON line per report.
"""
from __future__ import annotations

import argparse
import json
import sys

import numpy as np
import torch

from . import dyra as D
from . import synth
from .adapters import adapter_backward, adapter_forward
from .block_norm import block_norm_backward, block_norm_forward
from .q4 import Q4Weight, q4_backward, q4_forward, q4_pack, q4_quantise
from .vocab_loss import vocab_loss_backward, vocab_loss_forward


class AdaptedBlock:
    """A square projection (c -> c) with a pool of adapters and the norms around
    it.  layer: a DyraLayer, or a Q4Weight with its bias.  W: the dense weight
    [c][c] behind a DyraLayer, in its storage type, for backward() only."""

    def __init__(self, layer, A, B, pre_weight, post_weight=None, gate=None, rank=None, scale=None, W=None,
                 residual_scale=1.0, eps=1e-6, bias=None):
        self.q4 = isinstance(layer, Q4Weight)
        if bias is not None and not self.q4:
            raise ValueError("a DyraLayer has its own bias")
        self.c = layer.c1 if self.q4 else layer.spec.c1
        if self.c != (layer.c2 if self.q4 else layer.spec.c2):
            raise ValueError("a residual block needs a square layer")
        self.layer, self.A, self.B, self.rank, self.scale, self.W, self.bias = layer, A, B, rank, scale, W, bias
        self.norm = dict(pre="rms", post="none" if post_weight is None else "rms", pre_weight=pre_weight,
                         post_weight=post_weight, gate=gate, residual_scale=residual_scale, eps=eps)

    def _norm_args(self, offsets_dev):
        gate = self.norm["gate"]
        return dict(self.norm, offsets=offsets_dev if gate is not None and gate.dim() == 2 else None)

    def forward(self, x, z, offsets, offsets_dev, slots, keep=False):
        """(x', z', kept): rows of all requests, offsets on the host and (int32)
        on the device, the requests' slots on the device.  keep: what
        backward() needs, else None."""
        layer, n = self.layer, x.shape[0]
        if self.q4:
            Y = q4_forward(z, layer, bias=self.bias)
        else:
            Y = torch.empty((n, layer.spec.c2), dtype=x.dtype, device=x.device)
            need = D.workspace_size_varlen(layer.spec, offsets, layer.dtype, layer.half_steps)
            D.forward_varlen(layer.spec, layer.plan, z, layer.bias, Y, offsets, layer.dtype, layer.eps, layer.solver,
                             torch.empty(need, dtype=torch.uint8, device=x.device), offsets_dev=offsets_dev,
                             half_steps=layer.half_steps)
        out = adapter_forward(z, self.A, self.B, offsets_dev, slots, base=Y, rank=self.rank, scale=self.scale, out=Y,
                              save_h=keep)
        x_new, z_new = block_norm_forward(x, Y, **self._norm_args(offsets_dev))
        return x_new, z_new, (z, Y, out[1], x_new, offsets_dev, slots) if keep else None

    def backward(self, kept, dz_new, dx_new=None):
        """Gradients from those of z' and x': a dict of dx, dz, dA, dB and the
        norms' (d_pre_weight, d_post_weight, d_gate)."""
        z, Y, H, x_new, offsets_dev, slots = kept
        g = block_norm_backward(x_new, Y, dz_new, dx_new, **self._norm_args(offsets_dev))
        if self.q4:
            dz = q4_backward(g["dy"], self.layer)
        else:
            dz = torch.empty_like(z)
            D.dense_ref(g["dy"], self.W, None, dz, self.layer.dtype)
        _, dA, dB = adapter_backward(z, g.pop("dy"), H, self.A, self.B, offsets_dev, slots, dX_base=dz, dX=dz,
                                     rank=self.rank, scale=self.scale)
        return dict(g, dz=dz, dA=dA, dB=dB)


def synthetic_block(c=256, k=64, r=32, rank=16, slots=2, seed=3, device="cuda", base="dyra"):
    """A block of synthetic weights around a low-rank DyRA layer (base "dyra")
    or its dense weight in 4 bits ("q4"): (block, the layer's workload)."""
    if base not in ("dyra", "q4"):
        raise ValueError(f'base must be "dyra" or "q4", got {base!r}')
    w = synth.scaled(synth.WORKLOADS["vitl_fc1"], name="adapted_block", B=2, s=8, c1=c, c2=c, k=k, r=r)
    inp = synth.make_inputs(w)
    if base == "q4":
        # output-major, as a linear layer stores it
        dense = D.to_device(np.ascontiguousarray(inp.W.T), w.dtype, device)
        layer, extra = q4_pack(*q4_quantise(dense)), dict(bias=D.to_device(inp.bias, w.dtype, device))
    else:
        spec = D.spec_of(w)
        layer = D.DyraLayer(spec, D.prepare(inp.W, spec), w.dtype, bias=inp.bias, device=device)
        extra = dict(W=D.to_device(inp.W, w.dtype, device))
    gen = torch.Generator().manual_seed(seed)
    put = lambda t: t.to(device=device, dtype=torch.bfloat16)  # noqa: E731
    A = put(torch.randn((slots, rank, c), generator=gen) / c ** 0.5)
    B = put(torch.zeros((slots, c, rank)))
    ones = put(torch.ones(c))
    block = AdaptedBlock(layer, A, B, pre_weight=ones, post_weight=ones.clone(), gate=put(torch.full((c,), 0.5)),
                         rank=torch.full((slots,), rank, dtype=torch.int32, device=device),
                         scale=torch.full((slots,), 2.0, device=device), **extra)
    return block, w


def output_loss(z_new, target):
    """The mean squared distance of z' from a target, and its gradient."""
    err = z_new.float() - target.float()
    return float(err.square().mean()), (err * (2.0 / err.numel())).to(z_new.dtype)


def text_loss(z_new, head, targets):
    """The mean cross entropy of the tokens that follow, over the rows that have
    one (targets int32, -1: none), by a frozen head [v][c]; and its gradient."""
    loss, lse = vocab_loss_forward(z_new, head, targets)
    live = (targets >= 0) & (targets < head.shape[0])
    count = int(live.sum().clamp(min=1))
    dz, _ = vocab_loss_backward(z_new, head, targets, lse, live.float() / count, need_dw=False)
    return float(loss.sum()) / count, dz


def fine_tune(block, x, z, offsets, offsets_dev, slots, target, steps, lr=2e-2, report=None, head=None):
    """Adam steps on the block's adapters towards target = the wanted z', or
    (with a head) the tokens that follow.  Returns the loss before each step.
    The moments and a master copy of the weights are fp32; the pool holds their
    bf16 values."""
    master = [block.A.float(), block.B.float()]
    m, v = [torch.zeros_like(t) for t in master], [torch.zeros_like(t) for t in master]
    losses = []
    for step in range(1, steps + 1):
        _, z_new, kept = block.forward(x, z, offsets, offsets_dev, slots, keep=True)
        loss, dz_new = output_loss(z_new, target) if head is None else text_loss(z_new, head, target)
        losses.append(loss)
        if report:
            report(step, losses[-1])
        g = block.backward(kept, dz_new)
        for i, (name, pool) in enumerate((("dA", block.A), ("dB", block.B))):
            m[i].mul_(0.9).add_(g[name], alpha=0.1)
            v[i].mul_(0.99).addcmul_(g[name], g[name], value=0.01)
            update = (m[i] / (1 - 0.9 ** step)) / ((v[i] / (1 - 0.99 ** step)).sqrt() + 1e-10)
            master[i].add_(update, alpha=-lr)
            pool.copy_(master[i])
    return losses


def synthetic_requests(c, lens, ids, seed=4, device="cuda"):
    """Rows and requests: x, z (bf16), offsets on host and device, slots."""
    gen = torch.Generator().manual_seed(seed)
    n = int(sum(lens))
    rows = lambda: torch.randn((n, c), generator=gen).to(device=device, dtype=torch.bfloat16)  # noqa: E731
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    return (rows(), rows(), off, torch.from_numpy(off.astype(np.int32)).to(device),
            torch.tensor(ids, dtype=torch.int32, device=device))


def teacher_target(block, x, z, offsets, offsets_dev, slots, seed=5):
    """z' of the same block with other adapters: what fine_tune aims at."""
    gen = torch.Generator(device=x.device).manual_seed(seed)
    A, B = block.A, block.B
    block.A = (torch.randn(A.shape, generator=gen, device=x.device) / A.shape[2] ** 0.5).to(A.dtype)
    block.B = (torch.randn(B.shape, generator=gen, device=x.device) * 0.2).to(B.dtype)
    target = block.forward(x, z, offsets, offsets_dev, slots)[1]
    block.A, block.B = A, B
    return target


def synthetic_text(c, lens, vocab=5003, seed=7, device="cuda"):
    """A head [vocab][c] and the tokens that follow each row; a request's last
    row has none."""
    gen = torch.Generator().manual_seed(seed)
    head = (torch.randn((vocab, c), generator=gen) / c ** 0.5).to(device=device, dtype=torch.bfloat16)
    targets = torch.randint(0, vocab, (int(sum(lens)),), generator=gen, dtype=torch.int32)
    targets[torch.tensor(lens).cumsum(0) - 1] = -1
    return head, targets.to(device)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--base", choices=("dyra", "q4"), default="dyra")
    ap.add_argument("--loss", choices=("output", "text"), default="output")
    args = ap.parse_args(argv)
    block, _ = synthetic_block(c=args.width, base=args.base)
    lens, ids = [120, 37, 200, 64], [0, 1, -1, 1]
    req = synthetic_requests(args.width, lens, ids)
    head, target = synthetic_text(args.width, lens) if args.loss == "text" else (None, teacher_target(block, *req))
    fine_tune(block, *req, target, args.steps, head=head,
              report=lambda step, loss: print(json.dumps({"step": step, "loss": round(loss, 6)}), flush=True)
              if step in (1, args.steps) or step % 10 == 0 else None)
    x, z, off, off_dev, slots = synthetic_requests(args.width, [1] * 4, ids, seed=6)   # one new token of each request
    x_new, z_new, _ = block.forward(x, z, off, off_dev, slots)
    torch.cuda.synchronize()
    print(json.dumps({"decode_rows": x_new.shape[0], "finite": bool(torch.isfinite(z_new).all())}), flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
