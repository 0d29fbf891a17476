"""The layer, adapters and norms run together as a block: one forward and
backward against the float64 oracles on the device's own layer output, and a
short fine-tuning that has to approach its teacher."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from oracle import adapter_oracle, block_norm_oracle

from gpu_cases import log

pytestmark = pytest.mark.gpu

LENS, IDS, C = [120, 37, 200, 64], [0, 1, -1, 1], 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rel(a, b):
    return float(np.linalg.norm(host(a) - b) / np.linalg.norm(b))


def test_block_matches_the_oracles():
    """Relative Frobenius errors within 2^-7: each bf16 result of the chain
    (layer output, Y, x', z', dY, dz) adds at most 2^-9 of itself, and no
    more than four of them follow one another."""
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    block, _ = AB.synthetic_block(c=C)
    gen = torch.Generator(device="cuda").manual_seed(1)
    block.B.copy_(torch.randn(block.B.shape, generator=gen, device="cuda") * 0.2)
    req = AB.synthetic_requests(C, LENS, IDS)
    x, z, off, off_dev, slots = req
    A, B = host(block.A), host(block.B)
    pool = dict(rank=block.rank.cpu().numpy(), scale=block.scale.cpu().numpy())
    with_b = block.B.clone()
    block.B.zero_()
    base = host(block.forward(x, z, off, off_dev, slots, keep=True)[2][1])   # the layer's own output
    block.B.copy_(with_b)
    x_new, z_new, kept = block.forward(*req, keep=True)
    Y, H, _, _ = adapter_oracle.forward(host(z), A, B, off, IDS, base=base, **pool)
    par = dict(pre_weight=host(block.norm["pre_weight"]), pre_bias=None, post_weight=host(block.norm["post_weight"]),
               post_bias=None, gate=host(block.norm["gate"]))
    wx, wz = block_norm_oracle.forward(host(x), Y, "rms", "rms", par)
    dz_new = torch.randn(z_new.shape, generator=gen, device="cuda").bfloat16()
    g = block.backward(kept, dz_new)
    want = block_norm_oracle.backward(wx, Y, host(dz_new), None, "rms", "rms", par)
    dz_base = want["dy"] @ host(block.W).T
    dz, dA, dB, _, _, _ = adapter_oracle.backward(host(z), want["dy"], H, A, B, off, IDS, dX_base=dz_base, **pool)
    got = dict(x_new=(x_new, wx), z_new=(z_new, wz), dx=(g["dx"], want["dx"]), dz=(g["dz"], dz), dA=(g["dA"], dA),
               dB=(g["dB"], dB), d_gate=(g["d_gate"], want["d_gate"]),
               d_pre_weight=(g["d_pre_weight"], want["d_pre_weight"]),
               d_post_weight=(g["d_post_weight"], want["d_post_weight"]))
    for k, (a, b) in got.items():
        log(f"    {k}: relative error {rel(a, b):.2e}")
    assert all(rel(a, b) <= 2.0 ** -7 for a, b in got.values())


def test_fine_tuning_approaches_the_teacher():
    """Adapters that start at zero halve their distance to the teacher's
    output within 30 steps; a bare request's rows stay what they were."""
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    block, _ = AB.synthetic_block(c=C)
    req = AB.synthetic_requests(C, LENS, IDS)
    target = AB.teacher_target(block, *req)
    before = block.forward(*req)[1]
    losses = AB.fine_tune(block, *req, target, 30)
    after = block.forward(*req)[1]
    log(f"    loss {losses[0]:.5f} -> {losses[-1]:.5f}")
    assert losses[-1] < 0.5 * losses[0]
    bare = slice(157, 357)   # the third request
    assert torch.equal(before[bare], after[bare]) and torch.equal(before[bare], target[bare])
    x, z, off, off_dev, slots = AB.synthetic_requests(C, [1] * 4, IDS, seed=6)
    x_new, z_new, _ = block.forward(x, z, off, off_dev, slots)
    assert torch.isfinite(x_new).all() and torch.isfinite(z_new).all()
