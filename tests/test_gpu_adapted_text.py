"""A block around a 4-bit projection with adapters and norms, fine-tuned by the
vocabulary loss of a frozen head: values and gradients against the float64 oracles
on the same weights, and against differences."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D
from oracle import adapter_oracle, block_norm_oracle, q4_oracle, vocab_loss_oracle

from gpu_cases import log

pytestmark = pytest.mark.gpu

LENS, IDS, C, VOCAB = [120, 37, 200, 64], [0, 1, -1, 1], 256, 515


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def rel(a, b):
    return float(np.linalg.norm(host(a) - b) / np.linalg.norm(b))


def setup():
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    from input_adaptive_rank_amd import q4
    block, _ = AB.synthetic_block(c=C, base="q4")
    gen = torch.Generator(device="cuda").manual_seed(1)
    block.B.copy_(torch.randn(block.B.shape, generator=gen, device="cuda") * 0.2)
    W = q4.q4_dense(block.layer, torch.float32).double().cpu().numpy()
    return AB, block, W, AB.synthetic_requests(C, LENS, IDS), AB.synthetic_text(C, LENS, VOCAB)


def params(block):
    return dict(pre_weight=host(block.norm["pre_weight"]), pre_bias=None, post_weight=host(block.norm["post_weight"]),
                post_bias=None, gate=host(block.norm["gate"]))


def oracle_loss(block, W, req, head, targets, A, B):
    """The mean loss of the block in float64, and what a backward pass needs."""
    x, z, off, _, _ = req
    pool = dict(rank=block.rank.cpu().numpy(), scale=block.scale.cpu().numpy())
    base = q4_oracle.forward(host(z), W, host(block.bias))[0]
    Y, H, _, _ = adapter_oracle.forward(host(z), A, B, off, IDS, base=base, **pool)
    x_new, z_new = block_norm_oracle.forward(host(x), Y, "rms", "rms", params(block))
    loss, lse, _ = vocab_loss_oracle.forward(z_new, host(head), targets.cpu().numpy())
    count = int((targets.cpu().numpy() >= 0).sum())
    return loss.sum() / count, dict(Y=Y, H=H, x_new=x_new, z_new=z_new, lse=lse, count=count, pool=pool)


def test_loss_and_gradients_match_the_oracles():
    """Relative Frobenius errors: each bf16 result of the chain (Y, x', z', dz',
    dY, dz) adds at most 2^-8 of itself and no more than six follow one
    another; the loss's own gradient rounds d beside them."""
    AB, block, W, req, (head, targets) = setup()
    x, z, off, off_dev, slots = req
    x_new, z_new, kept = block.forward(*req, keep=True)
    loss, dz_new = AB.text_loss(z_new, head, targets)
    g = block.backward(kept, dz_new)
    A, B = host(block.A), host(block.B)
    want, k = oracle_loss(block, W, req, head, targets, A, B)
    log(f"    loss {loss:.6f}, oracle {want:.6f}")
    assert abs(loss - want) <= 2.0 ** -8 * abs(want)
    t = targets.cpu().numpy()
    dl = (t >= 0) / k["count"]
    dz_want, _, _, _ = vocab_loss_oracle.backward(k["z_new"], host(head), t, k["lse"], dl)
    n = block_norm_oracle.backward(k["x_new"], k["Y"], dz_want, None, "rms", "rms", params(block))
    dz, dA, dB, _, _, _ = adapter_oracle.backward(host(z), n["dy"], k["H"], A, B, off, IDS, dX_base=n["dy"] @ W, **k["pool"])
    for name, got, exact in (("dz_new", dz_new, dz_want), ("dz", g["dz"], dz), ("dA", g["dA"], dA), ("dB", g["dB"], dB),
                             ("d_gate", g["d_gate"], n["d_gate"]), ("dx", g["dx"], n["dx"])):
        log(f"    {name}: relative error {rel(got, exact):.2e}")
        assert rel(got, exact) <= 7 * 2.0 ** -8, name
    assert not bool(dz_new[targets < 0].any())


def test_adapter_gradients_match_differences():
    """Along random directions of A and B, fourth order differences of the
    float64 loss: within the chain's roundings (seven of 2^-8) of the sum of the
    magnitudes."""
    AB, block, W, req, (head, targets) = setup()
    _, z_new, kept = block.forward(*req, keep=True)
    g = block.backward(kept, AB.text_loss(z_new, head, targets)[1])
    A, B = host(block.A), host(block.B)
    rng = np.random.default_rng(4)
    for i, dev in enumerate((host(g["dA"]), host(g["dB"]))):
        step = rng.standard_normal(dev.shape)

        def at(s):
            moved = [A, B]
            moved[i] = moved[i] + s * step
            return oracle_loss(block, W, req, head, targets, *moved)[0]

        h = 1e-4
        slope = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
        log(f"    difference {slope:.6f}, gradient {(dev * step).sum():.6f}")
        assert abs(slope - (dev * step).sum()) <= 7 * 2.0 ** -8 * np.abs(dev * step).sum()


@pytest.mark.parametrize("base", ["dyra", "q4"])
def test_fine_tuning_by_text_runs(base):
    """A few steps leave a bare request's rows what they were and move the
    others; then single tokens."""
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    block, _ = AB.synthetic_block(c=C, base=base)
    req = AB.synthetic_requests(C, LENS, IDS)
    head, targets = AB.synthetic_text(C, LENS, VOCAB)
    before = block.forward(*req)[1]
    losses = AB.fine_tune(block, *req, targets, 3, head=head)
    after = block.forward(*req)[1]
    assert len(losses) == 3 and np.isfinite(losses).all()
    bare = slice(157, 357)   # the third request
    assert torch.equal(before[bare], after[bare]) and not torch.equal(before[:120], after[:120])
    x, z, off, off_dev, slots = AB.synthetic_requests(C, [1] * 4, IDS, seed=6)
    x_new, z_new, _ = block.forward(x, z, off, off_dev, slots)
    assert torch.isfinite(x_new).all() and torch.isfinite(z_new).all()


def test_command_runs(capsys):
    import json

    from input_adaptive_rank_amd import adapted_block as AB
    assert AB.main(["--steps", "2", "--base", "q4", "--loss", "text"]) == 0
    lines = [json.loads(line) for line in capsys.readouterr().out.splitlines()]
    assert lines[-1] == {"decode_rows": 4, "finite": True} and lines[0]["step"] == 1


def test_refusals():
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    from input_adaptive_rank_amd import q4
    with pytest.raises(ValueError, match="base must be"):
        AB.synthetic_block(c=C, base="q8")
    wide = q4.q4_pack(torch.zeros((64, 64), dtype=torch.uint8, device="cuda"),
                      torch.zeros((64, 1), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="square"):
        AB.AdaptedBlock(wide, None, None, None)
