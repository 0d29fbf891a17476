"""A layer's calls on another stream than the current one (they order nothing
between the two but by what they allocate)."""
import numpy as np
import pytest

from input_adaptive_rank_amd import dyra as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    D.lib()


@pytest.mark.parametrize("ragged", [True, False], ids=["ragged", "uniform"])
def test_other_work_on_the_current_stream(ragged):
    """The call waits behind some 70 ms of its own stream's work while the
    current one fills blocks of every size that the call may have freed; before
    it, blocks just freed there have readers still to run."""
    import torch
    from input_adaptive_rank_amd import adapted_block as AB
    block, _ = AB.synthetic_block(c=256)
    layer, n = block.layer, 4096
    X = torch.randn((n, 256), device="cuda").bfloat16()
    off = np.array([0, 1000, 1007, 4096])
    call = lambda **kw: layer.forward_varlen(X, off, **kw)[0] if ragged else layer.forward(X, 4, n // 4, **kw)  # noqa: E731
    want = call().clone()
    need = (D.workspace_size_varlen(layer.spec, off, layer.dtype) if ragged else
            D.workspace_size(layer.spec, 4, n // 4, layer.dtype))
    layer._ws = layer._ws_key = None
    a, s = torch.randn((4096, 4096), device="cuda"), torch.cuda.Stream()
    b = [torch.empty_like(a) for _ in range(2)]
    sizes = [2 * n * 256, need, 16]
    old = [torch.full((size,), 3, dtype=torch.uint8, device="cuda") for size in sizes]
    kept = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    for _ in range(50):
        torch.mm(a, a, out=b[0])
    for t, k in zip(old, kept):
        torch.add(t, 1, out=k)
    del t, old
    with torch.cuda.stream(s):
        for _ in range(50):
            torch.mm(a, a, out=b[1])
    got = call(stream=s)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for size in sizes]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((k == 4).all()) for k in kept) and all(bool((t == 255).all()) for t in junk)
