"""Nothing behind a workspace of exactly the size asked for is written by the 4-bit
projection, and what lies in it before a call does not matter."""
import pytest

from input_adaptive_rank_amd import dyra as D
from input_adaptive_rank_amd import synth

from test_gpu_q4 import make, pack, put

pytestmark = pytest.mark.gpu

F32, BF16 = synth.DT_F32, synth.DT_BF16
IDS = {F32: "fp32", BF16: "bf16"}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)
@pytest.mark.parametrize("n,c1,c2", [(1, 264, 520), (65, 2056, 776), (700, 1032, 2048), (1031, 1024, 1024), (4099, 520, 4104)])
def test_nothing_behind_the_workspace_is_written(n, c1, c2, dtype):
    import torch
    from input_adaptive_rank_amd import q4 as Q
    c = make(n, c1, c2, 64, True, dtype, seed=43)
    w, X, dY = pack(c), put(c["X"], dtype), put(c["dY"], dtype)
    for back, call, x in ((False, Q.q4_forward, X), (True, Q.q4_backward, dY)):
        size = Q.q4_workspace_size(c1, c2, n, dtype, back)
        want = call(x, w)
        for byte in (90, 255):   # 255: NaN in either type
            ws = torch.full((size + (1 << 23),), byte, dtype=torch.uint8, device="cuda")
            assert torch.equal(call(x, w, workspace=ws), want)
            assert bool((ws[size:] == byte).all())
