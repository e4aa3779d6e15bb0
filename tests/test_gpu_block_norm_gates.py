"""Gates of the block norm on their own: rows of +-1 have a root mean square of exactly 1, so
that r is the gate's value."""
import numpy as np
import pytest

from oracle import operators_oracle as OO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


@pytest.mark.parametrize("act,code", (("silu", 3), ("sigmoid", 4)))
@pytest.mark.parametrize("dtype", ("float32", "float16", "bfloat16"))
@pytest.mark.parametrize("cols", (64, 1021, 4096))
def test_gate_values(gpu_lib, cols, dtype, act, code):
    """A gate is its function's value to 9 roundings (and one of the product with u, which is +-1:
    none), from 16 bits as from 32, over all of the range in which fp32 holds it."""
    import torch
    td = getattr(torch, dtype)
    z = torch.linspace(-85, 85, 3 * cols, device="cuda").view(3, cols).to(td)
    x = torch.ones(3, cols, device="cuda")
    x[:, ::3] = -1
    one, r = torch.ones(cols, device="cuda"), torch.empty(3, cols, device="cuda")
    gpu_lib.ssd_block_norm(x.to(td), one, None, r, None, 0.0, gate=z, gate_act=code)
    ref = OO.activation(z.double().cpu().numpy(), act) * x.double().cpu().numpy()
    err = np.abs(r.double().cpu().numpy() - ref)
    assert (err <= 9 * U * np.abs(ref)).all(), np.max(err / np.abs(ref)) / U


@pytest.mark.parametrize("dtype", ("float32", "float16", "bfloat16"))
def test_gates_at_infinity(gpu_lib, dtype):
    """Infinite gates have their functions' limits, and NaN stays NaN."""
    import torch
    td = getattr(torch, dtype)
    z = torch.zeros(4, 64, dtype=td, device="cuda")
    z[1], z[2], z[3] = INF, -INF, float("nan")
    x, one, r = torch.ones(4, 64, dtype=td, device="cuda"), torch.ones(64, device="cuda"), torch.empty(4, 64, device="cuda")
    for code, want in ((3, (0.0, INF, 0.0)), (4, (0.5, 1.0, 0.0))):
        gpu_lib.ssd_block_norm(x, one, None, r, None, 0.0, gate=z, gate_act=code)
        for row, v in enumerate(want):
            assert (r[row] == v).all(), (code, row, r[row, 0])
        assert torch.isnan(r[3]).all()
