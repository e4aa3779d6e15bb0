"""The product with bias, activation and residual against its float64 definition.

Bounds, with u = 2^-24: a sum of K products of 16-bit elements (exact in fp32) has at
most K roundings of partial sums no larger than sum |a w| (fp32 products add one);
activations have a slope of at most 1.13 (RELU2: 2 |v|), and cost (v^2 / 2 + 16) u of
their value; then the residual's addition, and half a step of the output's type.
"""
import numpy as np
import pytest

from oracle import operators_oracle as OO
from tests import _helpers as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": "float32", "fp16": "float16", "bf16": "bfloat16"}
ACTS = ("none", "relu", "relu2", "silu", "sigmoid", "gelu", "gelu_tanh")


def _np(t):
    return t.detach().double().cpu().numpy()


def run(L, torch, M, N, K, dtype, out, act, bias, residual, cut, seed=3, same=False, room_for=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    td, to = getattr(torch, DT[dtype]), getattr(torch, DT[out])
    wide = r(M, K + cut + (0 if not cut else 3 if cut % 8 else 8)).to(td)  # cut of whole 16 bytes: rows stay aligned
    a, w = wide[:, cut:cut + K], (2 * r(N, K) / K ** 0.5).to(td)
    b = r(N) if bias else None
    res = (2 * r(M, N)).to(to) if residual else None
    # the output's neighbours stay as they are
    room = torch.full((M * N + 64,), 7.0, dtype=to, device="cuda")
    o = room[:M * N].view(M, N)
    o.fill_(float("nan"))
    if same and residual:
        o.copy_(res)
    ws = L.ssd_matmul_workspace(a, w, o) if room_for else None
    if room_for:
        assert (ws is None) == (dtype == "fp32")  # fp32 rows have no use for one
        if ws is not None:
            ws.fill_(0xff)  # NaN
    L.ssd_matmul(a, w, b, o, act=ACTS.index(act), residual=o if same and residual else res, workspace=ws)
    torch.cuda.synchronize()
    A, W = _np(a), _np(w)
    v = A @ W.T
    mag = np.abs(A) @ np.abs(W).T
    if bias:
        v, mag = v + _np(b), mag + np.abs(_np(b))
    y = OO.activation(v, act)
    slope = np.maximum(2 * np.abs(v), 1.0) if act == "relu2" else 1.13
    bound = slope * (K + 2) * U * mag + np.abs(y) * (v * v / 2 + 16) * U
    if act == "relu2":
        bound += ((K + 2) * U * mag) ** 2
    if residual:
        y = y + _np(res)
        bound += np.abs(y) * U
    got = _np(o)
    err = np.abs(got - y) - H.half_ulp(got, out)
    bad = ~(err <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.nanmax(err / (bound + 1e-300)):.3g} of the bound"
    assert (room[M * N:] == 7).all()


CASES = [
    # M, N, K, dtype, out, act, bias, residual, cut
    (1, 1, 1, "fp32", "fp32", "none", True, True, 0),
    (1, 16, 64, "fp16", "fp16", "none", False, False, 0),
    (3, 17, 33, "bf16", "bf16", "silu", True, True, 1),
    (8, 2560, 5120, "fp16", "fp16", "none", False, True, 0),
    (5, 96, 4104, "bf16", "fp32", "gelu", True, True, 8),
    (16, 40, 700, "fp32", "fp32", "gelu_tanh", True, False, 2),
    (20, 61, 1111, "fp16", "fp32", "sigmoid", True, True, 0),
    (31, 130, 70, "fp32", "fp32", "relu2", False, True, 3),
    (33, 65, 65, "bf16", "bf16", "relu", True, True, 5),
    (70, 200, 300, "fp16", "fp16", "relu2", True, False, 1),
    (64, 1064, 2560, "fp16", "fp16", "silu", True, True, 0),
    (333, 1000, 512, "bf16", "bf16", "gelu", True, True, 64),
    (333, 1064, 1048, "fp16", "fp32", "none", True, True, 16),
    (300, 700, 90, "fp32", "fp32", "silu", True, True, 0),
    (257, 515, 96, "fp32", "fp32", "gelu", False, True, 0),
    (1100, 1300, 136, "bf16", "fp32", "gelu_tanh", True, True, 0),
    (1024, 4096, 256, "fp16", "fp16", "sigmoid", False, True, 0),
    (2100, 4099, 264, "bf16", "bf16", "silu", True, True, 0),
    (4100, 4096, 512, "fp16", "fp16", "gelu", True, True, 0),
    (4100, 4101, 520, "fp16", "fp32", "none", True, True, 8),
    (3000, 4104, 129, "bf16", "bf16", "relu", True, True, 0),
    (2049, 2304, 128, "fp32", "fp32", "none", True, True, 0),
    (3000, 3500, 77, "fp32", "fp32", "none", False, True, 0),
    (32, 4099, 129, "bf16", "bf16", "silu", True, True, 0),
    (17, 9000, 67, "fp16", "fp32", "relu", True, True, 1),
    (100, 1001, 515, "fp32", "fp32", "gelu", True, True, 0),
    (65, 9001, 131, "fp32", "fp32", "silu", True, True, 2),
]


@pytest.mark.parametrize("same", (False, True), ids=("apart", "in_place"))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matmul(gpu_lib, case, same):
    import torch
    print("product", case, same, flush=True)
    run(gpu_lib, torch, *case, same=same)


# aligned rows that reach every kernel of the 16-bit dispatch (K in bytes halved)
SIZES = [(333, 8512, 1024), (1, 16, 1024), (1, 3870, 256), (3, 4281, 768), (2, 4427, 536), (1, 5236, 1544), (16, 9000, 1800), (2245, 33, 256),
         (2140, 33, 8), (18, 3004, 776), (103, 6937, 264), (99, 7287, 512), (41, 11479, 808), (333, 2560, 2560),
         (333, 2560, 2568), (333, 8512, 1032), (384, 3864, 432), (4099, 2571, 2568), (3000, 10576, 520), (687, 11060, 768),
         (1790, 4864, 2512), (900, 4608, 768), (2600, 2570, 128), (2100, 2600, 512), (4100, 4120, 1024), (4100, 8200, 640)]
KERNELS = [(m, n, k, ("fp16", "bf16")[i % 2], ("fp16", "bf16")[i % 2] if i % 3 else "fp32", ACTS[i % 7], i % 2 == 0, True,
            (0, 8)[i % 4 == 3]) for i, (m, n, k) in enumerate(SIZES)]


@pytest.mark.parametrize("case", KERNELS, ids=lambda c: "-".join(map(str, c)))
def test_matmul_every_kernel(gpu_lib, case):
    import torch
    print("product", case, flush=True)
    run(gpu_lib, torch, *case)
    run(gpu_lib, torch, *case, same=True)


# rows of no alignment that are copied into aligned ones: both operands, and a alone
PACKED = [
    (64, 200, 300, "fp16", "fp16", "relu2", True, False, 1),
    (64, 1, 65, "bf16", "fp32", "none", False, False, 0),
    (333, 1000, 512, "bf16", "bf16", "gelu", True, True, 3),
    (1100, 1300, 135, "bf16", "fp32", "gelu_tanh", True, True, 0),
    (4100, 4101, 515, "fp16", "fp32", "none", True, True, 7),
    (300, 700, 91, "fp32", "fp32", "silu", True, True, 1),
    (257, 514, 64, "fp32", "fp32", "gelu", False, True, 5),
    (4, 130, 1001, "bf16", "bf16", "silu", True, True, 0),
    (9, 4099, 519, "fp16", "fp16", "none", True, True, 3),
    (17, 61, 77, "bf16", "fp32", "gelu", True, True, 1),
    (40, 2600, 1031, "fp16", "fp32", "sigmoid", False, True, 0),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "-".join(map(str, c)))
def test_matmul_with_room_for_aligned_rows(gpu_lib, case):
    import torch
    print("packed product", case, flush=True)
    run(gpu_lib, torch, *case, room_for=True)
    run(gpu_lib, torch, *case, room_for=True, same=True)
