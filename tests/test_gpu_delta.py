"""The gated delta rule against its float64 recurrence.

Bounds, with u = 2^-24 one fp32 rounding. Every operand of the products is kept to
2^-22 of the largest of its column, every sum has at most N + 64 terms in fp32, and a
chunk has four products after one another (K S^T, T R, U^T K, and the sums within T):
8 (N + 64) u of the magnitudes that are added covers a chunk, and 2^-13 of them the
chunks together, as each leaves the share e^{sum dt A} of the ones before. Roundings are
of either sign: in the 2-norm a state is off by 4 products x 2^-22 / sqrt(3) x sqrt of
the chunks that are remembered (up to 16): 2^-18. Y's own terms are rounded to one fp16
number (2^-11 of the magnitudes), and Y to its type (half a step).
"""
import numpy as np
import pytest

from oracle import operators_oracle as OO
from tests import _helpers as H

pytestmark = pytest.mark.gpu

DT = {"fp32": "float32", "fp16": "float16", "bf16": "bfloat16"}


def _t(torch, dtype):
    return getattr(torch, DT[dtype])


def _np(t):
    return t.detach().double().cpu().numpy()


def make(torch, seed, B, L, H_, P, N, G, dtype, unit=True, logit=True, cut=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    td = _t(torch, dtype)
    size = 1.0 if unit else 0.8 / N ** 0.5
    c = {"X": r(B, L, H_, P).to(td), "K": (size * r(B, L, G, N)).to(td), "Q": (size * r(B, L, G, N)).to(td)}
    c["dt"] = torch.nn.functional.softplus(r(B, L, H_) - 3).to(td)
    c["A"] = -torch.exp(1.5 * torch.rand(H_, generator=g, device="cuda"))
    wide = r(B, L, 2 * H_ + cut)
    c["beta"] = (wide if logit else torch.sigmoid(wide)).to(td)[..., H_:2 * H_]
    c["init"] = 0.5 * r(B, H_, P, N)
    return c


def reference(c, scale, unit, logit, init, eps=1e-6):
    k, q = _np(c["K"]), _np(c["Q"])
    if unit:
        k, q = OO.unit(k, eps), OO.unit(q, eps)
    beta = OO.sigmoid(_np(c["beta"])) if logit else _np(c["beta"])
    s0 = _np(c["init"])
    return OO.delta(_np(c["X"]), _np(c["dt"]), _np(c["A"]), k, q, beta, scale, s0 if init else np.zeros_like(s0))


def check(got, ref, mag, dtype, tau, norm, what):
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref) - H.half_ulp(got, dtype)
    bad = ~(err <= tau * mag + 1e-30)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(err / (tau * mag + 1e-30)):.3g} of the bound"
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert rel <= norm, f"{what}: {rel:.3g} in the 2-norm, bound {norm:.3g}"


Y_TAU = {"fp32": 2.0 ** -13, "fp16": 2.0 ** -10, "bf16": 2.0 ** -10}
Y_NORM = {"fp32": 2.0 ** -18, "fp16": 2.0 ** -11 + 2.0 ** -18, "bf16": 2.0 ** -8}

CASES = [
    # B, L, H, P, N, G, dtype, unit, logit, initial state, beta's cut
    (1, 1, 4, 16, 16, 1, "fp16", True, True, True, 0),
    (2, 2, 3, 32, 32, 1, "bf16", True, False, True, 1),
    (1, 16, 2, 128, 64, 1, "fp32", False, True, True, 3),
    (1, 17, 2, 64, 128, 2, "fp32", True, True, False, 0),
    (1, 63, 3, 16, 16, 3, "fp32", True, True, True, 1),
    (2, 64, 4, 32, 32, 2, "fp16", True, False, True, 0),
    (1, 65, 6, 64, 64, 2, "bf16", True, True, True, 5),
    (3, 130, 5, 128, 128, 1, "bf16", True, True, True, 0),
    (2, 200, 8, 64, 128, 1, "fp16", False, True, True, 0),
    (1, 700, 4, 64, 128, 4, "fp16", True, True, True, 0),
    (2, 333, 9, 16, 64, 3, "bf16", False, False, False, 7),
    (1, 400, 2, 128, 16, 1, "fp32", True, True, True, 0),
    (1, 150, 2, 32, 64, 1, "fp32", False, True, True, 0),
    (1, 129, 3, 32, 32, 1, "fp32", True, True, True, 0),
    (1, 129, 20, 16, 32, 1, "bf16", True, True, True, 0),
    # heads enough for the wider slices, and more of a group's than a workgroup takes at a time
    (8, 70, 128, 32, 16, 2, "fp16", True, True, True, 0),
    (5, 66, 128, 64, 32, 1, "bf16", True, True, False, 0),
    (8, 65, 64, 64, 64, 64, "fp16", True, False, True, 0),
    (4, 67, 72, 128, 128, 8, "bf16", True, True, True, 0),
    (4, 65, 70, 128, 128, 1, "fp16", True, True, True, 0),
    (9, 65, 64, 64, 128, 1, "fp32", True, True, True, 0),
    (2, 40, 520, 32, 16, 1, "fp32", True, True, True, 0),
    (8, 33, 128, 32, 32, 128, "fp32", False, False, True, 0),
    (8, 18, 128, 32, 64, 1, "fp32", True, True, True, 0),
    # few positions of many heads: chunks from 9 positions on
    (16, 8, 64, 64, 128, 1, "fp16", True, True, True, 0),
    (16, 9, 64, 64, 128, 1, "fp16", True, True, True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_delta_forward(gpu_lib, case):
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G, dtype, unit, logit, init, cut = case
    print("delta", case, flush=True)
    c = make(torch, 7, B, Ln, H_, P, N, G, dtype, unit, logit, cut)
    sh = L.make_shape(B, Ln, H_, P, N, G, 64, dtype)
    Y = torch.full((B, Ln, H_, P), float("nan"), dtype=_t(torch, dtype), device="cuda")
    fin = torch.full((B, H_, P, N), float("nan"), device="cuda")
    ws = L.ssd_delta_workspace(sh)
    if ws is not None:
        ws.fill_(0xff)
    scale = N ** -0.5
    L.ssd_delta_forward(sh, c["X"], c["dt"], c["A"], c["K"], c["Q"], c["beta"], Y, final_state=fin,
                        initial_state=c["init"] if init else None, workspace=ws, scale=scale, unit=unit, logit=logit)
    torch.cuda.synchronize()
    y, s, ymag, smag = reference(c, scale, unit, logit, init)
    check(_np(fin), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
    check(_np(Y), y, ymag, dtype, Y_TAU[dtype], Y_NORM[dtype], "y")


@pytest.mark.parametrize("case", [(2, 40, 8, 32, 64, 1), (1, 64, 6, 64, 128, 2), (1, 130, 4, 128, 32, 1)],
                         ids=lambda c: "-".join(map(str, c)))
def test_delta_fp16_outputs_are_rounded_once(gpu_lib, case):
    """Y's terms are kept to 2^-15 (the weights' second part), so that what is lost is the
    rounding to fp16: a value that is d off before it goes to the other neighbour, a step s
    <= 2^-10 |y| away, with probability |d| / s, and the differences from the rounded exact
    values have a mean square of |d| s <= 2^-25 y^2. (One part alone, 2^-12 of a term, would
    give 2^-22.)"""
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G = case
    print("delta", case, flush=True)
    c = make(torch, 51, B, Ln, H_, P, N, G, "fp16")
    sh = L.make_shape(B, Ln, H_, P, N, G, 64, "fp16")
    Y = torch.empty(B, Ln, H_, P, dtype=torch.float16, device="cuda")
    L.ssd_delta_forward(sh, c["X"], c["dt"], c["A"], c["K"], c["Q"], c["beta"], Y, initial_state=c["init"], scale=0.3,
                        logit=True)
    torch.cuda.synchronize()
    y = reference(c, 0.3, True, True, True)[0]
    off = np.linalg.norm(_np(Y) - y.astype(np.float16).astype(np.float64)) / np.linalg.norm(y)
    assert off <= 2.0 ** -12.5, off


@pytest.mark.parametrize("case", [(1, 64, 64, 128, 1, "bf16"), (3, 5, 16, 16, 5, "fp16"), (2, 6, 128, 128, 2, "fp32"),
                                  (70, 80, 64, 128, 1, "fp16"), (600, 7, 32, 64, 1, "bf16"), (257, 33, 16, 32, 3, "fp32"),
                                  (40, 64, 128, 16, 1, "fp32")], ids=lambda c: "-".join(map(str, c)))
def test_delta_step(gpu_lib, case):
    import torch
    L = gpu_lib
    B, H_, P, N, G, dtype = case
    print("delta step", case, flush=True)
    c = make(torch, 9, B, 1, H_, P, N, G, dtype)
    sh = L.make_shape(B, 1, H_, P, N, G, 64, dtype)
    state, Y = c["init"].clone(), torch.empty(B, H_, P, dtype=_t(torch, dtype), device="cuda")
    L.ssd_delta_step(sh, c["X"][:, 0], c["dt"][:, 0], c["A"], c["K"][:, 0], c["Q"][:, 0], c["beta"][:, 0], state, Y,
                     scale=0.3, logit=True)
    y, s, ymag, smag = reference(c, 0.3, True, True, True)
    # the sums of a row cross N / 4 lanes: N u of the magnitudes
    check(_np(state), s, smag, "fp32", 2.0 ** -16, 2.0 ** -21, "state")
    check(_np(Y), y[:, 0], ymag[:, 0], dtype, 2.0 ** -16, {"fp32": 2.0 ** -21}.get(dtype, Y_NORM[dtype]), "y")
