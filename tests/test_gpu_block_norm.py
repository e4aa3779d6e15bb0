"""The norms between two blocks against their float64 definition.

Bounds, with u = 2^-24: a norm's sum of squares adds at most 40 roundings in any path
through its tree, half of which reach 1 / rms, and with the products 64 u covers it; a
gate read from 16 bits is within 2 (|z| + 8) u of its value, one from 32 within 20 u.
What r is off by enters y directly and through the mean: |dr| + |r| |dr|_2 / |r|_2.
Codes: half a step on top.
"""
import numpy as np
import pytest

from oracle import operators_oracle as OO
from tests import _helpers as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": "float32", "fp16": "float16", "bf16": "bfloat16"}


def _np(t):
    return t.detach().double().cpu().numpy()


def inputs(torch, rows, cols, dtype, res, gate, cut=0, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    td = getattr(torch, DT[dtype])
    c = {"x": (2 * r(rows, cols + 2 * cut)).to(td)[:, cut:cut + cols], "post": 1 + 0.2 * r(cols), "w": 1 + 0.2 * r(cols)}
    rt = {"none": None, "same": td, "fp32": torch.float32}[res]
    c["res"] = (3 * r(rows, cols)).to(rt) if rt is not None else None
    c["rt"] = rt if rt is not None else td
    per = {"none": 1, "token": 1, "all": rows, "three": 3}[gate]
    c["per"] = per
    c["gate"] = None if gate == "none" else r(-(-rows // per), cols + 2 * cut).to(td)[:, cut:cut + cols]
    return c


def reference(c, act, res_scale, dtype, eps=1e-5):
    x = _np(c["x"])
    z = np.ones_like(x) if c["gate"] is None else np.repeat(_np(c["gate"]), c["per"], 0)[:x.shape[0]]
    gate = z if c["gate"] is None else OO.activation(z, act)
    res = np.zeros_like(x) if c["res"] is None else _np(c["res"])
    r, y = OO.block_norm(x, _np(c["post"]), gate, res, res_scale, _np(c["w"]), eps)
    part = np.abs(r - res_scale * res)
    dr = part * U * (64 + (20 if dtype == "fp32" else 2 * (np.abs(z) + 8))) + 2 * U * np.abs(res_scale * res) + U * np.abs(r)
    n = np.sqrt((r * r).sum(-1, keepdims=True))
    rel = np.sqrt((dr * dr).sum(-1, keepdims=True)) / np.where(n > 0, n, 1)
    dy = (dr + np.abs(r) * rel) * OO.rms(r, eps) * np.abs(_np(c["w"])) + 64 * U * np.abs(y)
    return r, y, dr, dy


def within(got, ref, bound, dtype, what):
    err = np.abs(got - ref) - H.half_ulp(got, dtype)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(err / (bound + 1e-300)):.3g} of the bound"


def name_of(torch, t):
    return {torch.float32: "fp32", torch.float16: "fp16", torch.bfloat16: "bf16"}[t]


CASES = [
    # rows, cols, dtype, residual, gate, act, codes, cut
    (1, 1, "fp32", "same", "token", "none", False, 0),
    (3, 7, "bf16", "fp32", "all", "silu", True, 0),
    (5, 40, "fp16", "same", "three", "sigmoid", True, 1),
    (8, 2560, "fp16", "same", "all", "none", True, 0),
    (9, 512, "bf16", "fp32", "token", "sigmoid", True, 8),
    (130, 320, "fp32", "same", "token", "silu", False, 4),
    (67, 777, "bf16", "same", "token", "silu", False, 3),
    (16, 4096, "bf16", "fp32", "three", "none", True, 0),
    (5, 5000, "fp16", "fp32", "none", "none", False, 0),
    (4, 8191, "bf16", "none", "token", "sigmoid", True, 0),
    (3, 9000, "fp32", "fp32", "all", "silu", False, 0),
    (2, 16384, "fp16", "same", "token", "sigmoid", True, 0),
    (2, 16383, "fp32", "none", "none", "none", False, 1),
    (300, 64, "fp16", "none", "none", "none", True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_block_norm(gpu_lib, case):
    import torch
    L = gpu_lib
    rows, cols, dtype, res, gate, act, codes, cut = case
    print("block norm", case, flush=True)
    c = inputs(torch, rows, cols, dtype, res, gate, cut)
    td = getattr(torch, DT[dtype])
    nan = float("nan")
    out = torch.full((rows, cols), nan, dtype=td, device="cuda")
    kept = torch.full((rows, cols), nan, dtype=c["rt"], device="cuda")
    q = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda") if codes else None
    step = torch.full((rows,), nan, device="cuda") if codes else None
    kw = dict(gate=c["gate"], gate_act=OO_ACT[act], rows_per_gate=c["per"], res_scale=0.75)
    L.ssd_block_norm(c["x"], c["post"], c["res"], kept, c["w"], 1e-5, out, q, step, **kw)
    torch.cuda.synchronize()
    r, y, dr, dy = reference(c, act, 0.75, dtype)
    within(_np(kept), r, dr, name_of(torch, c["rt"]), "r")
    if not codes:
        within(_np(out), y, dy, dtype, "y")
    else:
        s = np.abs(y).max(-1) / 127
        ds = dy.max(-1) / 127 + 2 * U * s
        assert (np.abs(_np(step) - s) <= ds).all()
        v = _np(q) * _np(step)[:, None]
        assert (np.abs(v - y) <= _np(step)[:, None] * (0.5 + 2 * U * 127) + dy).all()
        within(_np(out), v, 2 * U * np.abs(v), dtype, "values of the codes")
    # in place: r over the residual, y over x
    if c["res"] is not None and not cut:
        x2, r2 = c["x"].clone(), c["res"].clone()
        L.ssd_block_norm(x2, c["post"], r2, r2, c["w"], 1e-5, x2, q, step, **kw)
        assert torch.equal(x2, out) and torch.equal(r2, kept)
    # r alone, and y alone
    only = torch.full((rows, cols), nan, dtype=c["rt"], device="cuda")
    L.ssd_block_norm(c["x"], c["post"], c["res"], only, None, 1e-5, **kw)
    assert torch.equal(only, kept)
    if c["res"] is not None:
        alone = torch.full((rows, cols), nan, dtype=td, device="cuda")
        L.ssd_block_norm(c["x"], c["post"], c["res"], None, c["w"], 1e-5, alone, q, step, **kw)
        assert torch.equal(alone, out)


OO_ACT = {"none": 0, "silu": 3, "sigmoid": 4}


def test_block_norm_special_rows(gpu_lib):
    """Rows of zeros without eps stay zeros; rows whose squares overflow or vanish are
    normalised; a row that holds NaN or infinity gets a step that is not finite, and its
    neighbours nothing of it."""
    import torch
    L = gpu_lib
    rows, cols = 8, 520
    c = inputs(torch, rows, cols, "fp32", "none", "none")
    x = c["x"].contiguous()
    x[1] = 0
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    out, q, step = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    kept = torch.empty_like(x)
    L.ssd_block_norm(x, c["post"], None, kept, c["w"], 0.0, out, q, step)
    torch.cuda.synchronize()
    assert not out[1].any() and not kept[1].any() and not q[1].any() and step[1] == 1
    assert not torch.isfinite(step[4]) and not torch.isfinite(step[5])
    good = [0, 2, 3, 6, 7]
    c["x"] = x[good]
    r, y, dr, dy = reference(c, "none", 1.0, "fp32", eps=0.0)
    within(_np(kept[good]), r, dr, "fp32", "r")
    v = _np(q[good]) * _np(step[good])[:, None]
    assert (np.abs(v - y) <= _np(step[good])[:, None] * 0.501 + dy).all()
