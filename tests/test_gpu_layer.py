"""The steps around the SSD in a layer against their float64 definitions.

Bounds are counted from the roundings made (u = 2^-24, one fp32 rounding):
  convolution  W + 1 multiply-adds on sum |w x| + |b|; SiLU has a slope of at
               most 1.1, its exponential and reciprocal cost (|u| + 8) u of it
  softplus     one addition (|v| u, slope over value at most 1) and 16 u
  norms        the sum of squares of a row adds at most 40 roundings in any
               path through its tree, half of which reach 1/rms; SiLU and the
               products add 20: 128 u covers them
  codes        half a step, and 127 times the norm's 128 u
  product      exact sums; their conversion, the step's product and the
               multiply-add: 3 u
and half a step of the stored type on top of each.
"""
import numpy as np
import pytest

from oracle import layer_oracle as LO
from oracle import ssd_oracle as SO
from tests import _helpers as H

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": "float32", "fp16": "float16", "bf16": "bfloat16"}


def _t(torch, dtype):
    return getattr(torch, DT[dtype])


def _np(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, bound, dtype, what):
    """|got - ref| <= bound + half a step of the type at got, everywhere."""
    err = np.abs(got - ref) - H.half_ulp(got, dtype)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(err / (bound + 1e-300)):.3g} of the bound"


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def _conv_case(torch, seed, B, L, H_, P, N, G, W, dtype, cut=0, bias=True):
    """In Proj rows z | xBC | dt (cut: columns dropped from z, which moves the slice's alignment)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d, cd = H_ * P, H_ * P + 2 * G * N
    full = (1.5 * r(B, L, d - cut + cd + H_)).to(_t(torch, dtype))
    c = {"xbc": full[..., d - cut:d - cut + cd], "raw": full[..., d - cut + cd:], "W": W, "cd": cd, "d": d}
    c["w"], c["b"] = 0.5 * r(cd, W), (0.2 * r(cd) if bias else None)
    c["dtb"] = (r(H_) - 3) if bias else None
    c["ring"] = r(B, W, cd).to(_t(torch, dtype))
    return c


def _conv_refs(c, pos, hist):
    w, b = _np(c["w"]), (_np(c["b"]) if c["b"] is not None else np.zeros(c["cd"]))
    u, mag = LO.conv(_np(c["xbc"]), w, b, hist)
    y = LO.silu(u)
    bound = 1.1 * (c["W"] + 2) * U * mag + np.abs(y) * (np.abs(u) + 8) * 2 * U
    v = _np(c["raw"]) + (_np(c["dtb"]) if c["dtb"] is not None else 0.0)
    dt = LO.softplus(v)
    return y, bound, dt, dt * (np.abs(v) + 16) * 2 * U


CONV = [
    # B, L, H, P, N, G, W, dtype, history, ragged, cut
    (1, 1, 4, 16, 16, 1, 4, "fp16", True, False, 0),
    (2, 2, 4, 16, 16, 1, 4, "bf16", True, True, 0),
    (3, 3, 5, 32, 16, 1, 4, "fp16", True, True, 1),
    (2, 37, 3, 64, 32, 3, 3, "bf16", True, True, 3),
    (1, 130, 6, 64, 64, 2, 2, "fp32", True, False, 1),
    (4, 65, 8, 16, 128, 8, 4, "fp32", False, True, 0),
    (2, 701, 80, 64, 128, 1, 4, "fp16", False, False, 0),
    (5, 300, 24, 64, 128, 8, 4, "bf16", True, True, 0),
    (1, 4097, 8, 32, 64, 1, 3, "fp16", False, False, 8),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c)))
def test_conv_forward(gpu_lib, case):
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G, W, dtype, history, ragged, cut = case
    print("conv", case, flush=True)
    c = _conv_case(torch, 11, B, Ln, H_, P, N, G, W, dtype, cut)
    td = _t(torch, dtype)
    # sequences at their start, one and two positions in, and far on
    pos = torch.tensor(([0, 1, 2, 7, 1000003] * B)[:B] if B > 1 else [5], dtype=torch.int32, device="cuda") if history else None
    ends = ([0, Ln, 1, max(0, Ln - 1), Ln + 5] * B)[:B] if ragged else [Ln] * B
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda") if ragged else None
    ends = [min(e, Ln) for e in ends]
    p = pos.tolist() if history else [0] * B
    ring0 = _np(c["ring"])
    hist = LO.conv_history(ring0, p, W) if history else np.zeros((B, W - 1, c["cd"]))
    nan = float("nan")
    X = torch.full((B, Ln, H_, P), nan, dtype=td, device="cuda")
    Bo, Co = (torch.full((B, Ln, G, N), nan, dtype=td, device="cuda") for _ in range(2))
    dt = torch.full((B, Ln, H_), nan, dtype=td, device="cuda")
    if history:  # slots of positions that never were hold nothing to be read
        for b in range(B):
            for s in range(W):
                if not any((q % W) == s for q in range(max(0, p[b] - W), p[b])):
                    c["ring"][b, s] = nan
    keep = c["ring"].clone()
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])
    sh = L.make_shape(B, Ln, H_, P, N, G, 64, dtype)
    L.ssd_conv_forward(sh, conv, c["xbc"], c["raw"], X, Bo, Co, dt, c["ring"], pos, lengths)
    torch.cuda.synchronize()
    y, bound, dref, dbound = _conv_refs(c, p, hist)
    for b, e in enumerate(ends):
        y[b, e:] = 0; bound[b, e:] = 0; dref[b, e:] = 0; dbound[b, e:] = 0  # noqa: E702
    got = np.concatenate([_np(X).reshape(B, Ln, -1), _np(Bo).reshape(B, Ln, -1), _np(Co).reshape(B, Ln, -1)], -1)
    # a row at or behind the end is exactly zero
    for b, e in enumerate(ends):
        assert not got[b, e:].any() and not _np(dt)[b, e:].any()
        got_b, ref_b = got[b, :e], y[b, :e]
        _within(got_b, ref_b, bound[b, :e], dtype, f"x|B|C of sequence {b}")
        _within(_np(dt)[b, :e], dref[b, :e], dbound[b, :e], dtype, f"dt of sequence {b}")
    ref = LO.ring_after(_np(keep), _np(c["xbc"]), p, ends, W)
    assert np.array_equal(_np(c["ring"]), ref, equal_nan=True)


def test_conv_forward_without_optional_parts(gpu_lib):
    """No bias, no dt_bias, no ring; batch 0 and length 0 enqueue nothing."""
    import torch
    L = gpu_lib
    c = _conv_case(torch, 5, 2, 40, 4, 16, 16, 1, 4, "fp16", bias=False)
    X = torch.empty((2, 40, 4, 16), dtype=torch.float16, device="cuda")
    Bo, Co = (torch.empty((2, 40, 1, 16), dtype=torch.float16, device="cuda") for _ in range(2))
    dt = torch.empty((2, 40, 4), dtype=torch.float16, device="cuda")
    L.ssd_conv_forward(L.make_shape(2, 40, 4, 16, 16, 1, 64, "fp16"), L.ConvParams(c["w"]), c["xbc"], c["raw"], X, Bo,
                       Co, dt)
    y, bound, dref, dbound = _conv_refs(c, None, np.zeros((2, 3, c["cd"])))
    got = np.concatenate([_np(X).reshape(2, 40, -1), _np(Bo).reshape(2, 40, -1), _np(Co).reshape(2, 40, -1)], -1)
    _within(got, y, bound, "fp16", "x|B|C")
    _within(_np(dt), dref, dbound, "fp16", "dt")
    before = X.clone()
    e = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")  # noqa: E731
    for b, n in ((0, 40), (2, 0)):
        L.ssd_conv_forward(L.make_shape(b, n, 4, 16, 16, 1, 64, "fp16"), L.ConvParams(c["w"]), e(b, n, 96),
                           e(b, n, 4), e(b, n, 4, 16), e(b, n, 1, 16), e(b, n, 1, 16), e(b, n, 4))
    torch.cuda.synchronize()
    assert torch.equal(before, X)


@pytest.mark.parametrize("dtype,W", [("fp16", 4), ("bf16", 3), ("fp32", 2)])
def test_conv_chunks_equal_the_whole(gpu_lib, dtype, W):
    """A prompt in chunks of 1, 2, 5, 64 and the rest, carried by the ring, gives the
    whole prompt's outputs and ring bit for bit."""
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G = 2, 200, 4, 32, 16, 2
    c = _conv_case(torch, 8, B, Ln, H_, P, N, G, W, dtype)
    td = _t(torch, dtype)
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])

    def run(x, raw, n, ring, pos):
        o = [torch.empty(s, dtype=td, device="cuda") for s in
             ((B, n, H_, P), (B, n, G, N), (B, n, G, N), (B, n, H_))]
        L.ssd_conv_forward(L.make_shape(B, n, H_, P, N, G, 64, dtype), conv, x, raw, *o, ring, pos)
        return o

    ring = torch.full((B, W, c["cd"]), float("nan"), dtype=td, device="cuda")
    whole = run(c["xbc"], c["raw"], Ln, ring, torch.zeros(B, dtype=torch.int32, device="cuda"))
    ring2 = torch.full_like(ring, float("nan"))
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    parts, at = [], 0
    for n in (1, 2, 5, 64, Ln - 72):
        # a chunk of the batch lies at unequal distances: it is a copy, as a projection of its own would be
        parts.append(run(c["xbc"][:, at:at + n].contiguous(), c["raw"][:, at:at + n].contiguous(), n, ring2, pos))
        pos += n
        at += n
    torch.cuda.synchronize()
    for k, w in enumerate(whole):
        assert torch.equal(H.bits(torch.cat([p[k] for p in parts], 1)), H.bits(w)), k
    assert torch.equal(H.bits(ring), H.bits(ring2))


def test_conv_long_tiles_equal_short_ones(gpu_lib):
    """A batch that fills the chip with tiles of 64 positions, with ragged ends in
    and between them, equals its sequences by themselves (shorter tiles) bit for bit."""
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G, W = 6, 2050, 80, 64, 128, 1, 4
    c = _conv_case(torch, 81, B, Ln, H_, P, N, G, W, "bf16")
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])
    lengths = torch.tensor([2050, 64, 1999, 0, 2048, 65], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1, 2, 3, 70, 0], dtype=torch.int32, device="cuda")

    def run(b0, b1):
        n = b1 - b0
        o = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in
             ((n, Ln, H_, P), (n, Ln, G, N), (n, Ln, G, N), (n, Ln, H_))]
        ring = c["ring"][b0:b1].clone()
        L.ssd_conv_forward(L.make_shape(n, Ln, H_, P, N, G, 64, "bf16"), conv, c["xbc"][b0:b1], c["raw"][b0:b1], *o,
                           ring, pos[b0:b1].clone(), lengths[b0:b1].clone())
        return [*o, ring]

    whole = run(0, B)
    for b in range(B):
        for w, s in zip(whole, run(b, b + 1)):
            assert torch.equal(H.bits(w[b:b + 1].contiguous()), H.bits(s)), b


# ---------------------------------------------------------------------------
# decode step
# ---------------------------------------------------------------------------

STEP = [
    # B, H, P, N, G, W, dtype, cut
    (1, 4, 16, 16, 1, 4, "fp16", 0),
    (3, 6, 32, 32, 3, 3, "bf16", 1),
    (2, 5, 64, 64, 1, 2, "fp32", 3),
    (4, 8, 16, 128, 8, 4, "bf16", 0),
    (7, 80, 64, 128, 1, 4, "fp16", 0),
    (2, 16, 64, 16, 2, 4, "fp32", 0),
    (3, 3, 32, 128, 3, 3, "fp16", 2),
    # several heads a workgroup, the last of a group with fewer
    (150, 13, 16, 32, 1, 4, "fp16", 0),
    (400, 6, 32, 16, 2, 3, "bf16", 1),
    (70, 40, 32, 64, 1, 2, "fp32", 0),
    (300, 20, 64, 16, 1, 4, "fp16", 3),
    (1100, 8, 16, 16, 1, 4, "bf16", 0),
    (60, 20, 16, 128, 1, 4, "fp16", 0),
]


def _step_case(torch, case, seed=21):
    B, H_, P, N, G, W, dtype, cut = case
    c = _conv_case(torch, seed, B, 1, H_, P, N, G, W, dtype, cut)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    c["xbc"], c["raw"] = c["xbc"][:, 0], c["raw"][:, 0]
    c["A"] = -torch.exp(2 * torch.rand(H_, generator=g, device="cuda"))
    c["D"] = torch.randn(H_, generator=g, device="cuda")
    c["h"] = torch.randn(B, H_, P, N, generator=g, device="cuda")
    c["pos"] = torch.tensor(([0, 1, 2, 3, 4, 999, 2147483647] * B)[:B], dtype=torch.int32, device="cuda")
    return c


@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c)))
def test_decode_step_float(gpu_lib, case):
    import torch
    L = gpu_lib
    B, H_, P, N, G, W, dtype, cut = case
    print("step float", case, flush=True)
    c = _step_case(torch, case)
    h0, ring0 = _np(c["h"]), _np(c["ring"])
    Y = torch.empty((B, H_, P), dtype=_t(torch, dtype), device="cuda")
    L.ssd_conv_decode_step(L.make_shape(B, 1, H_, P, N, G, 64, dtype), L.SSD_PATH_FLOAT,
                           L.ConvParams(c["w"], c["b"], c["dtb"]), c["xbc"], c["raw"], c["A"], c["D"], None, c["ring"],
                           c["pos"], c["h"], Y)
    torch.cuda.synchronize()
    p = c["pos"].tolist()
    x1 = {**c, "xbc": c["xbc"][:, None], "raw": c["raw"][:, None]}
    y, by, dt, bdt = _conv_refs(x1, p, LO.conv_history(ring0, p, W))
    y, by, dt, bdt = y[:, 0], by[:, 0], dt[:, 0], bdt[:, 0]
    d, gn, hpg = H_ * P, G * N, H_ // G
    part = lambda v: (v[:, :d].reshape(B, H_, P, 1),  # noqa: E731
                      np.repeat(v[:, d:d + gn].reshape(B, G, N), hpg, 1)[:, :, None],
                      np.repeat(v[:, d + gn:].reshape(B, G, N), hpg, 1)[:, :, None])
    (x, bm, cm), (ex, eb, ec) = part(y), part(by)
    A, D = _np(c["A"]), _np(c["D"])[:, None, None]
    dt, bdt = dt[:, :, None, None], bdt[:, :, None, None]
    arg = dt * A[:, None, None]
    decay = np.exp(arg)
    href = decay * h0 + dt * x * bm
    # the decay's exponent: dt's own error, one product, and the exponential's 4 u
    bdecay = decay * (np.abs(A[:, None, None]) * bdt + (np.abs(arg) + 4) * 2 * U)
    bh = np.abs(h0) * bdecay + dt * (np.abs(x) * eb + np.abs(bm) * ex) + np.abs(x * bm) * bdt \
        + 4 * U * (np.abs(decay * h0) + np.abs(dt * x * bm))
    _within(_np(c["h"]), href, bh, "fp32", "state")
    yref = (cm * href).sum(-1) + (D * x)[..., 0]
    ymag = np.abs(cm * href).sum(-1) + np.abs(D * x)[..., 0]
    bY = (np.abs(cm) * bh + ec * np.abs(href)).sum(-1) + (np.abs(D) * ex)[..., 0] + 16 * U * ymag
    _within(_np(Y), yref, bY, dtype, "Y")
    assert np.array_equal(_np(c["ring"]), LO.ring_after(ring0, _np(x1["xbc"]), [q % W for q in p], [1] * B, W))


@pytest.mark.parametrize("path", ["float", "int8"])
@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c)))
def test_decode_step_is_the_convolution_and_the_step(gpu_lib, case, path):
    """The fused step leaves the state that ssd_conv_forward over one position and
    ssd_decode_step leave when both run in fp32 (where nothing between them is
    rounded), the INT8 state bit for bit, and their Y to within the rounding into
    its type. The compiler may contract the two kernels' multiply-adds differently,
    so the sums agree to their roundings, not to the bit: INT8's Y is three products
    (up to three roundings each) and two additions, float's an N-term dot product
    (up to 7 roundings on a path through its tree) and D x, so that each side is
    within 8 u of the terms' magnitudes."""
    import torch
    L = gpu_lib
    B, H_, P, N, G, W, dtype, cut = case
    print("step equals", case, path, flush=True)
    c = _step_case(torch, case)
    td, i8 = _t(torch, dtype), path == "int8"
    p = L.SSD_PATH_INT8 if i8 else L.SSD_PATH_FLOAT
    sc = None
    if i8:
        rng = np.random.default_rng(4)
        am = (rng.uniform(2, 3, G), rng.uniform(2, 3, G), rng.uniform(0.1, 0.5, (H_, P)), rng.uniform(2, 4, (H_, P)))
        sc = L.ScalePack(SO.scale_pack(*am, H_))
        c["h"] = torch.randint(-127, 128, c["h"].shape, device="cuda", dtype=torch.int8)
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])
    h2, ring2 = c["h"].clone(), c["ring"].float()
    Y = torch.empty((B, H_, P), dtype=td, device="cuda")
    L.ssd_conv_decode_step(L.make_shape(B, 1, H_, P, N, G, 64, dtype), p, conv, c["xbc"], c["raw"], c["A"], c["D"], sc,
                           c["ring"], c["pos"], c["h"], Y)
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    sh = L.make_shape(B, 1, H_, P, N, G, 64, "fp32")
    X, Bo, Co, dt, Y2 = f(B, 1, H_, P), f(B, 1, G, N), f(B, 1, G, N), f(B, 1, H_), f(B, H_, P)
    L.ssd_conv_forward(sh, conv, c["xbc"].float()[:, None].contiguous(), c["raw"].float()[:, None].contiguous(), X, Bo,
                       Co, dt, ring2, c["pos"])
    L.ssd_decode_step(sh, p, X, dt, c["A"], Bo, Co, c["D"], sc, h2, Y2)
    torch.cuda.synchronize()
    assert torch.equal(c["ring"].float(), ring2)
    xh = X[:, 0].abs()
    skip = c["D"].abs()[:, None] * xh
    heads = lambda v: v[:, 0].abs().repeat_interleave(H_ // G, 1)  # noqa: E731
    if i8:
        assert torch.equal(c["h"], h2)
        sB, sC = (torch.from_numpy(sc.host[k]).cuda().repeat_interleave(H_ // G)[:, None] for k in ("s_B", "s_C"))
        # |Q(B) . Q(C)| s_B s_C is at most the sum of (|B| + s_B)(|C| + s_C)
        diag = ((heads(Bo) + sB) * (heads(Co) + sC)).sum(-1, keepdim=True) * dt[:, 0, :, None] * xh
        mag = Y2.abs() + 2 * (diag + skip)
    else:
        # the state: two products and a sum, 2 roundings each
        assert (c["h"] - h2).abs().max() <= 4 * U * max(1.0, 2 * float(h2.abs().max()))
        mag = (heads(Co)[:, :, None] * h2.abs()).sum(-1) + skip
    err = (Y.float() - Y2).abs().double().cpu().numpy() - H.half_ulp(_np(Y), dtype)
    assert (err <= 16 * U * _np(mag)).all(), float((err / (16 * U * _np(mag))).max())


def test_decode_steps_follow_a_prompt(gpu_lib):
    """A prompt of 7 positions and 5 single steps give the outputs of one prompt of 12."""
    import torch
    L = gpu_lib
    B, n0, n1, H_, P, N, G, W = 3, 7, 5, 4, 16, 16, 1, 4
    c = _conv_case(torch, 3, B, n0 + n1, H_, P, N, G, W, "fp32")
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])
    A = -torch.ones(H_, device="cuda")
    D = torch.ones(H_, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731

    def prompt(x, raw, n, ring, pos, fin):
        X, Bo, Co, dt, Y = f(B, n, H_, P), f(B, n, G, N), f(B, n, G, N), f(B, n, H_), f(B, n, H_, P)
        sh = L.make_shape(B, n, H_, P, N, G, 64, "fp32")
        L.ssd_conv_forward(sh, conv, x.contiguous(), raw.contiguous(), X, Bo, Co, dt, ring, pos)
        L.ssd_forward(sh, L.SSD_PATH_FLOAT, X, dt, A, Bo, Co, D, None, Y, final_state=fin)
        return Y

    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    whole = prompt(c["xbc"], c["raw"], n0 + n1, None, None, None)
    ring, h = f(B, W, c["cd"]), f(B, H_, P, N)
    prompt(c["xbc"][:, :n0], c["raw"][:, :n0], n0, ring, pos, h)
    pos += n0
    for t in range(n0, n0 + n1):
        Y = f(B, H_, P)
        L.ssd_conv_decode_step(L.make_shape(B, 1, H_, P, N, G, 64, "fp32"), L.SSD_PATH_FLOAT, conv, c["xbc"][:, t],
                               c["raw"][:, t], A, D, None, ring, pos, h, Y)
        pos += 1
        ref = whole[:, t]
        assert (Y - ref).abs().max() <= 1e-4 * ref.abs().max(), t


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

EPS = 1e-5
NORM = [(1, 1), (3, 5), (6, 512), (5, 509), (9, 100), (2, 8), (5, 64), (2, 777), (7, 1000), (4, 1025), (8, 2560), (3, 4096), (2, 5000), (3, 8200),
        (2, 16384), (2, 16383)]


def _check_rows(torch, L, y, bound, out, q, s, dtype):
    """out (values) and codes of rows whose exact values are y, known to within bound."""
    if q is None:
        _within(_np(out), y, bound, dtype, "out")
        return
    most = np.abs(y).max(-1)
    step = np.where(most > 0, most / 127, 1.0)
    slack = (bound.max(-1) / 127 + 4 * U * step)
    assert (np.abs(_np(s) - step) <= slack).all()
    codes, gs = q.cpu().numpy().astype(np.float64), _np(s)[:, None]
    rel = 127 * (bound.max(-1) / np.maximum(most, 1e-300) + 8 * U)[:, None]
    assert (np.abs(codes - y / gs) <= 0.5 + np.where(most[:, None] > 0, rel, 0)).all()
    assert (np.abs(codes) <= 127).all()
    if out is not None:
        # a product of two fp32 values in fp32 (one rounding, or none where it is rounded at once)
        v = _np(q) * _np(s)[:, None]
        _within(_np(out), v, U * np.abs(v), dtype, "the codes' values")


@pytest.mark.parametrize("dtype,res,codes", [("fp16", "same", True), ("bf16", "fp32", True), ("fp32", "same", True),
                                             ("bf16", "none", False), ("fp16", "fp32", False)])
@pytest.mark.parametrize("rows,cols", NORM)
def test_add_norm(gpu_lib, rows, cols, dtype, res, codes):
    import torch
    L = gpu_lib
    print("norm", rows, cols, dtype, res, codes, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows * 100003 + cols)
    td = _t(torch, dtype)
    pad = 0 if cols % 2 else 8
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").to(td)[:, pad:]  # rows of a wider tensor
    rt = {"same": td, "fp32": torch.float32, "none": None}[res]
    r = (3 * torch.randn(rows, cols, generator=g, device="cuda")).to(rt) if rt is not None else None
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    kept = torch.empty((rows, cols), dtype=rt if rt is not None else td, device="cuda")
    out = torch.empty((rows, cols), dtype=td, device="cuda")
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(rows, device="cuda") if codes else None
    L.ssd_add_norm(x, r, kept, w, EPS, out, q, s)
    torch.cuda.synchronize()
    total = x.float() + (r.float() if r is not None else 0)
    assert torch.equal(H.bits(kept), H.bits(total.to(kept.dtype)))
    v = _np(x) + (_np(r) if r is not None else 0)
    y = LO.rms_rows(v, 1, _np(w), EPS)
    # r's own rounding is relative to r; the rest to y
    _check_rows(torch, L, y, np.abs(y) * 129 * U, out, q, s, dtype)


@pytest.mark.parametrize("dtype,codes", [("fp16", True), ("bf16", True), ("fp32", False), ("bf16", False)])
@pytest.mark.parametrize("rows,cols,groups,cut", [(1, 16, 1, 0), (3, 96, 3, 1), (2, 60, 5, 0), (5, 1024, 8, 0),
                                                  (37, 8192, 8, 0), (4, 5120, 1, 0), (3, 5120, 1, 3), (2, 1536, 128, 0),
                                                  (2, 9000, 3, 0), (2, 16384, 2, 1), (3, 2001, 1, 0), (2, 2001, 23, 2),
                                                  (6, 96, 4, 0), (5, 480, 20, 1), (9, 512, 2, 0), (3, 960, 20, 0),
                                                  (2, 4096, 64, 1), (2, 8000, 25, 0), (4, 1400, 100, 0), (3, 1416, 3, 0)])
def test_gated_norm(gpu_lib, rows, cols, groups, cut, dtype, codes):
    import torch
    L = gpu_lib
    print("gated", rows, cols, groups, cut, dtype, codes, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    td = _t(torch, dtype)
    y = torch.randn(rows, cols, generator=g, device="cuda").to(td)
    z = (2 * torch.randn(rows, cols + 24 + cut, generator=g, device="cuda")).to(td)[:, cut:cut + cols]
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    out = torch.empty((rows, cols), dtype=td, device="cuda")
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(rows, device="cuda") if codes else None
    L.ssd_gated_norm(y, z, groups, w, EPS, out, q, s)
    torch.cuda.synchronize()
    n = LO.rms_rows(_np(y) * LO.silu(_np(z)), groups, _np(w), EPS)
    _check_rows(torch, L, n, np.abs(n) * (128 + 2 * np.abs(_np(z))) * U, out, q, s, dtype)


def test_norm_rows_of_zeros_tiny_and_not_finite(gpu_lib):
    """A row of zeros: step 1, codes 0. Rows of values near fp32's smallest keep their
    codes. A row with NaN or infinity has a step that is not finite; the rows beside
    it are as without it."""
    import torch
    L = gpu_lib
    cols = 320
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, cols, generator=g, device="cuda")
    x[1] = 0
    x[2] *= 1e-37
    x[3, 17] = float("nan")
    x[4, 300] = float("inf")
    w = torch.ones(cols, device="cuda")
    q = torch.empty((6, cols), dtype=torch.int8, device="cuda")
    s, out = torch.empty(6, device="cuda"), torch.empty_like(x)
    L.ssd_add_norm(x, None, None, w, 1.0, out, q, s)  # eps 1: the tiny row stays tiny
    torch.cuda.synchronize()
    assert s[1] == 1 and not q[1].any() and not out[1].any()
    ref, step = LO.row_codes(LO.rms_rows(_np(x[[0, 2, 5]]), 1, np.ones(cols), 1.0))
    got = q[[0, 2, 5]].cpu().numpy()
    # values of the tiny row carry a step of 2^-149 over 127 codes of about 1e-39: half a code and that
    assert np.abs(got - ref).max() <= 1
    assert np.abs(_np(s)[[0, 2, 5]] - step).max() <= 2.0 ** -16 * step.max()
    assert not torch.isfinite(s[3]) and not torch.isfinite(s[4])
    assert torch.isfinite(s[[0, 1, 2, 5]]).all()


def test_norms_in_place_and_empty(gpu_lib):
    """out over x, residual_out over residual, out over y; no rows."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(2)
    for cols in (2560, 777):
        x = torch.randn(5, cols, generator=g, device="cuda").half()
        r = torch.randn(5, cols, generator=g, device="cuda")
        w = torch.rand(cols, generator=g, device="cuda")
        o, k = torch.empty_like(x), torch.empty_like(r)
        L.ssd_add_norm(x, r, k, w, EPS, o)
        x2, r2 = x.clone(), r.clone()
        L.ssd_add_norm(x2, r2, r2, w, EPS, x2)
        assert torch.equal(x2, o) and torch.equal(r2, k)
        L.ssd_gated_norm(x, r.half(), 1, w, EPS, o)
        x2 = x.clone()
        L.ssd_gated_norm(x2, r.half(), 1, w, EPS, x2)
        assert torch.equal(x2, o)
        L.ssd_add_norm(x[:0], None, None, w, EPS, o[:0])
        L.ssd_gated_norm(x[:0], x[:0], 1, w, EPS, o[:0])
    torch.cuda.synchronize()


@pytest.mark.parametrize("cols", [4104, 4360, 8200, 12296])
def test_add_norm_over_the_residual_where_a_wave_has_no_piece(gpu_lib, cols):
    """Rows whose last wave lies behind the last piece: the codes do not depend on
    whether residual_out is the residual itself."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(cols)
    rows = 2000
    x = torch.randn(rows, cols, generator=g, device="cuda").half()
    r = torch.randn(rows, cols, generator=g, device="cuda")
    r[:, -8:] += 40 * torch.sign(x[:, -8:].float())  # the last piece decides the scale
    x[:, -8:] *= 20
    w = torch.ones(cols, device="cuda")

    def run(res, res_out):
        q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(rows, device="cuda")
        L.ssd_add_norm(x, res, res_out, w, EPS, None, q, s)
        return q, s, res_out

    a, b = run(r, torch.empty_like(r)), run(r2 := r.clone(), r2)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

MM = [(1, 1, 16), (1, 17, 64), (2, 64, 48), (7, 100, 5120), (8, 2560, 5120), (15, 33, 144), (16, 256, 2560),
      (17, 300, 272), (33, 129, 1040), (63, 64, 64), (65, 1000, 128), (100, 80, 8192), (128, 512, 4096),
      (130, 2568, 2560), (256, 256, 640), (257, 259, 656), (333, 8512, 2048), (1000, 777, 1024), (2048, 10576, 272),
      (3001, 130, 2560), (4096, 2560, 5120), (4100, 2061, 400),
      (4096, 2048, 48), (3001, 4000, 656), (1500, 2051, 512), (4096, 2048, 1024), (8354, 33, 2368)]


@pytest.mark.parametrize("M,N,K", MM)
def test_matmul(gpu_lib, M, N, K):
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 7 * K)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    a[0], w[0] = -128, -128  # the largest sum
    sa = (0.5 + torch.rand(M, generator=g, device="cuda")) / 128
    sw = (0.5 + torch.rand(N, generator=g, device="cuda")) / 128 / K ** 0.5
    bias = torch.randn(N, generator=g, device="cuda")
    acc = a.double() @ w.double().t()
    for dtype, b in (("fp32", bias), ("fp16", None), ("bf16", bias)):
        print("matmul", M, N, K, dtype, flush=True)
        # rows of a larger buffer: what lies behind the last row stays as it was
        buf = torch.full((M * N + 64,), 7.0, dtype=_t(torch, dtype), device="cuda")
        out = buf[:M * N].view(M, N)
        L.ssd_matmul_i8(a, sa, w, sw, b, out)
        torch.cuda.synchronize()
        assert (buf[M * N:] == 7).all()
        part = acc * sa.double()[:, None] * sw.double()
        ref = part + (b.double() if b is not None else 0)
        err = (out.double() - ref).abs()
        # half a step of the type: at most eps / 2 of the value, or of its smallest normal
        fi = torch.finfo(out.dtype)
        bound = 3 * U * part.abs() + U * ref.abs() + fi.eps / 2 * (1 + U * 8) * out.double().abs().clamp(min=fi.tiny)
        assert (err <= bound).all(), (dtype, float((err / bound).max()))


def test_matmul_is_the_same_every_time(gpu_lib):
    """Sums split over workgroups are whole numbers: any order gives the same bits."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(9)
    for M, N, K in ((8, 2560, 5120), (100, 80, 8192), (333, 512, 4096)):
        a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        sa, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        ws = L.ssd_matmul_i8_workspace(M, N, K)
        if ws is not None:
            ws.fill_(0x7b)  # nothing in it needs to start at zero
        first = torch.empty((M, N), device="cuda")
        L.ssd_matmul_i8(a, sa, w, sw, None, first, ws)
        for _ in range(5):
            again = torch.empty_like(first)
            L.ssd_matmul_i8(a, sa, w, sw, None, again, ws)
            assert torch.equal(first, again)


# ---------------------------------------------------------------------------
# a layer of them together
# ---------------------------------------------------------------------------

class _Layer:
    """One quantised Mamba-2 layer of the library's calls, and its float64 counterpart."""

    def __init__(self, L, torch, H_=8, P=32, N=32, G=2, model=192, W=4, dtype="bf16", seed=0):
        self.L, self.torch, self.dtype, self.td = L, torch, dtype, _t(torch, dtype)
        self.H, self.P, self.N, self.G, self.W, self.model = H_, P, N, G, W, model
        rng = np.random.default_rng(seed)
        self.d, self.cd = H_ * P, H_ * P + 2 * G * N
        self.wide = self.d + self.cd + H_
        w_in = (rng.standard_normal((self.wide, model)) / np.sqrt(model)).astype(np.float32)
        w_out = (rng.standard_normal((model, self.d)) / np.sqrt(self.d)).astype(np.float32)
        self.win, self.sin = L.ssd_pack_weight_i8(w_in)
        self.wout, self.sout = L.ssd_pack_weight_i8(w_out)
        self.cw = (0.5 * rng.standard_normal((self.cd, W))).astype(np.float32)
        self.cb = (0.1 * rng.standard_normal(self.cd)).astype(np.float32)
        self.dtb = (rng.standard_normal(H_) * 0.5 - 3).astype(np.float32)
        self.A = -np.exp(rng.uniform(0, 2, H_)).astype(np.float32)
        self.D = rng.standard_normal(H_).astype(np.float32)
        self.n1 = (1 + 0.1 * rng.standard_normal(model)).astype(np.float32)
        self.n2 = (1 + 0.1 * rng.standard_normal(self.d)).astype(np.float32)
        dev = {k: torch.from_numpy(v).cuda() for k, v in vars(self).items() if isinstance(v, np.ndarray)}
        self.dev = dev
        self.conv = L.ConvParams(dev["cw"], dev["cb"], dev["dtb"])

    def project_in(self, x, res):
        L, t, n = self.L, self.torch, x.numel() // self.model
        q = t.empty((n, self.model), dtype=t.int8, device="cuda")
        s = t.empty(n, device="cuda")
        L.ssd_add_norm(x.view(n, self.model), res, res, self.dev["n1"], EPS, None, q, s)
        proj = t.empty((*x.shape[:-1], self.wide), dtype=self.td, device="cuda")
        L.ssd_matmul_i8(q, s, self.dev["win"], self.dev["sin"], None, proj)
        return proj[..., :self.d], proj[..., self.d:self.d + self.cd], proj[..., self.d + self.cd:]

    def project_out(self, y, z):
        L, t, n = self.L, self.torch, y.numel() // self.d
        q = t.empty((n, self.d), dtype=t.int8, device="cuda")
        s = t.empty(n, device="cuda")
        L.ssd_gated_norm(y, z, self.G, self.dev["n2"], EPS, None, q, s)
        out = t.empty((*z.shape[:-1], self.model), dtype=self.td, device="cuda")
        L.ssd_matmul_i8(q, s, self.dev["wout"], self.dev["sout"], None, out)
        return out

    def prompt(self, x, res, ring, pos, lengths, h):
        L, t = self.L, self.torch
        B, n = x.shape[:2]
        z, xbc, raw = self.project_in(x, res)
        e = lambda *s: t.empty(s, dtype=self.td, device="cuda")  # noqa: E731
        X, Bo, Co, dt, Y = e(B, n, self.H, self.P), e(B, n, self.G, self.N), e(B, n, self.G, self.N), e(B, n, self.H), \
            e(B, n, self.H, self.P)
        sh = L.make_shape(B, n, self.H, self.P, self.N, self.G, 64, self.dtype)
        L.ssd_conv_forward(sh, self.conv, xbc, raw, X, Bo, Co, dt, ring, pos, lengths)
        L.ssd_forward(sh, L.SSD_PATH_FLOAT, X, dt, self.dev["A"], Bo, Co, self.dev["D"], None, Y, final_state=h,
                      initial_state=h.clone())
        return self.project_out(Y, z)

    def step(self, x, res, ring, pos, h):
        L, t = self.L, self.torch
        B = x.shape[0]
        z, xbc, raw = self.project_in(x, res)
        Y = t.empty((B, self.H, self.P), dtype=self.td, device="cuda")
        L.ssd_conv_decode_step(L.make_shape(B, 1, self.H, self.P, self.N, self.G, 64, self.dtype), L.SSD_PATH_FLOAT,
                               self.conv, xbc, raw, self.dev["A"], self.dev["D"], None, ring, pos, h, Y)
        return self.project_out(Y, z)

    def reference(self, x, lengths):
        """The layer in float64 (unquantised activations): outputs [B, n, model]."""
        B, n, _ = x.shape
        w_in = self.win * self.sin[:, None].astype(np.float64)
        w_out = self.wout * self.sout[:, None].astype(np.float64)
        p = LO.rms_rows(x.reshape(B * n, -1), 1, self.n1, EPS) @ w_in.T
        p = p.reshape(B, n, -1)
        z, xbc, raw = p[..., :self.d], p[..., self.d:self.d + self.cd], p[..., self.d + self.cd:]
        v = LO.silu(LO.conv(xbc, self.cw.astype(np.float64), self.cb.astype(np.float64),
                            np.zeros((B, self.W - 1, self.cd)))[0])
        dt = LO.softplus(raw + self.dtb)
        X = v[..., :self.d].reshape(B, n, self.H, self.P)
        gn = self.G * self.N
        Bm, Cm = v[..., self.d:self.d + gn].reshape(B, n, self.G, self.N), v[..., self.d + gn:].reshape(B, n, self.G, self.N)
        Y = SO.chunked(X, dt, self.A, Bm, Cm, self.D, 64)[0].reshape(B * n, -1)
        u = LO.rms_rows(Y * LO.silu(z.reshape(B * n, -1)), self.G, self.n2, EPS)
        return (u @ w_out.T).reshape(B, n, -1)


def test_layer_prompts_then_tokens(gpu_lib):
    """Prompts of different lengths in one padded batch, then tokens, through all the
    calls: the outputs follow the float64 layer (8-bit rows cost about
    1/127/sqrt(12) of a row's largest value at each of two projections: 3 % of the
    outputs' size covers them with the 16-bit roundings), and each sequence's
    tokens do not depend on the padding."""
    import torch
    L = gpu_lib
    ly = _Layer(L, torch)
    g = torch.Generator(device="cuda").manual_seed(6)
    B, n, more = 3, 70, 4
    ends = [70, 1, 33]
    x = torch.randn(B, n + more, ly.model, generator=g, device="cuda").bfloat16()
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")

    def serve(pad):
        ring = torch.full((B, ly.W, ly.cd), float("nan"), dtype=ly.td, device="cuda")
        pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        h = torch.zeros((B, ly.H, ly.P, ly.N), device="cuda")
        xs = x[:, :n].clone()
        for b, e in enumerate(ends):
            xs[b, e:] = pad
        outs = [ly.prompt(xs, torch.zeros(B * n, ly.model, device="cuda"), ring, pos, lengths, h)]
        pos += lengths
        for t in range(more):
            tok = torch.stack([x[b, ends[b] + t] for b in range(B)])
            outs.append(ly.step(tok, torch.zeros(B, ly.model, device="cuda"), ring, pos, h))
            pos += 1
        torch.cuda.synchronize()
        return outs

    a, b = serve(0.5), serve(-3.0)
    for t in range(more):
        assert torch.equal(H.bits(a[1 + t]), H.bits(b[1 + t])), t
    for s, e in enumerate(ends):
        ref = ly.reference(_np(x[s:s + 1, :e + more]), None)[0]
        got = np.concatenate([_np(a[0][s, :e]), np.stack([_np(a[1 + t][s]) for t in range(more)])])
        assert np.sqrt(np.mean((got - ref) ** 2)) <= 0.03 * np.sqrt(np.mean(ref ** 2)), s


def test_layer_step_replayed_from_a_graph(gpu_lib):
    """A layer's token step captured once on its own stream and replayed with eager
    work between the replays equals eager steps bit for bit."""
    import torch
    L = gpu_lib
    ly = _Layer(L, torch, dtype="fp16", seed=3)
    B, steps = 4, 5
    g = torch.Generator(device="cuda").manual_seed(8)
    xs = torch.randn(steps, B, ly.model, generator=g, device="cuda").half()

    def fresh():
        return (torch.zeros((B, ly.W, ly.cd), dtype=ly.td, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
                torch.zeros((B, ly.H, ly.P, ly.N), device="cuda"), torch.zeros(B, ly.model, device="cuda"))

    ring, pos, h, res = fresh()
    eager = []
    for t in range(steps):
        eager.append(ly.step(xs[t], res, ring, pos, h))
        pos += 1
    x_in = xs[0].clone()
    ring2, pos2, h2, res2 = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ly.step(x_in, *[v.clone() for v in (res2, ring2, pos2, h2)])  # warm-up on copies
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ly.step(x_in, res2, ring2, pos2, h2)
        pos2 += 1
    for t in range(steps):
        x_in.copy_(xs[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(H.bits(out), H.bits(eager[t])), t
        _ = (out.float() * 2).sum().item()
    assert torch.equal(H.bits(h), H.bits(h2)) and torch.equal(H.bits(ring), H.bits(ring2)) and torch.equal(pos, pos2)


def test_layer_with_padding_that_is_not_finite(gpu_lib):
    """What lies behind a sequence's end, NaN or infinity, reaches neither its
    outputs nor its states."""
    import torch
    L = gpu_lib
    ly = _Layer(L, torch, dtype="fp16", seed=5)
    g = torch.Generator(device="cuda").manual_seed(16)
    B, n = 3, 130
    ends = [130, 64, 0]
    x = torch.randn(B, n, ly.model, generator=g, device="cuda").half()
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")
    got = []
    for pad in (0.0, float("nan"), float("inf")):
        xs = x.clone()
        for b, e in enumerate(ends):
            xs[b, e:] = pad
        ring = torch.zeros((B, ly.W, ly.cd), dtype=ly.td, device="cuda")
        h = torch.ones((B, ly.H, ly.P, ly.N), device="cuda")
        pos = torch.full((B,), 9, dtype=torch.int32, device="cuda")
        out = ly.prompt(xs, torch.zeros(B * n, ly.model, device="cuda"), ring, pos, lengths, h)
        got.append([ring, h] + [out[b, :e].clone() for b, e in enumerate(ends)])
    for other in got[1:]:
        for u, v in zip(got[0], other):
            assert torch.isfinite(v).all() and torch.equal(u, v)
    assert torch.equal(got[0][1][2], torch.ones_like(got[0][1][2]))  # a sequence of no positions


def test_layer_steps_on_streams_and_in_two_graphs(gpu_lib):
    """Two layers at once: eagerly on two streams, and as two graphs that replay by
    turns and side by side, each as alone. A batch of 300 takes other kernels of the
    product than one of 4."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(18)
    steps, sizes = 4, (4, 300)
    layers = [_Layer(L, torch, dtype=d, seed=k) for k, d in ((7, "fp16"), (8, "bf16"))]
    xs = [torch.randn(steps, b, ly.model, generator=g, device="cuda").to(ly.td) for b, ly in zip(sizes, layers)]

    def fresh(i):
        ly, b = layers[i], sizes[i]
        return (torch.zeros(b, ly.model, device="cuda"), torch.zeros((b, ly.W, ly.cd), dtype=ly.td, device="cuda"),
                torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros((b, ly.H, ly.P, ly.N), device="cuda"))

    alone = []
    for i, ly in enumerate(layers):
        res, ring, pos, h = fresh(i)
        outs = []
        for t in range(steps):
            outs.append(ly.step(xs[i][t], res, ring, pos, h))
            pos += 1
        alone.append(outs)
    torch.cuda.synchronize()

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    state = [fresh(0), fresh(1)]
    torch.cuda.synchronize()
    outs = [[], []]
    for t in range(steps):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(layers[i].step(xs[i][t], *state[i]))
                state[i][2].add_(1)
    torch.cuda.synchronize()
    for i in range(2):
        for t in range(steps):
            assert torch.equal(H.bits(outs[i][t]), H.bits(alone[i][t])), (i, t)

    state, x_in = [fresh(0), fresh(1)], [xs[0][0].clone(), xs[1][0].clone()]
    torch.cuda.synchronize()
    graphs, out = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            out.append(layers[i].step(x_in[i], *state[i]))
            state[i][2].add_(1)
    for t in range(steps):
        for i in range(2):
            x_in[i].copy_(xs[i][t])
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            if t % 2:  # side by side
                with torch.cuda.stream(s):
                    graphs[i].replay()
            else:
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(H.bits(out[i]), H.bits(alone[i][t])), (i, t)


# ---------------------------------------------------------------------------
# offsets that pass 32 bits: the end of a large buffer equals a call on the end alone
# ---------------------------------------------------------------------------

def test_conv_offsets_past_32_bits(gpu_lib):
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G, W, n = 2, 210001, 80, 64, 128, 1, 4, 150
    d, cd = H_ * P, H_ * P + 2 * G * N
    g = torch.Generator(device="cuda").manual_seed(3)
    full = torch.zeros((B, Ln, d + cd + H_), dtype=torch.float16, device="cuda")  # 8.9 GB
    full[:, -n:] = torch.randn((B, n, d + cd + H_), generator=g, device="cuda").half()
    conv = L.ConvParams(torch.randn((cd, W), generator=g, device="cuda"))

    def run(x):
        b, t = x.shape[:2]
        o = [torch.empty(s, dtype=x.dtype, device="cuda") for s in ((b, t, H_, P), (b, t, G, N), (b, t, G, N), (b, t, H_))]
        ring = torch.empty((b, W, cd), dtype=x.dtype, device="cuda")
        L.ssd_conv_forward(L.make_shape(b, t, H_, P, N, G, 64, "fp16"), conv, x[..., d:d + cd], x[..., d + cd:], *o, ring)
        return o, ring

    whole, ring = run(full)
    assert whole[0].numel() * 2 > 2 ** 32
    part, _ = run(full[1:, -n:])
    for u, v in zip(whole, part):
        assert torch.equal(u[1, -n + W:], v[0, W:])
    t = torch.arange(Ln - W, Ln, device="cuda")
    assert torch.equal(ring[1, t % W], full[1, -W:, d:d + cd])


def test_step_offsets_past_32_bits(gpu_lib):
    import torch
    L = gpu_lib
    B, H_, P, N, W, n = 2100, 80, 64, 128, 4, 3
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d, cd = H_ * P, H_ * P + 2 * N
    conv, A, D = L.ConvParams(r(cd, W)), -torch.rand(H_, generator=g, device="cuda"), r(H_)
    proj, ring = r(B, cd + H_).half(), r(B, W, cd).half()
    pos = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    h = torch.zeros((B, H_, P, N), device="cuda")
    assert h.numel() * 4 > 2 ** 32
    h[-n:] = r(n, H_, P, N)

    def run(b0, h, ring):
        Y = torch.empty((B - b0, H_, P), dtype=torch.float16, device="cuda")
        L.ssd_conv_decode_step(L.make_shape(B - b0, 1, H_, P, N, 1, 64, "fp16"), L.SSD_PATH_FLOAT, conv, proj[b0:, :cd],
                               proj[b0:, cd:], A, D, None, ring, pos[b0:], h, Y)
        return Y

    h2, ring2 = h[-n:].clone(), ring[-n:].clone()
    Y2 = run(B - n, h2, ring2)
    Y = run(0, h, ring)
    assert torch.equal(ring[-n:], ring2)
    # other numbers of heads a workgroup may contract products differently: two roundings of each term
    assert torch.allclose(h[-n:], h2, rtol=4 * U, atol=4 * U * float(h2.abs().max()))
    assert torch.allclose(Y[-n:].float(), Y2.float(), rtol=2 ** -10, atol=(2 * N) * U * float(Y2.abs().max()) + 2 ** -10)


def test_norm_offsets_past_32_bits(gpu_lib):
    import torch
    L = gpu_lib
    rows, cols, n = 450001, 5120, 7
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    assert x.numel() * 2 > 2 ** 32
    x[-n:] = torch.randn((n, cols), generator=g, device="cuda").half()
    w = torch.rand(cols, generator=g, device="cuda")

    def run(call):
        out = []
        for v in (x, x[-n:]):
            o, q = torch.empty_like(v), torch.empty(v.shape, dtype=torch.int8, device="cuda")
            s = torch.empty(v.shape[0], device="cuda")
            call(v, o, q, s)
            out.append((o[-n:], q[-n:], s[-n:]))
        for a, b in zip(*out):
            assert torch.equal(a, b)

    run(lambda v, o, q, s: L.ssd_add_norm(v, v, None, w, EPS, o, q, s))
    run(lambda v, o, q, s: L.ssd_gated_norm(v, v, 8, w, EPS, o, q, s))


def test_matmul_offsets_past_32_bits(gpu_lib):
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(6)
    for M, N, K, n in ((230001, 10001, 64, 300), (300, 8000000, 64, 300)):
        a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        sa, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
        out = torch.empty((M, N), dtype=torch.float16, device="cuda")
        assert out.numel() * 2 > 2 ** 32
        L.ssd_matmul_i8(a, sa, w, sw, None, out)
        c = slice(N - 500, N)
        part = torch.empty((n, 500), dtype=torch.float16, device="cuda")
        L.ssd_matmul_i8(a[-n:].contiguous(), sa[-n:].contiguous(), w[c].contiguous(), sw[c].contiguous(), None, part)
        assert torch.equal(out[-n:, c], part)
        del out
