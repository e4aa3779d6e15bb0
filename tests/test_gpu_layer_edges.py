"""The steps around the SSD where a rounding, a size or a choice of kernel decides:
the norms' codes by their documented rule, rows whose squares leave fp32's range,
exponentials of large arguments, groups of odd sizes, products for every kernel, the
INT8 path from prompt to tokens.

Bounds are counted from the roundings made (u = 2^-24, one fp32 rounding).
"""
import numpy as np
import pytest

from oracle import layer_oracle as LO
from tests import _helpers as H
from tests.test_gpu_layer import EPS, U, _check_rows, _np, _t, _within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# codes
# ---------------------------------------------------------------------------

def _codes_by_rule(y):
    """q = RHAZ(y / scale), scale = max|y| / 127 (1 where that is zero), each in fp32."""
    with np.errstate(under="ignore"):
        scale = (np.abs(y).max(-1) / np.float32(127)).astype(np.float32)
        scale = np.where(scale > 0, scale, np.float32(1))
        v = y / scale[:, None]
    assert v.dtype == np.float32
    return np.clip(LO.rhaz(v), -127, 127).astype(np.int8), scale


def _norm_calls(torch, L, x, r, z, groups, w, eps):
    """The rows (in x's type) and, from a second call, the codes and their steps."""
    out, q = torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8, device="cuda")
    s = torch.empty(x.shape[0], device="cuda")
    for o, c, p in ((out, None, None), (None, q, s)):
        if z is None:
            L.ssd_add_norm(x, r, None, w, eps, o, c, p)
        else:
            L.ssd_gated_norm(x, z, groups, w, eps, o, c, p)
    torch.cuda.synchronize()
    return out, q, s


@pytest.mark.parametrize("rows,cols,groups", [(4000, 2560, 0), (3000, 5120, 1), (3000, 8192, 8), (2000, 4096, 64),
                                              (1000, 777, 0), (900, 320, 2), (900, 1400, 100), (500, 509, 1)])
def test_norm_codes_follow_the_documented_rule(gpu_lib, rows, cols, groups):
    """Codes and steps are what the rows themselves give by q = RHAZ(y / scale), to
    the bit, from ordinary rows to rows whose step is the smallest subnormal or
    rounds to zero (groups 0: ssd_add_norm)."""
    import torch
    L = gpu_lib
    print("codes", rows, cols, groups, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x[::7] *= 1e-37
    x[3::7] *= torch.logspace(-44.5, -36, len(range(3, rows, 7)), device="cuda")[:, None]
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    z = 2 * torch.randn(rows, cols, generator=g, device="cuda") if groups else None
    y, q, s = _norm_calls(torch, L, x, None, z, groups, w, 1.0)  # eps 1: tiny rows stay tiny
    ref, step = _codes_by_rule(y.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), step)
    bad = q.cpu().numpy() != ref
    assert not bad.any(), f"{bad.sum()} of {bad.size} codes, in {bad.any(-1).sum()} rows"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(4000, 2560), (3000, 777), (900, 320), (37, 8192)])
def test_norm_codes_do_not_depend_on_the_type(gpu_lib, rows, cols, dtype):
    """16-bit rows and the same values in fp32 give the same codes and steps: all that
    happens before the codes is fp32."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(_t(torch, dtype))
    r = 3 * torch.randn(rows, cols, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    _, q, s = _norm_calls(torch, L, x, r, None, 0, w, EPS)
    _, qf, sf = _norm_calls(torch, L, x.float(), r, None, 0, w, EPS)
    assert torch.equal(s, sf) and torch.equal(q, qf)


def test_norm_tiny_rows_have_steps_of_their_own(gpu_lib):
    """Each row's step against its own largest value (a subnormal step is off by half
    of 2^-149), its codes by that step, and `out` as the values they stand for."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(6, 320, generator=g, device="cuda")
    x *= torch.tensor([1.0, 1e-20, 1e-36, 1e-37, 1e-40, 0.0], device="cuda")[:, None]
    w = torch.ones(320, device="cuda")
    q, s, out = torch.empty((6, 320), dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(x)
    L.ssd_add_norm(x, None, None, w, 1.0, out, q, s)
    torch.cuda.synchronize()
    y = LO.rms_rows(_np(x), 1, np.ones(320), 1.0)
    step = np.abs(y).max(-1) / 127
    step[5] = 1
    # the row's 40 roundings and the step's; a subnormal y is off by 2^-150, its step by a 127th of that and 2^-150
    assert (np.abs(_np(s) - step) <= 64 * U * step + 2.0 ** -149).all()
    codes, gs = _np(q), _np(s)[:, None]
    slack = (64 * U * np.abs(y) + 2.0 ** -149) / gs + 2 * U * np.abs(codes)
    assert (np.abs(codes - np.clip(y / gs, -127, 127)) <= 0.5 + slack).all()
    assert (np.abs(_np(out) - codes * gs) <= U * np.abs(codes * gs) + 2.0 ** -150).all()


# ---------------------------------------------------------------------------
# squares outside fp32's range
# ---------------------------------------------------------------------------

SPECIAL = [(320, 0), (512, 2), (2560, 0), (777, 0), (8192, 8), (4096, 64), (5000, 1), (60, 5), (2001, 23), (16384, 0)]


@pytest.mark.parametrize("dtype,codes", [("fp32", False), ("fp32", True), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("cols,groups", SPECIAL)
def test_norm_rows_whose_squares_overflow_or_vanish(gpu_lib, cols, groups, dtype, codes):
    """Rows that are finite but whose squares or their sum are not, and (eps = 0) rows
    whose squares fall below fp32, next to ordinary rows: all are normalised."""
    import torch
    L = gpu_lib
    print("squares", cols, groups, dtype, codes, flush=True)
    g = torch.Generator(device="cuda").manual_seed(cols + groups)
    td = _t(torch, dtype)
    n = max(groups, 1)
    big = torch.tensor([1e20, 1.0, 2e18, 1e36, 1e19], device="cuda")
    low = torch.tensor([1e-25, 1.0, 1e-30, 1e-22, 3e-19], device="cuda")
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    for sizes, eps in ((big, EPS), (big, 0.0), (low, 0.0), (low, 1e-45)):
        x = torch.randn(5, cols, generator=g, device="cuda")
        z = None
        if groups:  # a group each of its own size, shifted from row to row
            size = torch.stack([sizes.roll(k).repeat(n // 5 + 1)[:n] for k in range(5)])
            x = (x.view(5, n, -1) * size[..., None]).view(5, cols)
            z = (1 + torch.rand(5, cols, generator=g, device="cuda")).to(td)
        else:
            x = x * sizes[:, None]
            x[1, cols // 2] = 3e38 if sizes is big else 1e-30  # one value of its own size
        x = x.to(td)
        out = torch.empty_like(x)
        q = torch.empty(x.shape, dtype=torch.int8, device="cuda") if codes else None
        s = torch.empty(5, device="cuda") if codes else None
        if groups:
            L.ssd_gated_norm(x, z, groups, w, eps, out, q, s)
        else:
            L.ssd_add_norm(x, None, None, w, eps, out, q, s)
        torch.cuda.synchronize()
        v = _np(x) * (LO.silu(_np(z)) if groups else 1.0)
        y = LO.rms_rows(v, n, _np(w), np.float64(np.float32(eps)))
        # a value 2^80 below its row's largest may have been scaled into the subnormals
        _check_rows(torch, L, y, np.abs(y) * 136 * U + 2.0 ** -126, out, q, s, dtype)


@pytest.mark.parametrize("cols,groups", SPECIAL)
def test_norm_rows_of_zeros_without_eps(gpu_lib, cols, groups):
    """eps = 0: a row (or group) of zeros gives zeros, with a step of 1 where all of
    the row is; a row that holds NaN or infinity still shows it in its step."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(cols)
    n = max(groups, 1)
    x = torch.randn(4, cols, generator=g, device="cuda")
    x[0] = 0
    x[1, :cols // n] = 0
    x[2, -1], x[3, 0] = float("nan"), float("inf")
    w, z = torch.ones(cols, device="cuda"), torch.full((4, cols), 3.0, device="cuda")
    out, q, s = torch.empty_like(x), torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    if groups:
        L.ssd_gated_norm(x, z, groups, w, 0.0, out, q, s)
    else:
        L.ssd_add_norm(x, None, None, w, 0.0, out, q, s)
    torch.cuda.synchronize()
    assert s[0] == 1 and not out[0].any() and not q[0].any()
    assert not out[1, :cols // n].any() and torch.isfinite(s[1]) and (n == 1 or out[1, cols // n:].any())
    assert not torch.isfinite(s[2:]).any()


# ---------------------------------------------------------------------------
# more rows than workgroups
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("cols,groups,rows", [(528, 0, 1 << 20), (528, 2, 1 << 20), (1024, 2, 1 << 20), (12, 4, 1 << 20),
                                              (16, 0, 1 << 22), (32, 2, 1 << 22)])
def test_norm_workgroups_that_take_several_rows(gpu_lib, cols, groups, rows):
    """Rows behind the last workgroup's, which go to workgroups that have done a row
    already (one of zeros, of huge values, of NaN, ...), are as in a call of their own;
    with the rows written over their inputs too."""
    import torch
    L = gpu_lib
    more = 3000
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows + more, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    for first in (7, rows + 200):
        x[first] = 0
        x[first + 4] *= 1e25
        x[first + 8, cols // 2] = float("nan")
        x[first + 12] *= 1e-25
        x[first + 16, 0] = float("inf")
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    z = torch.ones_like(x) if groups else None

    def run(x, z, eps, out, q, s):
        if groups:
            L.ssd_gated_norm(x, z, groups, w, eps, out, q, s)
        else:
            L.ssd_add_norm(x, None, None, w, eps, out, q, s)

    def outputs(x, z, codes, place):
        q = torch.empty(x.shape, dtype=torch.int8, device="cuda") if codes else None
        s = torch.empty(x.shape[0], device="cuda") if codes else None
        x = x.clone() if place else x
        out = x if place else torch.empty_like(x)
        run(x, z, 0.0, out, q, s)
        return [t for t in (out, q, s) if t is not None]

    for codes, place in ((True, False), (False, True), (True, True)):
        whole = outputs(x, z, codes, place)
        for part in (slice(0, 5000), slice(rows - 100, rows + more)):
            alone = outputs(x[part].contiguous(), None if z is None else z[part].contiguous(), codes, False)
            for a, b in zip(whole, alone):
                assert torch.equal(H.bits(a[part].contiguous()), H.bits(b)), (codes, place, part)
        del whole

# ---------------------------------------------------------------------------
# groups of odd sizes in long rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,codes", [("fp32", False), ("fp32", True), ("fp16", True), ("bf16", True), ("bf16", False)])
@pytest.mark.parametrize("rows,cols,groups", [(3, 5100, 25), (2, 8204, 7), (2, 16380, 4095), (2, 16384, 16384),
                                              (5, 4097, 17), (3, 16383, 3), (3, 12300, 615)])
def test_gated_norm_long_rows_of_odd_groups(gpu_lib, rows, cols, groups, dtype, codes):
    import torch
    L = gpu_lib
    print("odd groups", rows, cols, groups, dtype, codes, flush=True)
    g = torch.Generator(device="cuda").manual_seed(cols)
    td = _t(torch, dtype)
    y = torch.randn(rows, cols, generator=g, device="cuda").to(td)
    z = (2 * torch.randn(rows, cols + 3, generator=g, device="cuda")).to(td)[:, 3:]
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    out = torch.empty((rows, cols), dtype=td, device="cuda")
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda") if codes else None
    s = torch.empty(rows, device="cuda") if codes else None
    L.ssd_gated_norm(y, z, groups, w, EPS, out, q, s)
    torch.cuda.synchronize()
    n = LO.rms_rows(_np(y) * LO.silu(_np(z)), groups, _np(w), EPS)
    _check_rows(torch, L, n, np.abs(n) * (128 + 2 * np.abs(_np(z))) * U, out, q, s, dtype)


# ---------------------------------------------------------------------------
# exponentials of large arguments
# ---------------------------------------------------------------------------

def test_conv_silu_of_large_arguments(gpu_lib):
    """fp32 storage: SiLU of values from -87 to 88 (weights of 0 and 1, so that u is
    the input itself) to 10 roundings, whatever the size of its argument: the
    exponential 2 and its argument's product 2, the sum 1, the reciprocal 2, the
    products 3."""
    import torch
    L = gpu_lib
    B, Ln, H_, P, N = 2, 500, 4, 16, 16
    cd = H_ * P + 2 * N
    g = torch.Generator(device="cuda").manual_seed(2)
    x = -87 + 175 * torch.rand(B, Ln, cd, generator=g, device="cuda")
    x[0, :50] /= 50
    w = torch.tensor([0.0, 1.0], device="cuda").repeat(cd, 1)
    X, Bo, Co, dt = (torch.empty(s, device="cuda") for s in ((B, Ln, H_, P), (B, Ln, 1, N), (B, Ln, 1, N), (B, Ln, H_)))
    L.ssd_conv_forward(L.make_shape(B, Ln, H_, P, N, 1, 64, "fp32"), L.ConvParams(w), x,
                       torch.zeros(B, Ln, H_, device="cuda"), X, Bo, Co, dt)
    torch.cuda.synchronize()
    got = np.concatenate([_np(v).reshape(B, Ln, -1) for v in (X, Bo, Co)], -1)
    ref = LO.silu(_np(x))
    _within(got, ref, 10 * U * np.abs(ref), "fp32", "silu")


@pytest.mark.parametrize("cols,groups", [(512, 1), (4096, 8), (1400, 100)])
def test_gated_norm_silu_of_large_arguments(gpu_lib, cols, groups):
    """fp32 rows gated by z from -80 to 8: the gate's 10 roundings, the product's 1, at
    most 22 of the sum of squares on a path through its tree, halved by the root, and
    8 behind it."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(cols)
    z = -80 + 88 * torch.rand(6, cols, generator=g, device="cuda")
    y = torch.randn(6, cols, generator=g, device="cuda")
    w, out = torch.ones(cols, device="cuda"), torch.empty_like(y)
    L.ssd_gated_norm(y, z, groups, w, 0.0, out)
    torch.cuda.synchronize()
    ref = LO.rms_rows(_np(y) * LO.silu(_np(z)), groups, np.ones(cols), 0.0)
    _within(_np(out), ref, 30 * U * np.abs(ref) + 2.0 ** -126, "fp32", "gated")


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_decode_step_exponentials_of_large_arguments(gpu_lib, dtype):
    """The step's decay and SiLU stay in fp32 in any storage type. With x = 0 the state
    is decay times what it was (dt A exact: exponential 2 roundings, product 1); with
    a state of zeros it is dt silu(u) silu(u_B) (10 roundings each and 2)."""
    import torch
    L = gpu_lib
    B, H_, P, N = 3, 80, 16, 16
    td, cd = _t(torch, dtype), H_ * P + 2 * N
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.tensor([0.0, 1.0], device="cuda").repeat(cd, 1)
    A, D = -torch.arange(H_, device="cuda") / 64.0, torch.zeros(H_, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step(x, raw, h):
        Y = torch.empty((B, H_, P), dtype=td, device="cuda")
        ring = torch.zeros((B, 2, cd), dtype=td, device="cuda")
        L.ssd_conv_decode_step(L.make_shape(B, 1, H_, P, N, 1, 64, dtype), L.SSD_PATH_FLOAT, L.ConvParams(w), x, raw, A,
                               D, None, ring, pos, h, Y)
        torch.cuda.synchronize()

    raw = torch.full((B, H_), 32.0, dtype=td, device="cuda")  # softplus(32) is 32 in fp32
    h0 = torch.randn(B, H_, P, N, generator=g, device="cuda")
    h = h0.clone()
    step(torch.zeros((B, cd), dtype=td, device="cuda"), raw, h)
    ref = _np(h0) * np.exp(32 * _np(A))[:, None, None]
    _within(_np(h), ref, 3 * U * np.abs(ref), "fp32", "decay")

    x = torch.empty(B, cd, device="cuda").uniform_(-60, 8, generator=g).to(td)
    x[:, H_ * P:] = (1 + 3 * torch.rand(B, 2 * N, generator=g, device="cuda")).to(td)
    h = torch.zeros((B, H_, P, N), device="cuda")
    step(x, raw, h)
    v = LO.silu(_np(x))
    ref = 32 * v[:, :H_ * P].reshape(B, H_, P, 1) * v[:, None, None, H_ * P:H_ * P + N]
    _within(_np(h), ref, 22 * U * np.abs(ref), "fp32", "dt x B")


# ---------------------------------------------------------------------------
# products for every kernel
# ---------------------------------------------------------------------------

# with test_gpu_layer.MM: every kernel of the dispatch, with and without a tail of K,
# with sums shorter and longer than its buffers, and with tiles that end with the
# matrix (test_layer_native.py asserts it)
MM_KERNELS = [(1, 16, 2048), (1, 3870, 512), (3, 4281, 1536), (2, 4427, 1072), (1, 5236, 3088), (1, 5357, 3584),
              (16, 9000, 3600), (2245, 33, 512), (2140, 33, 16), (3698, 17, 544), (18, 3004, 1552), (103, 6937, 528),
              (99, 7287, 1024), (41, 11479, 1616), (333, 2560, 5120), (333, 2560, 5136), (333, 8512, 2064),
              (340, 8500, 1040), (384, 3864, 864), (165, 7380, 1024), (4099, 2571, 5136), (3000, 10576, 1040),
              (687, 11060, 1536), (1790, 4864, 5024)]


@pytest.mark.parametrize("M,N,K", MM_KERNELS)
def test_matmul_every_kernel(gpu_lib, M, N, K):
    """Sums of both signs up to the largest, with and without bias, in the three types:
    exact sums, so 3 roundings and the type's."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + 7 * K)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    a[-1], w[-1] = -128, -128
    sa = (0.5 + torch.rand(M, generator=g, device="cuda")) / 128
    sw = (0.5 + torch.rand(N, generator=g, device="cuda")) / 128 / K ** 0.5
    bias = torch.randn(N, generator=g, device="cuda")
    acc = a.double() @ w.double().t().contiguous()
    part = acc * sa.double()[:, None] * sw.double()
    for dtype in ("fp32", "fp16", "bf16"):
        for b in (None, bias):
            print("matmul", M, N, K, dtype, b is not None, flush=True)
            buf = torch.full((M * N + 128,), 7.0, dtype=_t(torch, dtype), device="cuda")
            out = buf[64:64 + M * N].view(M, N)
            L.ssd_matmul_i8(a, sa, w, sw, b, out)
            torch.cuda.synchronize()
            assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
            ref = part + (b.double() if b is not None else 0)
            fi = torch.finfo(out.dtype)
            bound = 3 * U * part.abs() + U * ref.abs() + fi.eps / 2 * (1 + U * 8) * out.double().abs().clamp(min=fi.tiny)
            err = (out.double() - ref).abs()
            assert (err <= bound).all(), (dtype, b is not None, float((err / bound).max()))


def test_matmul_sums_are_exact_on_every_call(gpu_lib):
    """With steps of powers of two and sums below 2^24 the fp32 outputs are the whole
    numbers themselves: split sums lose nothing, on any call."""
    import torch
    L = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(9)
    for M, N, K in ((8, 2560, 1024), (100, 80, 1040), (333, 2560, 1024), (333, 8512, 1040), (4099, 2571, 768)):
        a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        sa, sw = torch.full((M,), 0.25, device="cuda"), torch.full((N,), 4.0, device="cuda")
        ref = (a.double() @ w.double().t().contiguous()).float()  # |sums| <= 127^2 K < 2^24
        for _ in range(4):
            out = torch.full((M, N), float("nan"), device="cuda")
            L.ssd_matmul_i8(a, sa, w, sw, None, out)
            assert torch.equal(out, ref), (M, N, K)


# ---------------------------------------------------------------------------
# the INT8 path from prompt to tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_int8_prompts_then_tokens(gpu_lib, dtype):
    """Convolution, the INT8 forward of ragged prompts on scales calibrated from the
    convolution's own outputs, then fused INT8 steps on the 8-bit state: states are
    the oracle's to the bit, outputs within the INT8 path's error. The oracle takes
    what the GPU hands from call to call (X, B, C, dt, each held to its definition by
    its own tests; a step's are those of a convolution that rounds nothing)."""
    import torch
    from oracle import ssd_oracle as SO
    from tests.test_gpu_layer import _conv_case
    L = gpu_lib
    B, n, more, H_, P, N, G, W = 3, 150, 6, 8, 32, 64, 2, 4
    td = _t(torch, dtype)
    c = _conv_case(torch, 31, B, n + more, H_, P, N, G, W, dtype)
    conv = L.ConvParams(c["w"], c["b"], c["dtb"])
    g = torch.Generator(device="cuda").manual_seed(32)
    A, D = -torch.exp(2 * torch.rand(H_, generator=g, device="cuda")), torch.randn(H_, generator=g, device="cuda")
    ends = [150, 1, 97]
    lengths = torch.tensor(ends, dtype=torch.int32, device="cuda")

    def convolve(x, raw, ring, pos, lens, t):
        b, k = x.shape[:2]
        o = [torch.empty(s, dtype=t, device="cuda") for s in ((b, k, H_, P), (b, k, G, N), (b, k, G, N), (b, k, H_))]
        sh = L.make_shape(b, k, H_, P, N, G, 64, "fp32" if t is torch.float32 else dtype)
        L.ssd_conv_forward(sh, conv, x, raw, *o, ring, pos, lens)
        return sh, o

    ring = torch.zeros((B, W, c["cd"]), dtype=td, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    sh, (X, Bo, Co, dt) = convolve(c["xbc"][:, :n].contiguous(), c["raw"][:, :n].contiguous(), ring, pos, lengths, td)
    sc = L.calibrate(lambda s: sh, [{"x": X, "dt": dt, "B": Bo, "C": Co}], A)
    h = torch.empty((B, H_, P, N), dtype=torch.int8, device="cuda")
    Y = torch.empty((B, n, H_, P), dtype=td, device="cuda")
    L.ssd_forward(sh, L.SSD_PATH_INT8, X, dt, A, Bo, Co, D, sc, Y, final_state=h)
    torch.cuda.synchronize()
    An, Dn = _np(A), _np(D)
    scales = {k: v.astype(np.float64).reshape((H_, P) if v.size == H_ * P else (G,)) for k, v in sc.host.items()}
    states = []
    for b, e in enumerate(ends):
        v = [_np(t[b:b + 1, :e]) for t in (X, dt, Bo, Co)]
        r = SO.forward_int8(v[0], v[1], An, v[2], v[3], Dn, scales, 64)
        states.append(r["passed"][:, -1])
        assert np.array_equal(h[b].cpu().numpy(), states[-1][0]), f"prompt {b}"
        # single positions have no spread to measure by: the largest prompts' channels
        if e > 64:
            assert H.chan_err(_np(Y[b:b + 1, :e]), r["y"], dtype) <= 5e-2
    ref = np.concatenate(states)
    pos += lengths
    ys, rs = [], []
    for t in range(more):
        x = torch.stack([c["xbc"][b, ends[b] + t] for b in range(B)])
        raw = torch.stack([c["raw"][b, ends[b] + t] for b in range(B)])
        _, o = convolve(x.float()[:, None].contiguous(), raw.float()[:, None].contiguous(), ring.float(), pos, None,
                        torch.float32)
        Xs, Bs, Cs, dts = (_np(k)[:, 0] for k in o)
        y = torch.empty((B, H_, P), dtype=td, device="cuda")
        L.ssd_conv_decode_step(L.make_shape(B, 1, H_, P, N, G, 64, dtype), L.SSD_PATH_INT8, conv, x, raw, A, D, sc,
                               ring, pos, h, y)
        pos += 1
        torch.cuda.synchronize()
        s = SO.decode_step_int8(Xs, dts, An, Bs, Cs, Dn, scales, ref)
        ref = s["h"]
        assert np.array_equal(h.cpu().numpy(), ref), t
        ys.append(_np(y))
        rs.append(s["y"])
    assert H.chan_err(np.stack(ys, 1), np.stack(rs, 1), dtype) <= 5e-2
