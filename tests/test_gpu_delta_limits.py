"""The gated delta rule where its numbers reach the ends of what its products hold: states
that grow evenly, values and decays of very different sizes in one chunk, terms that cancel,
values that are not finite.

Bounds as in test_gpu_delta.py, but where a test says otherwise.
"""
import numpy as np
import pytest

from tests import test_gpu_delta as D
from tests.test_gpu_operators import _np, forward

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def inputs(torch, dtype, X, K, Q, dt, A, beta, init=None):
    """Inputs of one sequence from float64 arrays: X [L, H, P], K, Q [L, G, N], dt, beta [L, H], A [H]."""
    td = getattr(torch, D.DT[dtype])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=td)  # noqa: E731
    c = {"X": t(X)[None], "K": t(K)[None], "Q": t(Q)[None], "dt": t(dt)[None], "beta": t(beta)[None]}
    c["A"] = torch.from_numpy(np.asarray(A)).float().cuda()
    H_, P, N = X.shape[1], X.shape[2], K.shape[2]
    s0 = np.zeros((1, H_, P, N)) if init is None else init[None]
    c["init"] = torch.from_numpy(s0).float().cuda()
    return c


def compare(c, dtype, Y, fin, unit, logit, scale=0.3, eps=1e-6):
    y, s, ymag, smag = D.reference(c, scale, unit, logit, True, eps=eps)
    D.check(_np(fin), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
    D.check(_np(Y), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y")


@pytest.mark.parametrize("dtype,unit,k,step,beta,init", [
    # one key, just below a power of two, and values that grow by the same amount
    ("fp32", True, 1.9999, 1.99965, 1.0, 0.0),
    ("fp32", True, 1.9999, 1.99965, 1.0, 0.99),
    ("fp32", False, 1.0 - 2.0 ** -15, 1.99965, 1.0, 0.0),
    ("fp32", False, 1.0 - 2.0 ** -15, 1.99965, 1.0, 0.99),
    # the same value at every position, weakly written
    ("fp32", False, 1.9999, 0.0, 2.0 ** -20, 0.0),
    ("fp16", False, 2047 / 1024, 0.0, 2.0 ** -20, 1.99 * 2.0 ** -20),
    ("bf16", False, 1.9921875, 0.0, 2.0 ** -20, 1.98 * 2.0 ** -20),
], ids=str)
def test_delta_states_that_grow_evenly(gpu_lib, dtype, unit, k, step, beta, init):
    """Changes of one sign and the largest mantissas, whose sum over a chunk is the largest that
    a chunk can add to the state."""
    import torch
    n, H_, P, N = 192, 2, 16, 32
    K = np.zeros((n, 1, N))
    K[..., 0] = k
    Q = np.ones((n, 1, N))
    x = step * (np.arange(n) + 1.0) if step else np.full(n, k)
    X = np.broadcast_to(x[:, None, None], (n, H_, P))
    s0 = np.zeros((H_, P, N))
    s0[..., 0] = init
    c = inputs(torch, dtype, X, K, Q, np.zeros((n, H_)), -np.ones(H_), np.full((n, H_), beta), s0)
    Y, fin = forward(gpu_lib, torch, c, unit=unit, logit=False)
    compare(c, dtype, Y, fin, unit, False)


@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("size", (100.0, 1e4))
def test_delta_large_values_that_are_forgotten(gpu_lib, dtype, size):
    """A large value at a chunk's first position, which its decays forget before its end."""
    import torch
    c = D.make(torch, 61, 2, 200, 3, 32, 64, 1, dtype)
    c["dt"][:] = 0.7
    c["A"][:] = -1.0
    c["X"][:, ::64] *= size
    c["init"].zero_()
    Y, fin = forward(gpu_lib, torch, c)
    compare(c, dtype, Y, fin, True, True)


def test_delta_values_of_different_sizes(gpu_lib):
    """Each position writes a place of its own, one of them a value 4096 times the others. The
    changes and the remainders keep 2^-22 of themselves and 2^-33 of the largest of their
    column, T 2^-22: with the sums, 2^-19 of a value and 2^-30 of the largest."""
    import torch
    rng = np.random.default_rng(5)
    n, H_, P, N = 128, 2, 32, 128
    for big in (0, 40, 63, 100, 127):
        X = rng.standard_normal((n, H_, P))
        X[big] = 4096.0
        K = np.eye(N)[:, None, :]
        Q = rng.standard_normal((n, 1, N))
        c = inputs(torch, "fp32", X, K, Q, np.full((n, H_), 1e-3), -np.ones(H_), np.ones((n, H_)))
        Y, fin = forward(gpu_lib, torch, c, unit=False, logit=False, scale=1.0)
        s = D.reference(c, 1.0, False, False, True)[1]
        err = np.abs(_np(fin) - s)
        assert (err <= 2.0 ** -19 * np.abs(s) + 2.0 ** -30 * 4096).all(), (big, err.max())


@pytest.mark.parametrize("size", (2.0 ** -105, 2.0 ** -60, 2.0 ** 60, 2.0 ** 118))
def test_delta_values_of_any_size(gpu_lib, size):
    """Values far from 1, up to a few steps below fp32's largest, from zeros."""
    import torch
    c = D.make(torch, 63, 1, 150, 2, 32, 64, 1, "fp32")
    d = dict(c, X=c["X"] * size, init=c["init"] * 0)
    y, s, ymag, smag = D.reference(c | {"init": c["init"] * 0}, 0.3, True, True, True)
    Y, fin = forward(gpu_lib, torch, d)
    D.check(_np(fin) / size, s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
    D.check(_np(Y) / size, y, ymag, "fp32", D.Y_TAU["fp32"], D.Y_NORM["fp32"], "y")


@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
@pytest.mark.parametrize("n", (7, 150))
def test_delta_decays_after_one_out_of_range(gpu_lib, dtype, n):
    """Ordinary decays keep their effect behind positions that forget everything."""
    import torch
    c = D.make(torch, 65, 1, n, 2, 32, 64, 1, dtype)
    c["A"][:] = -1.0
    c["dt"][:] = 0.125
    for size in (2.0 ** 11, 2.0 ** 45, 3e38):
        at = [p for p in (2, 10, 64, 100, 101) if p < n]
        d = dict(c, dt=c["dt"].clone())
        d["dt"][:, at] = size
        Y, fin = forward(gpu_lib, torch, d)
        compare(d, dtype, Y, fin, True, True)


@pytest.mark.parametrize("n", (7, 150))
def test_delta_growth(gpu_lib, n):
    """dt A above 0: a state that grows between its writes."""
    import torch
    c = D.make(torch, 67, 2, n, 3, 32, 64, 1, "fp32")
    c["A"] = -c["A"]
    c["A"][1] *= -1
    c["dt"] *= 0.1
    Y, fin = forward(gpu_lib, torch, c)
    compare(c, "fp32", Y, fin, True, True)


def off_from_rounded(torch, Y, y, dtype):
    """The distance of Y from the rounded exact outputs, and that of these from the exact ones,
    relative to y in the 2-norm."""
    r = _np(torch.from_numpy(y).to(Y.dtype))
    return np.linalg.norm(_np(Y) - r) / np.linalg.norm(y), np.linalg.norm(r - y) / np.linalg.norm(y)


@pytest.mark.parametrize("dtype,bound", (("bf16", 2.0 ** -11), ("fp16", 2.0 ** -14.5)))
@pytest.mark.parametrize("case", [(2, 40, 8, 32, 64, 1), (1, 64, 6, 64, 128, 2), (1, 130, 4, 128, 32, 1), (2, 300, 4, 64, 128, 1)],
                         ids=lambda c: "-".join(map(str, c)))
def test_delta_outputs_are_rounded_once(gpu_lib, case, dtype, bound):
    """What Y loses is its rounding. A value that is d off before it goes to its other neighbour,
    a step s away, with probability |d| / s, so that differences from the rounded exact values
    have a mean square of |d| s. bf16: terms kept to 2^-15, s <= 2^-7 |y|: 2^-22 y^2, 2^-11 in the
    2-norm. fp16: terms kept to 2^-19 by their sums and 22 bits, s <= 2^-10 |y|: 2^-29 y^2."""
    import torch
    B, Ln, H_, P, N, G = case
    print("delta", case, dtype, flush=True)
    c = D.make(torch, 51, B, Ln, H_, P, N, G, dtype)
    Y, fin = forward(gpu_lib, torch, c)
    y, s, ymag, smag = D.reference(c, 0.3, True, True, True)
    off, own = off_from_rounded(torch, Y, y, dtype)
    assert off <= bound, off
    # and Y is as far from the exact outputs as the rounding is
    rel = np.linalg.norm(_np(Y) - y) / np.linalg.norm(y)
    assert rel <= own * (1 + 2.0 ** -8), (rel, own)


@pytest.mark.parametrize("dtype", ("fp32", "fp16", "bf16"))
def test_delta_outputs_whose_terms_cancel(gpu_lib, dtype):
    """Queries that see little of a large state: its parts cancel 256 times over in Y. They are
    kept to 2^-22 of the largest of a row of the state, and summed in fp32: N / 2 roundings of
    the largest partial sum at most, far less than Y's own rounding in 16 bits."""
    import torch
    rng = np.random.default_rng(9)
    n, H_, P, N = 100, 2, 32, 64
    half = rng.standard_normal((n, 1, N // 2))
    Q = np.concatenate([half, -half], -1)
    K = rng.standard_normal((n, 1, N))
    K -= K.mean(-1, keepdims=True)
    s0 = 30.0 + 0.1 * rng.standard_normal((H_, P, N))
    c = inputs(torch, dtype, 0.1 * rng.standard_normal((n, H_, P)), K, Q, np.zeros((n, H_)), -np.ones(H_), np.full((n, H_), 0.01),
               s0)
    Y, fin = forward(gpu_lib, torch, c, logit=False)
    y, s, ymag, smag = D.reference(c, 0.3, True, False, True)
    cancel = np.median(ymag) / np.sqrt((y * y).mean())
    assert cancel > 256
    half_step = {"fp32": 0.0, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    rel = np.linalg.norm(_np(Y) - y) / np.linalg.norm(y)
    assert rel <= half_step + cancel * 2.0 ** -19, rel


def hidden_ends(c, n):
    """Where sequences end that are padded with dt = 0 and keys of zeros."""
    ends = (n, n // 2, 1)
    for b, end in enumerate(ends):
        for k in ("dt", "K"):
            c[k][b, end:] = 0
    return ends


@pytest.mark.parametrize("dtype", ("fp32", "fp16", "bf16"))
@pytest.mark.parametrize("n,P", ((7, 32), (12, 16), (100, 32), (130, 64), (130, 128)))
def test_delta_values_of_zero_keys(gpu_lib, dtype, n, P):
    """Whatever stands in X where the key is zeros, as behind the ends of padded sequences,
    reaches neither the state nor another position's outputs."""
    import torch
    c = D.make(torch, 71, 3, n, 4, P, 64, 2, dtype)
    ends = hidden_ends(c, n)
    want = forward(gpu_lib, torch, c)
    for bad in (NAN, INF, -INF):
        d = dict(c, X=c["X"].clone(), beta=c["beta"].clone())
        for b, end in enumerate(ends):
            d["X"][b, end:] = bad
            d["beta"][b, end:] = bad
        Y, fin = forward(gpu_lib, torch, d)
        assert torch.equal(fin, want[1]), bad
        assert torch.equal(Y, want[0]), bad


@pytest.mark.parametrize("bad", (NAN, INF))
@pytest.mark.parametrize("dtype", ("fp32", "fp16", "bf16"))
def test_delta_chunks_before_a_value_that_is_not_finite(gpu_lib, dtype, bad):
    """A value that is not finite leaves all outputs before its 64 positions, those of other
    sequences and of heads that do not read it as they are."""
    import torch
    c = D.make(torch, 73, 3, 200, 4, 32, 64, 2, dtype)
    Y, fin = forward(gpu_lib, torch, c)
    for k in ("X", "K", "Q", "dt", "beta"):
        for at in (64, 140, 199):
            d = dict(c)
            d[k] = c[k].clone()
            d[k][1, at, 0] = bad
            Y2, fin2 = forward(gpu_lib, torch, d)
            first = at // 64 * 64
            assert torch.equal(Y2[::2], Y[::2]) and torch.equal(fin2[::2], fin[::2]), (k, at)
            assert torch.equal(Y2[1, :first], Y[1, :first]), (k, at)
            assert torch.equal(Y2[1, :, 2:], Y[1, :, 2:]) and torch.equal(fin2[1, 2:], fin[1, 2:]), (k, at)


def test_delta_one_position_of_more_heads_than_a_launch_of_four_passes_holds(gpu_lib):
    """2^22 heads of 128 x 128 and more, which without a state before or after is a GB: every
    output is scale beta x (k.q), to half a step of fp16 and 2^-16 for the sum of 128 terms."""
    import torch
    L = gpu_lib
    B, H_, P, N = 65535, 65, 128, 128
    assert B * H_ > 1 << 22
    g = torch.Generator(device="cuda").manual_seed(77)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
    X, K, Q, beta = r(B, 1, H_, P), r(B, 1, 1, N), r(B, 1, 1, N), r(B, 1, H_)
    dt, A = torch.ones(B, 1, H_, dtype=torch.float16, device="cuda"), -torch.ones(H_, device="cuda")
    Y = torch.full_like(X, NAN)
    L.ssd_delta_forward(L.make_shape(B, 1, H_, P, N, 1, 64, "fp16"), X, dt, A, K, Q, beta, Y, scale=0.1, unit=False)
    torch.cuda.synchronize()
    for b in range(0, B, 4096):
        kq = (K[b:b + 4096].double() * Q[b:b + 4096].double())
        y = 0.1 * beta[b:b + 4096].double()[..., None] * X[b:b + 4096].double() * kq.sum(-1, keepdim=True)
        mag = 0.1 * (beta[b:b + 4096].double()[..., None] * X[b:b + 4096].double()).abs() * kq.abs().sum(-1, keepdim=True)
        assert ((Y[b:b + 4096].double() - y).abs() <= 2.0 ** -11 * y.abs() + 2.0 ** -16 * mag + 2.0 ** -25).all(), b


@pytest.mark.parametrize("dtype", ("fp32", "fp16", "bf16"))
@pytest.mark.parametrize("case", [(2, 70, 6, 64, 64, 2), (1, 200, 4, 32, 16, 2), (1, 130, 3, 128, 128, 1), (1, 300, 2, 16, 32, 1)],
                         ids=lambda c: "-".join(map(str, c)))
def test_delta_keys_of_different_lengths(gpu_lib, case, dtype):
    """Keys and queries that are not taken to length 1 and differ in length by factors of
    thousands, with strengths as their stability asks: every row of the state to 2^-18 in the
    2-norm, and Y's positions to its rounding and 2^-13 of their magnitudes."""
    import torch
    B, Ln, H_, P, N, G = case
    c = D.make(torch, 81, B, Ln, H_, P, N, G, dtype, unit=False, logit=False)
    g = torch.Generator(device="cuda").manual_seed(82)
    for k in ("K", "Q"):
        size = torch.exp(2 * torch.randn(B, Ln, G, 1, generator=g, device="cuda"))
        c[k] = (c[k].float() * size).to(c[k].dtype)
    length = (c["K"].float() ** 2).sum(-1).repeat_interleave(H_ // G, 2)
    c["beta"] = (1.9 * torch.rand(B, Ln, H_, generator=g, device="cuda") / length).clamp(max=30000.0).to(c["X"].dtype)
    Y, fin = forward(gpu_lib, torch, c, unit=False, logit=False)
    y, s, ymag, smag = D.reference(c, 0.3, False, False, True)
    rows = lambda a: np.linalg.norm(a, axis=-1)  # noqa: E731
    assert (rows(_np(fin) - s) <= 2.0 ** -18 * rows(s)).all(), (rows(_np(fin) - s) / rows(s)).max()
    half_step = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    # (half the smallest step of fp16, where outputs are that small)
    bound = half_step * rows(y) + 2.0 ** -13 * rows(ymag) + (P ** 0.5 * 2.0 ** -25 if dtype == "fp16" else 0)
    assert (rows(_np(Y) - y) <= bound).all(), (rows(_np(Y) - y) / bound).max()
    D.check(_np(Y), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y")
