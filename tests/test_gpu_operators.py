"""The gated delta rule, the product with an epilogue and the block norm as they are used:
together in layers, over prompts in pieces and token by token, on streams and in graphs,
and at the edges of what their calls allow."""
import numpy as np
import pytest

from oracle import operators_oracle as OO
from tests import test_gpu_delta as D

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _np(t):
    return t.detach().double().cpu().numpy()


def forward(L, torch, c, unit=True, logit=True, init=True, scale=0.3, eps=1e-6, n=None, start=0, ws="own", stream=None):
    """Y and the final state of positions start .. start + n - 1 of c."""
    B, Ln, H_, P = c["X"].shape
    G, N = c["K"].shape[2:]
    n = Ln - start if n is None else n
    td = {torch.float32: "fp32", torch.float16: "fp16", torch.bfloat16: "bf16"}[c["X"].dtype]
    sh = L.make_shape(B, n, H_, P, N, G, 64, td)
    part = {k: c[k][:, start:start + n].contiguous() for k in ("X", "dt", "K", "Q", "beta")}
    Y = torch.full((B, n, H_, P), NAN, dtype=c["X"].dtype, device="cuda")
    fin = torch.full((B, H_, P, N), NAN, device="cuda")
    ws = L.ssd_delta_workspace(sh) if ws == "own" else ws
    st = c["init"] if init is True else init
    L.ssd_delta_forward(sh, part["X"], part["dt"], c["A"], part["K"], part["Q"], part["beta"], Y, final_state=fin,
                        initial_state=st if st is not False else None, workspace=ws, scale=scale, unit=unit, logit=logit,
                        eps=eps, stream=stream)
    return Y, fin


@pytest.mark.parametrize("dtype", ("fp32", "fp16", "bf16"))
def test_prompts_in_pieces_and_tokens(gpu_lib, dtype):
    """A prompt at once, in pieces that continue one another (each on a path of its own),
    and token by token: the same states and outputs to the bounds of the whole."""
    import torch
    L = gpu_lib
    c = D.make(torch, 21, 2, 150, 6, 32, 64, 2, dtype)
    y, s, ymag, smag = D.reference(c, 0.3, True, True, True)
    at, Y = c["init"], []
    for start, n in ((0, 1), (1, 16), (17, 17), (34, 64), (98, 52)):
        print("piece", start, n, flush=True)
        part, at = forward(L, torch, c, init=at, n=n, start=start)
        Y.append(part)
    torch.cuda.synchronize()
    D.check(_np(at), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state of pieces")
    D.check(_np(torch.cat(Y, 1)), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y of pieces")
    state, Y = c["init"].clone(), torch.empty(2, 150, 6, 32, dtype=c["X"].dtype, device="cuda")
    sh = L.make_shape(2, 1, 6, 32, 64, 2, 64, dtype)
    for t in range(150):
        out = torch.empty(2, 6, 32, dtype=c["X"].dtype, device="cuda")
        L.ssd_delta_step(sh, c["X"][:, t].contiguous(), c["dt"][:, t].contiguous(), c["A"], c["K"][:, t].contiguous(),
                         c["Q"][:, t].contiguous(), c["beta"][:, t], state, out, scale=0.3, logit=True)
        Y[:, t] = out
    torch.cuda.synchronize()
    D.check(_np(state), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state of steps")
    D.check(_np(Y), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y of steps")


def test_delta_forward_without_positions(gpu_lib):
    """The state after no positions: a copy of the one before, or zeros."""
    import torch
    L = gpu_lib
    sh = L.make_shape(3, 0, 4, 16, 32, 2, 64, "fp16")
    e = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    args = (e(3, 0, 4, 16), e(3, 0, 4), -torch.ones(4, device="cuda"), e(3, 0, 2, 32), e(3, 0, 2, 32), e(3, 0, 4))
    init, fin = torch.randn(3, 4, 16, 32, device="cuda"), torch.full((3, 4, 16, 32), NAN, device="cuda")
    L.ssd_delta_forward(sh, *args, e(3, 0, 4, 16), final_state=fin, initial_state=init)
    assert torch.equal(fin, init)
    L.ssd_delta_forward(sh, *args, e(3, 0, 4, 16), final_state=fin)
    assert not fin.any()


@pytest.mark.parametrize("n", (9, 130))
def test_delta_states_in_place_and_not_wanted(gpu_lib, n):
    """initial_state and final_state in one buffer, and no final state: the same outputs."""
    import torch
    L = gpu_lib
    c = D.make(torch, 5, 3, n, 8, 64, 128, 2, "bf16")
    Y, fin = forward(L, torch, c)
    sh = L.make_shape(3, n, 8, 64, 128, 2, 256, "bf16")  # another chunk of the shape: no influence
    both, Y2, Y3 = c["init"].clone(), torch.empty_like(Y), torch.empty_like(Y)
    for fs, y in ((both, Y2), (None, Y3)):
        L.ssd_delta_forward(sh, c["X"], c["dt"], c["A"], c["K"], c["Q"], c["beta"], y, final_state=fs,
                            initial_state=both if fs is not None else c["init"], scale=0.3, logit=True)
    torch.cuda.synchronize()
    assert torch.equal(both, fin) and torch.equal(Y2, Y) and torch.equal(Y3, Y)


def test_delta_positions_that_change_nothing(gpu_lib):
    """dt = 0 and a key of zeros: the state stays, whatever beta and the values are; and a
    beta of zero only forgets."""
    import torch
    L = gpu_lib
    for n in (7, 100):
        c = D.make(torch, 8, 2, n, 4, 16, 32, 1, "fp16", logit=False)
        c["dt"].zero_()
        c["K"].zero_()
        _, fin = forward(L, torch, c, logit=False)
        # held times powers of two and as two parts in between: 22 bits are not lost once fp32 holds them
        assert torch.equal(fin, c["init"])
        c = D.make(torch, 8, 2, n, 4, 16, 32, 1, "fp16", logit=False)
        c["beta"].zero_()
        _, fin = forward(L, torch, c, logit=False)
        s = _np(c["init"]) * np.exp((_np(c["dt"]) * _np(c["A"])).sum(1))[..., None, None]
        assert np.abs(_np(fin) - s).max() <= 2.0 ** -20 * np.abs(s).max()


def test_delta_workspace_of_another_stream(gpu_lib):
    """A workspace that the call takes for itself is none that the current stream still uses, or
    takes again before the call's stream is done."""
    import torch
    L = gpu_lib
    c = D.make(torch, 41, 2, 700, 16, 64, 128, 1, "bf16")
    ref = forward(L, torch, c)
    need = L.ssd_delta_workspace_bytes(L.make_shape(2, 700, 16, 64, 128, 1, 64, "bf16"))
    side = torch.cuda.Stream()
    X, beta = c["X"], c["beta"].contiguous()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream, None):
        busy = torch.empty(need, dtype=torch.uint8, device="cuda")
        for i in range(200):
            busy.fill_(0xff)
        del busy  # the current stream's memory, to be had again by its next request
        sh = L.make_shape(2, 700, 16, 64, 128, 1, 64, "bf16")
        Y, fin = torch.empty_like(c["X"]), torch.empty_like(c["init"])
        ws = L.ssd_delta_forward(sh, X, c["dt"], c["A"], c["K"], c["Q"], beta, Y, final_state=fin, initial_state=c["init"],
                                 scale=0.3, logit=True, stream=given)
        assert ws.numel() == need
        del ws
        again = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff)
        torch.cuda.synchronize()
        assert torch.equal(Y, ref[0]) and torch.equal(fin, ref[1]), given
        del again


@pytest.mark.parametrize("unit", (True, False))
@pytest.mark.parametrize("eps", (0.0, 1e-6))
def test_delta_beta_of_zero_keys(gpu_lib, unit, eps):
    """Whatever stands in beta where the key is zeros, as behind the ends of padded
    sequences, changes nothing: the same bits as with ones there."""
    import torch
    L = gpu_lib
    for dtype in ("fp32", "fp16"):
        for n, logit in ((7, True), (100, False), (130, True)):
            c = D.make(torch, 31, 3, n, 4, 32, 64, 2, dtype, unit=unit, logit=logit)
            for b, end in enumerate((n, n // 2, 1)):
                for k in ("X", "dt", "K", "Q"):
                    c[k][b, end:] = 0
            wide = c["beta"]
            y, s, ymag, smag = D.reference(c, 0.3, unit, logit, True, eps=1e-30 if eps == 0 else eps)
            ones = forward(L, torch, c, unit=unit, logit=logit, eps=eps)
            for bad in (NAN, float("inf"), float("-inf")):
                c["beta"] = wide.clone()
                for b, end in enumerate((n, n // 2, 1)):
                    c["beta"][b, end:] = bad
                Y, fin = forward(L, torch, c, unit=unit, logit=logit, eps=eps)
                assert torch.equal(Y, ones[0]) and torch.equal(fin, ones[1]), (dtype, n, bad)
            D.check(_np(ones[1]), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
            D.check(_np(ones[0]), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y")
            assert not ones[0][1, n // 2:].any()


def test_delta_decays_out_of_range(gpu_lib):
    """dt A below fp32's range: everything before is forgotten, at the ends of the 16 and
    64 positions as within them."""
    import torch
    L = gpu_lib
    for n in (7, 150):
        c = D.make(torch, 33, 1, n, 2, 16, 32, 1, "fp32")
        c["A"][:] = -3e38
        at = [p for p in (0, 3, 5, 15, 16, 40, 63, 64, 100, 101) if p < n]
        c["dt"].zero_()
        c["dt"][:, at] = 3e38
        Y, fin = forward(L, torch, c)
        ref = dict(c, dt=c["dt"] * (1e-32 / 3), A=c["A"] * (1e-34 / 3))  # -1e10: forgotten as well
        y, s, ymag, smag = D.reference(ref, 0.3, True, True, True)
        D.check(_np(fin), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
        D.check(_np(Y), y, ymag, "fp32", D.Y_TAU["fp32"], D.Y_NORM["fp32"], "y")


@pytest.mark.parametrize("dtype", ("fp32", "bf16"))
def test_delta_sizes_of_keys_and_values(gpu_lib, dtype):
    """Keys and queries of any size are taken to length 1; values far from 1 in either
    direction, and rows of zeros, keep their precision."""
    import torch
    L = gpu_lib
    for n in (12, 100):
        c = D.make(torch, 13, 1, n, 4, 32, 64, 1, dtype)
        c["K"][:, ::2] *= 2.0 ** 40
        c["Q"][:, 1::2] *= 2.0 ** 30
        c["K"][:, 5] = 0
        c["Q"][:, 3] = 0
        for size in (2.0 ** -40, 2.0 ** 40):
            d = dict(c, X=c["X"] * size, init=c["init"] * size)
            y, s, ymag, smag = D.reference(d, 0.3, True, True, True)
            Y, fin = forward(L, torch, d)
            D.check(_np(fin), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
            D.check(_np(Y), y, ymag, dtype, D.Y_TAU[dtype], D.Y_NORM[dtype], "y")
        assert not Y[:, 3].any()
    # without eps a key of zeros stays zeros
    Y, fin = forward(L, torch, c, eps=0.0)
    assert torch.isfinite(Y).all() and torch.isfinite(fin).all()


def test_delta_hard_keys(gpu_lib):
    """The same key at every position with strengths up to 2, and keys of alternating sign:
    the triangles whose inverses have the largest entries."""
    import torch
    L = gpu_lib
    c = D.make(torch, 17, 1, 130, 2, 16, 32, 1, "fp32", logit=False)
    c["K"][:] = c["K"][:, :1]
    c["K"][:, 1::2] *= -1
    c["dt"] *= 0.01
    for beta in (1.0, 1.99):
        c["beta"][:] = beta
        y, s, ymag, smag = D.reference(c, 0.3, True, False, True)
        Y, fin = forward(L, torch, c, logit=False)
        # each position's error stays (a strength near 2 mirrors what it meets): 130 positions of 8 roundings
        big = 130 * 8 * 2.0 ** -24 * max(np.abs(s).max(), np.abs(_np(c["X"])).max(), 1)
        assert np.abs(_np(fin) - s).max() <= big
        assert np.abs(_np(Y) - y).max() <= big * 0.3 * 32 ** 0.5


def test_delta_many_chunks_and_strong_decay(gpu_lib):
    """A long sequence, and decays that forget everything within a few positions."""
    import torch
    L = gpu_lib
    c = D.make(torch, 19, 1, 5000, 2, 16, 32, 1, "bf16")
    c["dt"][:, 2000:2100] = 40.0
    y, s, ymag, smag = D.reference(c, 0.3, True, True, True)
    Y, fin = forward(L, torch, c)
    D.check(_np(fin), s, smag, "fp32", 2.0 ** -13, 2.0 ** -18, "state")
    D.check(_np(Y), y, ymag, "bf16", D.Y_TAU["bf16"], D.Y_NORM["bf16"], "y")


@pytest.mark.parametrize("n", (5, 70))
def test_delta_sequences_do_not_touch_each_other(gpu_lib, n):
    """NaN in one sequence's inputs stays in it."""
    import torch
    L = gpu_lib
    c = D.make(torch, 23, 3, n, 4, 64, 64, 2, "fp16")
    Y, fin = forward(L, torch, c)
    for k in ("X", "K", "Q", "dt"):
        bad = dict(c)
        bad[k] = c[k].clone()
        bad[k][1, n // 2] = NAN
        Y2, fin2 = forward(L, torch, bad)
        assert torch.equal(Y2[::2], Y[::2]) and torch.equal(fin2[::2], fin[::2]), k
        assert torch.equal(Y2[1, :n // 2], Y[1, :n // 2]) or n > 16, k  # before it, where positions go one by one


def test_outputs_keep_to_their_buffers(gpu_lib):
    """What lies around Y, the states and the workspace stays as it is."""
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G = 2, 75, 3, 16, 16, 3
    c = D.make(torch, 29, B, Ln, H_, P, N, G, "fp16")
    sh = L.make_shape(B, Ln, H_, P, N, G, 64, "fp16")
    need = L.ssd_delta_workspace_bytes(sh)
    room = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    ybuf = torch.full((B * Ln * H_ * P + 64,), 7.0, dtype=torch.float16, device="cuda")
    sbuf = torch.full((B * H_ * P * N + 64,), 7.0, device="cuda")
    Y, fin = ybuf[32:-32].view(B, Ln, H_, P), sbuf[32:-32].view(B, H_, P, N)
    L.ssd_delta_forward(sh, c["X"], c["dt"], c["A"], c["K"], c["Q"], c["beta"], Y, final_state=fin, initial_state=c["init"],
                        workspace=room[256:-256], scale=0.3, logit=True)
    torch.cuda.synchronize()
    for b, n in ((room, 256), (ybuf, 32), (sbuf, 32)):
        assert (b[:n] == b[0]).all() and (b[-n:] == b[0]).all()
    y, s, ymag, smag = D.reference(c, 0.3, True, True, True)
    D.check(_np(Y), y, ymag, "fp16", D.Y_TAU["fp16"], D.Y_NORM["fp16"], "y")


def layer(torch, seed, dtype, d_model, H_, P, N, G, W=4):
    """Weights of a layer around the gated delta rule: In Proj's rows are z | x B C | dt | beta."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    td = getattr(torch, D.DT[dtype])
    d, cd = H_ * P, H_ * P + 2 * G * N
    rows = d + cd + 2 * H_
    return {"in": (r(rows, d_model) / d_model ** 0.5).to(td), "out": (r(d_model, d) / d ** 0.5).to(td),
            "conv": 0.5 * r(cd, W), "conv_b": 0.1 * r(cd), "dt_b": r(H_) - 3, "A": -torch.exp(r(H_)),
            "norm": 1 + 0.1 * r(d_model), "gate": 1 + 0.1 * r(d), "post": 1 + 0.1 * r(d_model), "next": 1 + 0.1 * r(d_model),
            "bias": 0.1 * r(rows), "d": d, "cd": cd, "rows": rows}


def layer_prompts(L, torch, w, res, dims, lengths=None, stream=None, bufs=None):
    """One layer over prompts: norm, In Proj, convolution, gated delta rule, gated norm, Out Proj,
    block norm. Returns everything that it wrote."""
    B, Ln, H_, P, N, G, dtype = dims
    td = res.dtype
    e = (lambda *s, dt=td: torch.empty(*s, dtype=dt, device="cuda"))
    d, cd = w["d"], w["cd"]
    o = bufs or {"x": e(B, Ln, res.shape[-1]), "r": e(B, Ln, res.shape[-1]), "p": e(B, Ln, w["rows"]), "X": e(B, Ln, H_, P),
                 "K": e(B, Ln, G, N), "Q": e(B, Ln, G, N), "dt": e(B, Ln, H_), "Y": e(B, Ln, H_, P),
                 "S": e(B, H_, P, N, dt=torch.float32), "ring": torch.zeros(B, 4, cd, dtype=td, device="cuda"),
                 "g": e(B, Ln, d), "m": e(B, Ln, res.shape[-1]), "r2": e(B, Ln, res.shape[-1]), "x2": e(B, Ln, res.shape[-1])}
    sh = L.make_shape(B, Ln, H_, P, N, G, 64, dtype)
    if bufs is None:
        o["ws"] = L.ssd_delta_workspace(sh)
    L.ssd_add_norm(res, None, o["r"], w["norm"], 1e-5, o["x"], stream=stream)
    L.ssd_matmul(o["x"], w["in"], w["bias"], o["p"], stream=stream)
    conv = L.ConvParams(w["conv"], w["conv_b"], w["dt_b"])
    L.ssd_conv_forward(sh, conv, o["p"][..., d:d + cd], o["p"][..., d + cd:d + cd + H_], o["X"], o["K"], o["Q"], o["dt"],
                       o["ring"], None, lengths, stream=stream)
    L.ssd_delta_forward(sh, o["X"], o["dt"], w["A"], o["K"], o["Q"], o["p"][..., d + cd + H_:], o["Y"], final_state=o["S"],
                        workspace=o["ws"], scale=N ** -0.5, logit=True, stream=stream)
    L.ssd_gated_norm(o["Y"].view(B, Ln, d), o["p"][..., :d], 1, w["gate"], 1e-5, o["g"], stream=stream)
    L.ssd_matmul(o["g"], w["out"], None, o["m"], stream=stream)
    L.ssd_block_norm(o["m"], w["post"], o["r"], o["r2"], w["next"], 1e-5, o["x2"], stream=stream)
    return o


def layer_reference(w, res, dims, lengths):
    """The same in float64, each call's results rounded to nothing."""
    from oracle import layer_oracle as LO
    B, Ln, H_, P, N, G, dtype = dims
    d, cd = w["d"], w["cd"]
    f = {k: _np(v) for k, v in w.items() if hasattr(v, "detach")}
    r = _np(res)
    x = LO.rms_rows(r.reshape(B * Ln, -1), 1, f["norm"], 1e-5)
    p = (x @ f["in"].T + f["bias"]).reshape(B, Ln, -1)
    u, _ = LO.conv(p[..., d:d + cd], f["conv"], f["conv_b"], np.zeros((B, 3, cd)))
    v, dt = LO.silu(u), LO.softplus(p[..., d + cd:d + cd + H_] + f["dt_b"])
    for b, n in enumerate(lengths):
        v[b, n:] = 0
        dt[b, n:] = 0
    k, q = OO.unit(v[..., d:d + G * N].reshape(B, Ln, G, N), 1e-6), OO.unit(v[..., d + G * N:].reshape(B, Ln, G, N), 1e-6)
    y, s, _, _ = OO.delta(v[..., :d].reshape(B, Ln, H_, P), dt, f["A"], k, q, OO.sigmoid(p[..., d + cd + H_:]), N ** -0.5,
                          np.zeros((B, H_, P, N)))
    z = p[..., :d].reshape(B * Ln, d)
    g = LO.rms_rows(y.reshape(B * Ln, d) * LO.silu(z), 1, f["gate"], 1e-5)
    r2, x2 = OO.block_norm(g @ f["out"].T, f["post"], 1.0, r.reshape(B * Ln, -1), 1.0, f["next"], 1e-5)
    return s, r2.reshape(r.shape), x2.reshape(r.shape)


# relative errors in the 2-norm: eight roundings to the type follow one another (each half a step, and the
# nonlinear steps and norms in between multiply them by less than 2)
LAYER = {"fp32": 1e-5, "fp16": 8 * 2.0 ** -11, "bf16": 8 * 2.0 ** -8}


@pytest.mark.parametrize("dims", [(2, 90, 4, 64, 128, 1, "bf16"), (3, 33, 6, 32, 64, 2, "fp16"), (2, 70, 4, 128, 64, 4, "fp16"),
                                  (2, 10, 4, 16, 32, 2, "fp32"), (1, 130, 3, 64, 64, 1, "fp32")],
                         ids=lambda c: "-".join(map(str, c)))
def test_layer(gpu_lib, dims):
    import torch
    L = gpu_lib
    B, Ln, H_, P, N, G, dtype = dims
    print("layer", dims, flush=True)
    w = layer(torch, 3, dtype, 96, H_, P, N, G)
    g = torch.Generator(device="cuda").manual_seed(4)
    res = torch.randn(B, Ln, 96, generator=g, device="cuda").to(getattr(torch, D.DT[dtype]))
    lengths = [Ln, 1, Ln // 2][:B]
    o = layer_prompts(L, torch, w, res, dims, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    s, r2, x2 = layer_reference(w, res, dims, lengths)
    for what, got, ref in (("state", o["S"], s), ("r", o["r2"], r2), ("x", o["x2"], x2)):
        got = _np(got)
        for b, n in enumerate(lengths):
            a, e = (got[b], ref[b]) if what == "state" else (got[b, :n], ref[b, :n])
            rel = np.linalg.norm(a - e) / np.linalg.norm(e)
            assert rel <= LAYER[dtype], f"{what} of sequence {b}: {rel:.3g}"


def test_layer_on_streams_and_in_graphs(gpu_lib):
    """Two layers on two streams at once, and captured graphs that are replayed among eager
    work: the bits of the eager run each time."""
    import torch
    L = gpu_lib
    dims = (2, 90, 4, 64, 128, 1, "bf16")
    w = layer(torch, 3, "bf16", 96, 4, 64, 128, 1)
    g = torch.Generator(device="cuda").manual_seed(4)
    ins = [torch.randn(2, 90, 96, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [{k: v.clone() for k, v in layer_prompts(L, torch, w, x, dims).items() if k not in ("ws", "ring")} for x in ins]
    torch.cuda.synchronize()

    def same(o, e):
        return all(torch.equal(o[k], e[k]) for k in e)

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for x, st in zip(ins, streams):
        with torch.cuda.stream(st):
            outs.append(layer_prompts(L, torch, w, x, dims))
    torch.cuda.synchronize()
    assert all(same(o, e) for o, e in zip(outs, want))
    graphs = []
    static = [x.clone() for x in ins]
    for x, o in zip(static, outs):
        o["ring"].zero_()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            layer_prompts(L, torch, w, x, dims, bufs=o)
        graphs.append(gr)
    for turn in range(4):
        for i in (0, 1):
            static[i].copy_(ins[(i + turn) % 2])
            for k in want[i]:
                outs[i][k].fill_(1.0)
        torch.cuda.synchronize()
        for st, gr in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                gr.replay()
        layer_prompts(L, torch, w, ins[0], dims)  # eager work beside them
        torch.cuda.synchronize()
        for i in (0, 1):
            assert same(outs[i], want[(i + turn) % 2]), turn


def test_step_in_graph(gpu_lib):
    """A captured step, replayed: each replay takes the state on by one position."""
    import torch
    L = gpu_lib
    c = D.make(torch, 31, 4, 1, 8, 64, 128, 1, "fp16")
    sh = L.make_shape(4, 1, 8, 64, 128, 1, 64, "fp16")
    args = [c[k][:, 0].contiguous() for k in ("X", "dt")] + [c["A"]] + [c[k][:, 0].contiguous() for k in ("K", "Q", "beta")]
    state, Y = c["init"].clone(), torch.empty(4, 8, 64, dtype=torch.float16, device="cuda")
    eager, Ye = c["init"].clone(), torch.empty_like(Y)
    L.ssd_delta_step(sh, *args, c["init"].clone(), Y, logit=True)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        L.ssd_delta_step(sh, *args, state, Y, logit=True)
    state.copy_(c["init"])
    for _ in range(4):
        gr.replay()
        L.ssd_delta_step(sh, *args, eager, Ye, logit=True)
        torch.cuda.synchronize()
        assert torch.equal(state, eager) and torch.equal(Y, Ye)


def test_product_special_values(gpu_lib):
    """Infinities have the activations' limits, NaN stays NaN, and neither leaves its row."""
    import torch
    L = gpu_lib
    for m, k in ((5, 64), (40, 65), (300, 64)):
        a = torch.zeros(m, k, device="cuda")
        a[:, 0] = torch.linspace(-3, 3, m, device="cuda")
        a[1, 0], a[2, 0], a[3, 0] = float("inf"), -float("inf"), NAN
        w = torch.zeros(16, k, device="cuda")
        w[:, 0] = 1
        ref = a[:, :1].double().cpu().numpy()
        for name, code in (("relu", 1), ("relu2", 2), ("silu", 3), ("sigmoid", 4), ("gelu", 5), ("gelu_tanh", 6)):
            out = torch.empty(m, 16, device="cuda")
            L.ssd_matmul(a, w, None, out, act=code)
            got = out.cpu().numpy()
            assert np.isnan(got[3]).all(), name
            top, low = {"sigmoid": (1.0, 0.0)}.get(name, (np.inf, 0.0))
            assert (got[1] == top).all() and (got[2] == low).all(), (name, got[1, 0], got[2, 0])
            rest = [i for i in range(m) if i not in (1, 2, 3)]
            e = OO.activation(ref[rest], name)
            assert np.abs(got[rest] - e).max() <= 40 * 2.0 ** -24 * 9, name


def test_offsets_past_32_bits(gpu_lib):
    """Rows that lie more than 2^32 bytes into their buffers, of each operand."""
    import torch
    L = gpu_lib
    h = torch.float16
    g = torch.Generator(device="cuda").manual_seed(2)
    # a: 2300 rows, 2^20 elements apart; out: 2^31 elements and more
    a = torch.zeros(2300, 1 << 20, dtype=h, device="cuda")
    a[:, 8:72] = torch.randn(2300, 64, generator=g, device="cuda").to(h)
    w = torch.randn(264, 64, generator=g, device="cuda").to(h)
    out = torch.empty(2300, 264, dtype=h, device="cuda")
    few = torch.empty(4, 264, dtype=h, device="cuda")
    ref = a[:, 8:72].float() @ w.float().t()
    L.ssd_matmul(a[:, 8:72], w, None, out)
    assert (out.float() - ref).abs().max() <= 2.0 ** -10 * ref.abs().max()
    L.ssd_matmul(a[-4:, 8:72], w, None, few)
    assert torch.equal(few, out[-4:]) or (few.float() - ref[-4:]).abs().max() <= 2.0 ** -10 * ref.abs().max()
    x = a[:, 8:72]
    y, kept = torch.empty(2300, 64, dtype=h, device="cuda"), torch.empty(2300, 64, dtype=h, device="cuda")
    one = torch.ones(64, device="cuda")
    L.ssd_block_norm(x, one, None, kept, one, 1e-5, y, gate=x)
    part, kp = torch.empty(300, 64, dtype=h, device="cuda"), torch.empty(300, 64, dtype=h, device="cuda")
    L.ssd_block_norm(x[-300:].contiguous(), one, None, kp, one, 1e-5, part, gate=x[-300:].contiguous())
    assert torch.equal(part, y[-300:]) and torch.equal(kp, kept[-300:])
    del a, x
    # the state's last heads
    B, H_, P, N = 70, 520, 128, 128
    st = torch.zeros(B, H_, P, N, device="cuda")
    st[-1] = torch.randn(H_, P, N, generator=g, device="cuda")
    c = D.make(torch, 3, 1, 1, H_, P, N, 1, "fp16")
    rep = {k: c[k][:, 0].expand(B, *c[k].shape[2:]).contiguous() for k in ("X", "dt", "K", "Q", "beta")}
    Y = torch.empty(B, H_, P, dtype=h, device="cuda")
    one_st = st[-1:].clone()
    L.ssd_delta_step(L.make_shape(B, 1, H_, P, N, 1, 64, "fp16"), rep["X"], rep["dt"], c["A"], rep["K"], rep["Q"], rep["beta"], st, Y)
    Y1 = torch.empty(1, H_, P, dtype=h, device="cuda")
    L.ssd_delta_step(L.make_shape(1, 1, H_, P, N, 1, 64, "fp16"), *(rep[k][:1].contiguous() for k in ("X", "dt")), c["A"],
                     *(rep[k][:1].contiguous() for k in ("K", "Q", "beta")), one_st, Y1)
    assert torch.equal(st[-1:], one_st) and torch.equal(Y[-1:], Y1)
    assert (st[:-1].abs().amax() > 0) and torch.equal(st[0], st[-2])


def test_refusals_on_the_gpu(gpu_lib):
    """Tensors of the wrong size, type or place are refused before anything runs."""
    import torch
    L = gpu_lib
    c = D.make(torch, 3, 2, 20, 4, 16, 32, 1, "fp16")
    sh = L.make_shape(2, 20, 4, 16, 32, 1, 64, "fp16")
    Y = torch.empty(2, 20, 4, 16, dtype=torch.float16, device="cuda")

    def call(final=None, init=None, ws=None, **kw):
        v = dict(c, Y=Y)
        v.update(kw)
        L.ssd_delta_forward(sh, v["X"], v["dt"], v["A"], v["K"], v["Q"], v["beta"], v["Y"], final_state=final,
                            initial_state=init, workspace=ws)

    call()
    for k in ("X", "dt", "A", "K", "Q", "beta", "Y"):
        t = Y if k == "Y" else c[k]
        for bad in (t.cpu(), t.double(), t[..., :-1]):
            with pytest.raises(ValueError):
                call(**{k: bad})
    for k in ("X", "K", "Y"):
        with pytest.raises(ValueError, match="contiguous"):
            call(**{k: (Y if k == "Y" else c[k]).transpose(0, 1)})
    for bad in (c["init"].half(), c["init"][:1], c["init"].cpu()):
        with pytest.raises(ValueError):
            call(final=bad)
        with pytest.raises(ValueError):
            call(init=bad)
    with pytest.raises(L.SSDError) as e:
        call(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == L.SSD_E_WORKSPACE
    a, w, o = torch.zeros(4, 64, device="cuda"), torch.zeros(8, 64, device="cuda"), torch.zeros(4, 8, device="cuda")
    L.ssd_matmul(a, w, None, o)
    for args, kw in (((a.half(), w, None, o), {}), ((a, w.cpu(), None, o), {}), ((a, w, o[0].half(), o), {}),
                     ((a, w, None, o[:2]), {}), ((a, w, None, o), {"residual": o.half()}), ((a, w, None, o.t()), {})):
        with pytest.raises(ValueError):
            L.ssd_matmul(*args, **kw)
    with pytest.raises(L.SSDError):
        L.ssd_matmul(a, w, None, o, act=9)
    x, one, out = torch.zeros(6, 16, device="cuda"), torch.ones(16, device="cuda"), torch.zeros(6, 16, device="cuda")
    L.ssd_block_norm(x, one, None, None, one, 1e-5, out, gate=x[:2].contiguous(), rows_per_gate=3)
    for gate, per in ((x[:2].contiguous(), 2), (x[:1], 0), (x.half(), 1), (x[:, :8], 1)):
        with pytest.raises(ValueError):
            L.ssd_block_norm(x, one, None, None, one, 1e-5, out, gate=gate, rows_per_gate=per)
