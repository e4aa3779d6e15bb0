"""The operators around the SSD block of a Mamba-2 layer, as measurable cases.

A served layer is  residual + RMSNorm -> In Proj -> causal convolution, SiLU and
softplus -> SSD -> gated RMSNorm -> Out Proj.  Each case is one pass through
one of these steps, on tensors of the layer shapes that the library's own
workloads have (1.3B-, 2.7B- and 8B-shaped layers) and on generic odd sizes.

``run`` computes a step either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the
library. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    conv = {"op": "conv", "P": 64, "N": 128, "width": 4}
    step = {"op": "step", "P": 64, "N": 128, "width": 4}
    return [
        # a whole batch of prompts through the 2.7B-shaped layer's convolution
        {"name": "conv_prompts", **conv, "B": 8, "L": 2048, "H": 80, "G": 1, "history": False, "ragged": False,
         "dtype": "fp16"},
        # a chunk of some prompts of different lengths that continue, 8B-shaped layer (B and C in 8 groups)
        {"name": "conv_ragged_chunk", **conv, "B": 3, "L": 701, "H": 128, "G": 8, "history": True, "ragged": True,
         "dtype": "bf16"},
        # one token of one sequence, 1.3B-shaped layer: the latency of a single user
        {"name": "step_one", **step, "B": 1, "H": 64, "G": 1, "path": "float", "dtype": "bf16"},
        # one token of a small batch on the persistent 8-bit state, 2.7B-shaped layer
        {"name": "step_int8", **step, "B": 8, "H": 80, "G": 1, "path": "int8", "dtype": "fp16"},
        # one token of a large serving batch, 2.7B-shaped layer
        {"name": "step_batch", **step, "B": 256, "H": 80, "G": 1, "path": "float", "dtype": "fp16"},
        # before In Proj: a decode batch, the residual in the activations' type
        {"name": "norm_tokens", "op": "norm", "rows": 8, "cols": 2560, "residual": "same", "codes": True,
         "dtype": "fp16"},
        # before In Proj: the prompts, the residual in 32 bits
        {"name": "norm_prompts", "op": "norm", "rows": 16384, "cols": 2560, "residual": "fp32", "codes": True,
         "dtype": "bf16"},
        # before Out Proj: some tokens of the 8B-shaped layer, a norm for each of 8 groups
        {"name": "gated_tokens", "op": "gated", "rows": 37, "H": 128, "P": 64, "G": 8, "codes": True,
         "dtype": "bf16"},
        # before Out Proj: the prompts of the 2.7B-shaped layer
        {"name": "gated_prompts", "op": "gated", "rows": 16384, "H": 80, "P": 64, "G": 1, "codes": True,
         "dtype": "fp16"},
        # Out Proj of a decode batch, 2.7B-shaped layer: the weight is read for eight rows
        {"name": "matmul_tokens", "op": "matmul", "M": 8, "K": 5120, "N": 2560, "bias": True, "dtype": "fp16"},
        # In Proj of a mixed batch of tokens and a short prompt, 1.3B-shaped layer
        {"name": "matmul_mixed", "op": "matmul", "M": 333, "K": 2048, "N": 8512, "bias": False, "dtype": "bf16"},
        # In Proj of the prompts, 2.7B-shaped layer
        {"name": "matmul_prompts", "op": "matmul", "M": 16384, "K": 2560, "N": 10576, "bias": False,
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    """Heads, groups that divide them, channels of a head and of the state."""
    g = rng.choice((1, 1, 2, 4, 8))
    return {"H": g * max(1, _log(rng, 2, most) // g), "G": g, "P": rng.choice((16, 32, 64, 64)),
            "N": rng.choice((16, 32, 64, 128, 128))}


def draw(rng):
    op = rng.choice(("conv", "step", "norm", "gated", "matmul"))
    dtype = rng.choice(("fp16", "bf16", "fp16", "bf16", "fp32"))
    half = dtype != "fp32"
    if op == "conv":
        c = {"op": op, **_heads(rng, 128), "width": rng.choice((2, 3, 4, 4)), "B": _log(rng, 1, 8)}
        channels = c["H"] * c["P"] + 2 * c["G"] * c["N"]
        most = min(4096, 8 * 2048 * 5376 // (2 if half else 4) * 2 // (channels * c["B"]))
        return {**c, "L": _log(rng, 1, max(1, most)), "history": rng.random() < 0.5, "ragged": rng.random() < 0.5,
                "dtype": dtype}
    if op == "step":
        c = {"op": op, **_heads(rng, 128), "width": rng.choice((2, 3, 4, 4))}
        most = min(1024, 256 * 80 * 64 * 128 // (c["H"] * c["P"] * c["N"]))
        # codes that a 32-bit value decides are returned as 16-bit values, so the 8-bit state goes with these types
        return {**c, "B": _log(rng, 1, max(1, most)), "path": rng.choice(("float", "int8")) if half else "float",
                "dtype": dtype}
    if op == "norm":
        cols = _log(rng, 32, 8192)
        cols = cols if rng.random() < 0.3 else max(64, cols // 64 * 64)
        most = min(16384, 16384 * 2560 // cols)
        return {"op": op, "rows": _log(rng, 1, most), "cols": cols, "residual": rng.choice(("none", "same", "fp32")),
                "codes": half and rng.random() < 0.7, "dtype": dtype}
    if op == "gated":
        c = _heads(rng, 128)
        most = min(16384, 16384 * 5120 // (c["H"] * c["P"]) // (1 if half else 2))
        return {"op": op, "rows": _log(rng, 1, most), "H": c["H"], "P": c["P"], "G": c["G"],
                "codes": half and rng.random() < 0.7, "dtype": dtype}
    k, n = 16 * _log(rng, 4, 512), _log(rng, 16, 18560)
    most = min(16384, 16384 * 2560 * 10576 // (k * n))
    return {"op": op, "M": _log(rng, 1, most), "K": k, "N": n, "bias": rng.random() < 0.5, "dtype": dtype}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def _uniform(gen, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=DEVICE)


def _round_away(v):
    return torch.sign(v) * torch.floor(torch.abs(v) + 0.5)


def _layer(c, gen):
    """The layer's constants: convolution, step sizes, decays, skip, 8-bit steps of the state."""
    H, P, N, G, W = c["H"], c["P"], c["N"], c["G"], c["width"]
    cd = H * P + 2 * G * N
    s = {"conv_w": _uniform(gen, -1, 1, cd, W) / math.sqrt(W) * 1.5, "conv_b": 0.1 * _normal(gen, cd)}
    s["dt_bias"] = torch.log(torch.expm1(torch.exp(_uniform(gen, math.log(1e-3), math.log(0.1), H))))
    s["A"] = -torch.exp(_uniform(gen, 0.0, math.log(16.0), H))
    s["D"] = _normal(gen, H)
    return s


def _projected(c, gen, rows):
    """In Proj's output, rows of z | x B C | dt, of which the convolution takes the last two parts in place."""
    H, P, N, G = c["H"], c["P"], c["N"], c["G"]
    d = H * P
    cd = d + 2 * G * N
    full = _normal(gen, *rows, d + cd + H)
    full[..., d:d + cd] *= torch.exp(0.3 * _normal(gen, cd))
    full[..., d + cd:] *= 0.5
    full = full.to(TYPES[c["dtype"]])
    return full, full[..., d:d + cd], full[..., d + cd:]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    t = TYPES[c["dtype"]]
    s = {"case": c, "op": c["op"]}
    if own:
        from mamba_ssd_chunked_amd import _lib as L
        s["L"] = L
    if c["op"] in ("conv", "step"):
        B, H, P, N, G, W = c["B"], c["H"], c["P"], c["N"], c["G"], c["width"]
        cd = H * P + 2 * G * N
        s.update(_layer(c, gen))
        length = c["L"] if c["op"] == "conv" else 1
        full, xbc, raw = _projected(c, gen, (B, length))
        s["xbc"], s["raw"] = (xbc, raw) if c["op"] == "conv" else (xbc[:, 0], raw[:, 0])
        # the inputs of the last W positions, each in slot (position mod W)
        s["ring"] = _normal(gen, B, W, cd).to(t)
        if c["op"] == "conv":
            s["pos"] = torch.randint(0, 5000, (B,), generator=gen, device=DEVICE, dtype=torch.int32) \
                if c["history"] else None
            s["lengths"] = torch.randint(0, length + 1, (B,), generator=gen, device=DEVICE, dtype=torch.int32) \
                if c["ragged"] else None
        else:
            s["pos"] = torch.randint(0, 5000, (B,), generator=gen, device=DEVICE, dtype=torch.int32)
            s["state"] = 0.3 * _normal(gen, B, H, P, N)
            if c["path"] == "int8":
                # static steps: the largest value that calibration saw, over 127
                k = {"s_B": _uniform(gen, 3.0, 4.0, G) / 127, "s_C": _uniform(gen, 3.0, 4.0, G) / 127,
                     "s_X": _uniform(gen, 0.05, 0.2, H, P) / 127, "s_S": _uniform(gen, 0.8, 1.2, H, P) / 127}
                k["inv_B"], k["inv_C"], k["inv_X"] = 1 / k["s_B"], 1 / k["s_C"], 1 / k["s_X"]
                k["M_req"] = k["s_X"] * k["s_B"].repeat_interleave(H // G)[:, None] / k["s_S"]
                s["steps"] = k
                s["state"] = torch.clamp(_round_away(s["state"] / k["s_S"][..., None]), -127, 127).to(torch.int8)
                s["values"] = torch.empty(s["state"].shape, dtype=t, device=DEVICE)
        if own:
            s["conv"] = L.ConvParams(s["conv_w"], s["conv_b"], s["dt_bias"])
            s["shape"] = L.make_shape(B, length, H, P, N, G, 64, c["dtype"])
            if c["op"] == "conv":
                s["out"] = [torch.empty((B, length, H, P), dtype=t, device=DEVICE),
                            torch.empty((B, length, G, N), dtype=t, device=DEVICE),
                            torch.empty((B, length, G, N), dtype=t, device=DEVICE),
                            torch.empty((B, length, H), dtype=t, device=DEVICE)]
            else:
                s["y"] = torch.empty((B, H, P), dtype=t, device=DEVICE)
                s["scales"] = None
                if c["path"] == "int8":
                    s["scales"] = L.ScalePack({n: v.cpu().numpy() for n, v in s["steps"].items()}, DEVICE)
        return s
    if c["op"] == "norm":
        rows, cols = c["rows"], c["cols"]
        s["x"] = _normal(gen, rows, cols).to(t)
        s["weight"] = 1 + 0.1 * _normal(gen, cols)
        rt = {"none": None, "same": t, "fp32": torch.float32}[c["residual"]]
        # the sum of the layers so far, with a few channels far larger than the rest
        size = torch.exp(0.5 * _normal(gen, cols)) * torch.where(_uniform(gen, 0, 1, cols) < 0.01, 10.0, 1.0)
        s["residual"] = (2 * _normal(gen, rows, cols) * size).to(rt) if rt is not None else None
        s["sum"] = torch.empty((rows, cols), dtype=rt if rt is not None else t, device=DEVICE)
    elif c["op"] == "gated":
        rows, cols = c["rows"], c["H"] * c["P"]
        s["y"] = (_normal(gen, rows, cols) * torch.exp(0.3 * _normal(gen, cols))).to(t)
        # z is the first part of In Proj's rows
        wide = cols + cols + 2 * c["G"] * 128 + c["H"]
        s["z"] = _normal(gen, rows, wide).to(t)[:, :cols]
        s["weight"] = 1 + 0.1 * _normal(gen, cols)
    else:
        M, K, N = c["M"], c["K"], c["N"]
        # codes of rows whose largest value is 127: most are far smaller
        s["a"] = torch.clamp(torch.round(32 * _normal(gen, M, K)), -127, 127).to(torch.int8)
        s["w"] = torch.clamp(torch.round(32 * _normal(gen, N, K)), -127, 127).to(torch.int8)
        s["sa"] = _uniform(gen, 2.0, 6.0, M) / 127
        s["sw"] = _uniform(gen, 2.0, 6.0, N) / 127 / math.sqrt(K)
        s["bias"] = 0.1 * _normal(gen, N) if c["bias"] else None
        if own:
            s["out"] = torch.empty((M, N), dtype=t, device=DEVICE)
            s["workspace"] = L.ssd_matmul_i8_workspace(M, N, K, DEVICE)
        return s
    s["out"] = torch.empty((rows, cols), dtype=t, device=DEVICE)
    s["q"] = torch.empty((rows, cols), dtype=torch.int8, device=DEVICE) if c["codes"] else None
    s["scale"] = torch.empty((rows,), device=DEVICE) if c["codes"] else None
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_conv_inputs(s, c, x, length):
    """The convolution's inputs with the W - 1 that went before them, in 32 bits: [B, W - 1 + length, Cd]."""
    B, W = c["B"], c["width"]
    if s["pos"] is None:
        before = torch.zeros((B, W - 1, x.shape[-1]), device=DEVICE)
    else:
        at = s["pos"].long()[:, None] + torch.arange(-(W - 1), 0, device=DEVICE)
        before = s["ring"].float().gather(1, (at % W)[..., None].expand(-1, -1, x.shape[-1]))
        before = torch.where((at >= 0)[..., None], before, torch.zeros((), device=DEVICE))
    return torch.cat([before, x], 1)


def _plain_silu_conv(s, c, x, length):
    W = c["width"]
    padded = _plain_conv_inputs(s, c, x, length)
    if length > 1:
        # tap by tap: the windows as one array would be W times the input
        u = padded[:, 0:length] * s["conv_w"][:, 0] + padded[:, 1:1 + length] * s["conv_w"][:, 1]
        if W > 2:
            u = u + padded[:, 2:2 + length] * s["conv_w"][:, 2]
        if W > 3:
            u = u + padded[:, 3:3 + length] * s["conv_w"][:, 3]
    else:
        u = (padded * s["conv_w"].t()).sum(1, keepdim=True)
    u = u + s["conv_b"]
    return u / (1 + torch.exp(-u))


def _plain_softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _plain_keep(s, c, x, length):
    """The last W inputs of each sequence into their slots."""
    W = c["width"]
    n = s["lengths"].long()[:, None] if s.get("lengths") is not None else torch.full((c["B"], 1), length, device=DEVICE)
    at = n - W + torch.arange(W, device=DEVICE)  # places in this call
    slot = ((s["pos"].long()[:, None] if s["pos"] is not None else 0) + at) % W
    wide = (-1, -1, x.shape[-1])
    old = s["ring"].gather(1, slot[..., None].expand(*wide))
    new = x.gather(1, at.clamp(0)[..., None].expand(*wide)).to(old.dtype)
    s["ring"].scatter_(1, slot[..., None].expand(*wide), torch.where((at >= 0)[..., None], new, old))


def _plain_conv(s):
    c = s["case"]
    B, L, H, P, N, G = (c[k] for k in "BLHPNG")
    t = TYPES[c["dtype"]]
    x = s["xbc"].float()
    v = _plain_silu_conv(s, c, x, L)
    dt = _plain_softplus(s["raw"].float() + s["dt_bias"])
    if s["lengths"] is not None:
        live = (torch.arange(L, device=DEVICE) < s["lengths"][:, None])[..., None]
        zero = torch.zeros((), device=DEVICE)
        v, dt = torch.where(live, v, zero), torch.where(live, dt, zero)
    _plain_keep(s, c, x, L)
    d = H * P
    return [v[..., :d].reshape(B, L, H, P).to(t), v[..., d:d + G * N].reshape(B, L, G, N).to(t),
            v[..., d + G * N:].reshape(B, L, G, N).to(t), dt.to(t), s["ring"]]


def _plain_step(s):
    c = s["case"]
    B, H, P, N, G = (c[k] for k in "BHPNG")
    t = TYPES[c["dtype"]]
    x = s["xbc"].float()[:, None]
    v = _plain_silu_conv(s, c, x, 1)[:, 0]
    dt = _plain_softplus(s["raw"].float() + s["dt_bias"])
    _plain_keep(s, c, x, 1)
    d = H * P
    xh = v[:, :d].reshape(B, H, P)
    bm, cm = v[:, d:d + G * N].reshape(B, G, N), v[:, d + G * N:].reshape(B, G, N)
    if c["path"] == "float":
        bh, ch = bm.repeat_interleave(H // G, 1), cm.repeat_interleave(H // G, 1)
        s["state"].mul_(torch.exp(dt * s["A"])[..., None, None]).add_((dt[..., None] * xh)[..., None] * bh[:, :, None])
        y = (s["state"] * ch[:, :, None]).sum(-1) + s["D"][:, None] * xh
        return [y.to(t), s["state"], s["ring"]]
    k = s["steps"]
    qb = torch.clamp(_round_away(bm * k["inv_B"][:, None]), -127, 127).repeat_interleave(H // G, 1)
    qc = torch.clamp(_round_away(cm * k["inv_C"][:, None]), -127, 127).repeat_interleave(H // G, 1)
    qx = torch.clamp(_round_away((dt[..., None] * xh) * k["inv_X"]), -127, 127)
    sb, sc = k["s_B"].repeat_interleave(H // G), k["s_C"].repeat_interleave(H // G)
    old = s["state"].float()
    # the decay next to a border between two codes is decided in 64 bits
    decay = torch.exp(dt.double() * s["A"].double())
    qd = torch.clamp(torch.floor(128 * decay + 0.5), max=128).float()
    y = (decay.float() * sc)[..., None] * k["s_S"] * (qc[:, :, None] * old).sum(-1)
    y = y + (((qc * qb).sum(-1) * sc * sb * dt)[..., None] + s["D"][:, None]) * xh
    local = torch.clamp(_round_away(qx[..., None] * qb[:, :, None] * k["M_req"][..., None]), -127, 127)
    kept = qd[..., None, None] * old
    kept = torch.sign(kept) * torch.floor((torch.abs(kept) + 64) / 128)
    s["state"].copy_(torch.clamp(local + kept, -127, 127))
    return [y.to(t), torch.mul(s["state"], k["s_S"][..., None], out=s["values"]), s["ring"]]


def _plain_codes(s, y, t):
    """The values that the rows' 8-bit codes stand for, the codes' steps; the rows themselves where no codes are asked for."""
    if not s["case"]["codes"]:
        return [y.to(t)]
    most = y.abs().amax(-1, keepdim=True)
    step = torch.where(most > 0, most / 127, torch.ones((), device=DEVICE))
    q = _round_away(y / step)
    return [(q * step).to(t), step[:, 0]]


def _plain_norm(s):
    t = TYPES[s["case"]["dtype"]]
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    return _plain_codes(s, y, t) + [r.to(s["sum"].dtype)]


def _plain_gated(s):
    c = s["case"]
    t = TYPES[c["dtype"]]
    z = s["z"].float()
    u = s["y"].float() * (z / (1 + torch.exp(-z)))
    g = u.reshape(c["rows"], c["G"], -1)
    y = (g / torch.sqrt((g * g).mean(-1, keepdim=True) + EPS)).reshape(u.shape) * s["weight"]
    return _plain_codes(s, y, t)


def _plain_matmul(s):
    y = s["a"].float() @ s["w"].float().t() * s["sa"][:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[s["case"]["dtype"]])


_plain = {"conv": _plain_conv, "step": _plain_step, "norm": _plain_norm, "gated": _plain_gated,
          "matmul": _plain_matmul}


def _own_conv(s):
    X, B, C, dt = s["out"]
    s["L"].ssd_conv_forward(s["shape"], s["conv"], s["xbc"], s["raw"], X, B, C, dt, s["ring"], s["pos"], s["lengths"])
    return [X, B, C, dt, s["ring"]]


def _own_step(s):
    L = s["L"]
    path = L.SSD_PATH_FLOAT if s["scales"] is None else L.SSD_PATH_INT8
    L.ssd_conv_decode_step(s["shape"], path, s["conv"], s["xbc"], s["raw"], s["A"], s["D"], s["scales"], s["ring"],
                           s["pos"], s["state"], s["y"])
    if s["scales"] is None:
        return [s["y"], s["state"], s["ring"]]
    # what the 8-bit state stands for
    return [s["y"], torch.mul(s["state"], s["steps"]["s_S"][..., None], out=s["values"]), s["ring"]]


def _own_norm(s):
    s["L"].ssd_add_norm(s["x"], s["residual"], s["sum"], s["weight"], EPS, s["out"], s["q"], s["scale"])
    return [s["out"], s["scale"], s["sum"]] if s["q"] is not None else [s["out"], s["sum"]]


def _own_gated(s):
    s["L"].ssd_gated_norm(s["y"], s["z"], s["case"]["G"], s["weight"], EPS, s["out"], s["q"], s["scale"])
    return [s["out"], s["scale"]] if s["q"] is not None else [s["out"]]


def _own_matmul(s):
    s["L"].ssd_matmul_i8(s["a"], s["sa"], s["w"], s["sw"], s["bias"], s["out"], s["workspace"])
    return s["out"]


_own = {"conv": _own_conv, "step": _own_step, "norm": _own_norm, "gated": _own_gated, "matmul": _own_matmul}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] in ("conv", "step"):
        B, H, P, N, W = c["B"], c["H"], c["P"], c["N"], c["width"]
        cd = H * P + 2 * c["G"] * N
        rows = B * c.get("L", 1)
        weights = 4 * cd * (W + 1) + 12 * H
        taps = rows * cd * (2 * W + 5)
        if c["op"] == "conv":
            ring = B * W * cd * e * (2 if c["history"] else 1)
            return {"bytes": 2 * e * rows * (cd + H) + weights + ring, "flops": taps + 6 * rows * H}
        size = 4 if c["path"] == "float" else 1
        values = 0 if c["path"] == "float" else 3  # the 8-bit state is read once more and its values written
        return {"bytes": B * H * P * N * (2 * size + values) + weights + e * B * ((W + 1) * cd + H + H * P),
                "flops": taps + 6 * B * H * P * N}
    if c["op"] in ("norm", "gated"):
        n = c["rows"] * (c["cols"] if c["op"] == "norm" else c["H"] * c["P"])
        codes = n + 4 * c["rows"] if c["codes"] else 0
        if c["op"] == "gated":
            return {"bytes": 3 * e * n + codes + 4 * c["H"] * c["P"], "flops": 13 * n}
        er = {"none": 0, "same": e, "fp32": 4}[c["residual"]]
        return {"bytes": n * (2 * e + er + (er or e)) + codes + 4 * c["cols"], "flops": 8 * n}
    M, K, N = c["M"], c["K"], c["N"]
    return {"bytes": M * K + N * K + e * M * N + 4 * (M + N + (N if c["bias"] else 0)), "flops": 2 * M * N * K}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "step": _exact_step, "norm": _exact_norm, "gated": _exact_gated,
            "matmul": _exact_matmul}[case["op"]](s, case)


def _exact_mixed(s, c, x, pos, ends):
    """silu(convolution) of x [B, L, Cd], and the ring after it; one sequence at a time, from the list of its inputs."""
    W, B, L = c["width"], x.shape[0], x.shape[1]
    w = s["conv_w"].double()
    u = torch.zeros(x.shape, dtype=torch.float64, device=DEVICE)
    ring = s["ring"].double().clone()
    for b in range(B):
        for back in range(W):  # the input `back` positions before the output's
            tap = w[:, W - 1 - back]
            if back < L:
                u[b, back:] += x[b, :L - back] * tap
            for i in range(min(back, L)):
                if pos[b] + i - back >= 0 and s["pos"] is not None:
                    u[b, i] += s["ring"][b, (pos[b] + i - back) % W].double() * tap
        for i in range(max(0, ends[b] - W), ends[b]):
            ring[b, (pos[b] + i) % W] = x[b, i]
    u += s["conv_b"].double()
    return u * torch.sigmoid(u), ring


def _exact_dt(s):
    v = s["raw"].double() + s["dt_bias"].double()
    return torch.logaddexp(v, torch.zeros_like(v))


def _exact_conv(s, c):
    B, L, H, P, N, G = (c[k] for k in "BLHPNG")
    pos = s["pos"].tolist() if s["pos"] is not None else [0] * B
    ends = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    v, ring = _exact_mixed(s, c, s["xbc"].double(), pos, ends)
    dt = _exact_dt(s)
    for b in range(B):
        v[b, ends[b]:] = 0
        dt[b, ends[b]:] = 0
    x, bm, cm = v.split([H * P, G * N, G * N], -1)
    return [x.reshape(B, L, H, P), bm.reshape(B, L, G, N), cm.reshape(B, L, G, N), dt, ring]


def _exact_step(s, c):
    B, H, P, N, G = (c[k] for k in "BHPNG")
    v, ring = _exact_mixed(s, c, s["xbc"].double()[:, None], s["pos"].tolist(), [1] * B)
    x, bm, cm = v[:, 0].split([H * P, G * N, G * N], -1)
    dt = _exact_dt(s).reshape(B, G, H // G)
    x = x.reshape(B, G, H // G, P)
    bm, cm = bm.reshape(B, G, N), cm.reshape(B, G, N)
    decay = torch.exp(dt * s["A"].double().reshape(G, H // G))
    skip = x * s["D"].double().reshape(G, H // G, 1)
    if c["path"] == "float":
        h = s["state"].double().reshape(B, G, H // G, P, N)
        h *= decay[..., None, None]
        h += (x * dt[..., None])[..., None] * bm[:, :, None, None]
        y = torch.matmul(h.reshape(B * G, -1, N), cm.reshape(B * G, N, 1)).reshape(x.shape) + skip
        return [y.reshape(B, H, P), h.reshape(B, H, P, N), ring]

    def code(v):
        return torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).clamp(-127, 127)

    k = {n: v.double() for n, v in s["steps"].items()}
    qb, qc = code(bm / k["s_B"][:, None]), code(cm / k["s_C"][:, None])
    qx = code(x * dt[..., None] / k["s_X"].reshape(G, H // G, P))
    h = s["state"].double().reshape(B, G, H // G, P, N)
    qd = torch.trunc(decay * 128 + 0.5).clamp(max=128)
    ss = k["s_S"].reshape(G, H // G, P)
    off = torch.matmul(h.reshape(B * G, -1, N), qc.reshape(B * G, N, 1)).reshape(x.shape)
    y = off * ss * (decay * k["s_C"][:, None])[..., None] + skip
    y += ((qb * qc).sum(-1) * k["s_B"] * k["s_C"])[..., None, None] * dt[..., None] * x
    new = code(qx[..., None] * qb[:, :, None, None] * k["M_req"].reshape(G, H // G, P, 1))
    h = (new + torch.trunc((qd[..., None, None] * h + torch.copysign(torch.full_like(h, 64.0), h)) / 128)).clamp(-127, 127)
    return [y.reshape(B, H, P), (h * ss[..., None]).reshape(B, H, P, N), ring]


def _exact_codes(c, y):
    if not c["codes"]:
        return [y]
    step = y.abs().max(-1).values / 127
    step[step == 0] = 1
    scaled = y / step[:, None]
    return [torch.trunc(scaled + torch.copysign(torch.full_like(scaled, 0.5), scaled)) * step[:, None], step]


def _exact_norm(s, c):
    r = s["x"].double()
    if s["residual"] is not None:
        r += s["residual"].double()
    y = r * torch.rsqrt(r.square().sum(-1) / c["cols"] + EPS)[:, None] * s["weight"].double()
    return _exact_codes(c, y) + [r]


def _exact_gated(s, c):
    z = s["z"].double()
    u = s["y"].double() * z * torch.sigmoid(z)
    size = u.shape[-1] // c["G"]
    for g in range(c["G"]):
        part = u[:, g * size:(g + 1) * size]
        part *= torch.rsqrt(part.square().sum(-1) / size + EPS)[:, None]
    return _exact_codes(c, u * s["weight"].double())


def _exact_matmul(s, c):
    # products of codes and their sums are whole numbers below 2^53
    y = torch.matmul(s["a"].double(), s["w"].double().t().contiguous())
    y *= s["sa"].double()[:, None]
    y *= s["sw"].double()
    return y if s["bias"] is None else y + s["bias"].double()
