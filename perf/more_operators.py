"""Operators of layers that stand beside the SSD block, as measurable cases.

The gated delta rule takes the SSD's place in a layer (its chunked form for
prompts, its recurrent form for single tokens), the product with bias,
activation and residual is the projection of a layer in 16 or 32 bits, and the
block norm joins a block's output to the residual between two norms. Each case
is one pass through one of them, on the layer shapes that the library's own
workloads have (1.3B-, 2.7B- and 8B-shaped layers) and on generic odd sizes.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, where ``own`` is true,
through the library. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5        # of the row norms
EPS_UNIT = 1e-6   # of keys' and queries' lengths
CHUNK = 64        # positions that the plain form takes at a time


def listed():
    unit = {"unit": True, "logit": True}
    return [
        # one user's prompt, 1.3B-shaped layer
        {"name": "delta_one_prompt", "op": "delta", "B": 1, "L": 2048, "H": 64, "G": 1, "P": 64, "N": 128, **unit,
         "history": False, "dtype": "bf16"},
        # a whole batch of prompts, 2.7B-shaped layer
        {"name": "delta_prompts", "op": "delta", "B": 8, "L": 2048, "H": 80, "G": 1, "P": 64, "N": 128, **unit,
         "history": False, "dtype": "fp16"},
        # chunks of prompts that continue, 8B-shaped layer (keys and queries in 8 groups)
        {"name": "delta_continued", "op": "delta", "B": 3, "L": 701, "H": 128, "G": 8, "P": 64, "N": 128, **unit,
         "history": True, "dtype": "bf16"},
        # long prompts, few wide heads that share keys and queries in pairs
        {"name": "delta_wide_heads", "op": "delta", "B": 4, "L": 4096, "H": 32, "G": 16, "P": 128, "N": 128, **unit,
         "history": False, "dtype": "bf16"},
        # one token of one sequence, 1.3B-shaped layer: the latency of a single user
        {"name": "delta_step_one", "op": "delta_step", "B": 1, "H": 64, "G": 1, "P": 64, "N": 128, **unit,
         "dtype": "bf16"},
        # one token of a large serving batch, 2.7B-shaped layer
        {"name": "delta_step_batch", "op": "delta_step", "B": 256, "H": 80, "G": 1, "P": 64, "N": 128, **unit,
         "dtype": "fp16"},
        # Out Proj of a decode batch with the residual, 2.7B-shaped layer: the weight is read for eight rows
        {"name": "product_tokens", "op": "product", "M": 8, "K": 5120, "N": 2560, "bias": False, "act": "none",
         "residual": True, "out": "same", "part": False, "dtype": "fp16"},
        # a block's first product for a mixed batch, with its activation; rows are a part of wider ones
        {"name": "product_mixed", "op": "product", "M": 333, "K": 2048, "N": 8512, "bias": True, "act": "silu",
         "residual": False, "out": "same", "part": True, "dtype": "bf16"},
        # sizes that are aligned to nothing, the sum kept in 32 bits
        {"name": "product_odd", "op": "product", "M": 1065, "K": 2579, "N": 4099, "bias": True, "act": "gelu",
         "residual": True, "out": "fp32", "part": False, "dtype": "bf16"},
        # In Proj of the prompts, 2.7B-shaped layer
        {"name": "product_prompts", "op": "product", "M": 16384, "K": 2560, "N": 10576, "bias": False,
         "act": "none", "residual": False, "out": "same", "part": False, "dtype": "fp16"},
        # between two blocks: a decode batch, a learned gate for each channel
        {"name": "block_norm_tokens", "op": "block_norm", "rows": 8, "cols": 2560, "residual": "same",
         "gate": "channel", "act": "none", "codes": True, "dtype": "fp16"},
        # between two blocks: the prompts, a gate for each token and channel, the residual in 32 bits
        {"name": "block_norm_prompts", "op": "block_norm", "rows": 16384, "cols": 2560, "residual": "fp32",
         "gate": "token", "act": "sigmoid", "codes": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("delta", "delta", "delta_step", "product", "product", "block_norm"))
    dtype = rng.choice(("fp16", "bf16", "fp16", "bf16", "fp32"))
    half = dtype != "fp32"
    if op in ("delta", "delta_step"):
        g = rng.choice((1, 1, 2, 4, 8, 16))
        c = {"op": op, "H": g * max(1, _log(rng, 2, 128) // g), "G": g, "P": rng.choice((16, 32, 64, 64, 128)),
             "N": rng.choice((16, 32, 64, 128, 128)), "unit": rng.random() < 0.8, "logit": rng.random() < 0.7,
             "dtype": dtype}
        size = c["H"] * c["P"] * c["N"]
        if op == "delta_step":
            return {**c, "B": _log(rng, 1, max(1, min(1024, 256 * 80 * 64 * 128 // size)))}
        c["B"] = _log(rng, 1, 8)
        most = 8 * 2048 * 80 * 64 * 128 // (1 if half else 4) // (size * c["B"])
        return {**c, "L": _log(rng, 1, max(1, min(4096, most))), "history": rng.random() < 0.5}
    if op == "product":
        k, n = _log(rng, 64, 8192), _log(rng, 16, 18560)
        if rng.random() < 0.7:
            k, n = k // 64 * 64, max(16, n // 16 * 16)
        most = min(16384, 16384 * 2560 * 10576 // (k * n) // (1 if half else 8))
        return {"op": op, "M": _log(rng, 1, max(1, most)), "K": k, "N": n, "bias": rng.random() < 0.5,
                "act": rng.choice(("none", "none", "relu", "relu2", "silu", "gelu", "gelu_tanh", "sigmoid")),
                "residual": rng.random() < 0.5, "out": rng.choice(("same", "same", "fp32")),
                "part": rng.random() < 0.3, "dtype": dtype}
    cols = _log(rng, 32, 8192)
    cols = cols if rng.random() < 0.3 else max(64, cols // 64 * 64)
    return {"op": op, "rows": _log(rng, 1, min(16384, 16384 * 2560 // cols)), "cols": cols,
            "residual": rng.choice(("none", "same", "fp32")), "gate": rng.choice(("none", "channel", "token")),
            "act": rng.choice(("none", "sigmoid", "silu")), "codes": half and rng.random() < 0.5, "dtype": dtype}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE)


def _uniform(gen, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(*shape, generator=gen, device=DEVICE)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    t = TYPES[c["dtype"]]
    s = {"case": c, "op": c["op"]}
    if own:
        from mamba_ssd_chunked_amd import _lib as L
        s["L"] = L
    if c["op"] in ("delta", "delta_step"):
        B, H, P, N, G = (c[k] for k in "BHPNG")
        n = c.get("L", 1)
        at = (B, n) if c["op"] == "delta" else (B,)
        s["X"] = (_normal(gen, *at, H, P) * torch.exp(0.3 * _normal(gen, H, P))).to(t)
        # keys and queries of length about 1 where the operator does not make them so
        size = torch.exp(0.3 * _normal(gen, G, N)) * (1.0 if c["unit"] else 0.8 / math.sqrt(N))
        s["K"], s["Q"] = (_normal(gen, *at, G, N) * size).to(t), (_normal(gen, *at, G, N) * size).to(t)
        bias = torch.log(torch.expm1(torch.exp(_uniform(gen, math.log(1e-3), math.log(0.1), H))))
        raw = 0.5 * _normal(gen, *at, H) + bias
        s["dt"] = (torch.clamp(raw, min=0) + torch.log1p(torch.exp(-torch.abs(raw)))).to(t)
        s["A"] = -torch.exp(_uniform(gen, 0.0, math.log(16.0), H))
        # the write strengths are the last columns of In Proj's rows
        wide = _normal(gen, *at, 3 * H)
        s["beta"] = (wide if c["logit"] else torch.sigmoid(wide)).to(t)[..., 2 * H:]
        s["scale"] = 1.0 / math.sqrt(N)
        s["state"] = 0.3 * _normal(gen, B, H, P, N) if c.get("history", True) else None
        if own:
            s["shape"] = L.make_shape(B, n, H, P, N, G, 64, c["dtype"])
            s["Y"] = torch.empty(*at, H, P, dtype=t, device=DEVICE)
            if c["op"] == "delta":
                s["final"] = torch.empty(B, H, P, N, device=DEVICE)
                s["workspace"] = L.ssd_delta_workspace(s["shape"], DEVICE)
        return s
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        # rows on their own, or the middle of wider ones
        s["a"] = _normal(gen, M, 2 * K + 64).to(t)[:, 64:64 + K] if c["part"] else _normal(gen, M, K).to(t)
        s["w"] = (_normal(gen, N, K) / math.sqrt(K)).to(t)
        s["bias"] = 0.1 * _normal(gen, N) if c["bias"] else None
        ot = torch.float32 if c["out"] == "fp32" else t
        s["residual"] = (2 * _normal(gen, M, N)).to(ot) if c["residual"] else None
        s["out"] = torch.empty((M, N), dtype=ot, device=DEVICE)
        if own:
            s["workspace"] = L.ssd_matmul_workspace(s["a"], s["w"], s["out"])
        return s
    rows, cols = c["rows"], c["cols"]
    size = torch.exp(0.5 * _normal(gen, cols)) * torch.where(_uniform(gen, 0, 1, cols) < 0.01, 10.0, 1.0)
    s["x"] = (_normal(gen, rows, cols) * torch.exp(0.3 * _normal(gen, cols))).to(t)
    s["post"], s["weight"] = 1 + 0.1 * _normal(gen, cols), 1 + 0.1 * _normal(gen, cols)
    rt = {"none": None, "same": t, "fp32": torch.float32}[c["residual"]]
    s["residual"] = (2 * _normal(gen, rows, cols) * size).to(rt) if rt is not None else None
    s["gate"] = {"none": lambda: None, "channel": lambda: (1 + 0.3 * _normal(gen, 1, cols)).to(t),
                 # a part of the rows of the product before
                 "token": lambda: _normal(gen, rows, cols + 64).to(t)[:, :cols]}[c["gate"]]()
    s["sum"] = torch.empty((rows, cols), dtype=rt if rt is not None else t, device=DEVICE)
    s["out"] = torch.empty((rows, cols), dtype=t, device=DEVICE)
    s["q"] = torch.empty((rows, cols), dtype=torch.int8, device=DEVICE) if c["codes"] else None
    s["step"] = torch.empty((rows,), device=DEVICE) if c["codes"] else None
    s["res_scale"] = 0.7071
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_unit(v, c):
    v = v.float()
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) + EPS_UNIT) if c["unit"] else v


def _plain_beta(s):
    b = s["beta"].float()
    return 1 / (1 + torch.exp(-b)) if s["case"]["logit"] else b


def _plain_delta_step(s):
    c = s["case"]
    r = c["H"] // c["G"]
    k = _plain_unit(s["K"], c).repeat_interleave(r, -2)
    q = _plain_unit(s["Q"], c).repeat_interleave(r, -2) * s["scale"]
    h = s["state"].mul_(torch.exp(s["dt"].float() * s["A"])[..., None, None])
    u = _plain_beta(s)[..., None] * (s["X"].float() - (h * k[:, :, None]).sum(-1))
    h.add_(u[..., None] * k[:, :, None])
    return [(h * q[:, :, None]).sum(-1).to(s["X"].dtype), h]


def _plain_chunks(v, c, n):
    """[B, L, heads, ...] as [B, heads, chunks, positions, ...], zeros behind the end."""
    v = torch.cat([v, v.new_zeros((c["B"], n * CHUNK - c["L"]) + v.shape[2:])], 1)
    return v.reshape((c["B"], n, CHUNK) + v.shape[2:]).movedim(3, 1)


def _plain_inverse(lower):
    """(1 + lower)^-1 of strictly lower triangles: inverses of two diagonal blocks make that of a block twice as large."""
    at = torch.arange(CHUNK, device=DEVICE)
    inverse = torch.eye(CHUNK, device=DEVICE) - lower * ((at % 2 == 1)[:, None] & (at[:, None] == at + 1))
    for size in (2, 4, 8, 16, 32):
        beside = ((at // size) % 2 == 1)[:, None] & (at[:, None] // size == at // size + 1)
        inverse = inverse - inverse @ (lower * beside) @ inverse
    return inverse


def _plain_delta(s):
    c = s["case"]
    n = -(-c["L"] // CHUNK)
    r = c["H"] // c["G"]
    k, q = (_plain_chunks(_plain_unit(s[v], c), c, n) for v in "KQ")
    q = q * s["scale"]
    v, beta = _plain_chunks(s["X"].float(), c, n), _plain_chunks(_plain_beta(s), c, n)[..., None]
    # decays from the start of a chunk: sums in 64 bits, of which differences are taken
    g = _plain_chunks(s["dt"].double() * s["A"].double(), c, n).cumsum(-1)
    at = torch.arange(CHUNK, device=DEVICE)
    back = (at[:, None] >= at)
    gamma = torch.exp(torch.where(back, g[..., :, None] - g[..., None, :], -math.inf)).float()
    first, rest = torch.exp(g).float()[..., None], torch.exp(g[..., -1:] - g).float()[..., None]
    kh, qh = k.repeat_interleave(r, 1), q.repeat_interleave(r, 1)
    within = (q @ k.transpose(-1, -2)).repeat_interleave(r, 1) * gamma
    lower = beta * (k @ k.transpose(-1, -2)).repeat_interleave(r, 1) * gamma * (at[:, None] > at)
    both = _plain_inverse(lower) @ (beta * torch.cat([v, first * kh], -1))
    new, old = both[..., :c["P"]], both[..., c["P"]:]
    kh, qh, last = kh * rest, qh * first, first[..., -1:, :]
    h = s["state"] if s["state"] is not None else torch.zeros((c["B"], c["H"], c["P"], c["N"]), device=DEVICE)
    y = torch.empty(v.shape, device=DEVICE)
    for i in range(n):  # a chunk needs the state that the one before leaves
        u = new[:, :, i] - old[:, :, i] @ h.transpose(-1, -2)
        y[:, :, i] = qh[:, :, i] @ h.transpose(-1, -2) + within[:, :, i] @ u
        h = last[:, :, i] * h + u.transpose(-1, -2) @ kh[:, :, i]
    return [y.movedim(1, 3).reshape(c["B"], n * CHUNK, c["H"], c["P"])[:, :c["L"]].to(s["X"].dtype), h]


def _plain_act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "relu2":
        return torch.clamp(v, min=0) * torch.clamp(v, min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_product(s):
    y = s["a"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _plain_act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out"].dtype)


def _plain_rms(v, w):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * w


def _plain_block_norm(s):
    c = s["case"]
    t = TYPES[c["dtype"]]
    r = _plain_rms(s["x"].float(), s["post"])
    if s["gate"] is not None:
        r = r * _plain_act(s["gate"].float(), c["act"])
    if s["residual"] is not None:
        r = r + s["res_scale"] * s["residual"].float()
    y = _plain_rms(r, s["weight"])
    kept = r.to(s["sum"].dtype)
    if not c["codes"]:
        return [y.to(t), kept]
    # the values that the rows' 8-bit codes stand for, and the codes' steps
    most = y.abs().amax(-1, keepdim=True)
    step = torch.where(most > 0, most / 127, torch.ones((), device=DEVICE))
    v = y / step
    return [(torch.sign(v) * torch.floor(torch.abs(v) + 0.5) * step).to(t), step[:, 0], kept]


_plain = {"delta": _plain_delta, "delta_step": _plain_delta_step, "product": _plain_product,
          "block_norm": _plain_block_norm}


def _own_delta(s):
    c = s["case"]
    s["L"].ssd_delta_forward(s["shape"], s["X"], s["dt"], s["A"], s["K"], s["Q"], s["beta"], s["Y"],
                             final_state=s["final"], initial_state=s["state"], workspace=s["workspace"],
                             scale=s["scale"], unit=c["unit"], logit=c["logit"], eps=EPS_UNIT)
    return [s["Y"], s["final"]]


def _own_delta_step(s):
    c = s["case"]
    s["L"].ssd_delta_step(s["shape"], s["X"], s["dt"], s["A"], s["K"], s["Q"], s["beta"], s["state"], s["Y"],
                          scale=s["scale"], unit=c["unit"], logit=c["logit"], eps=EPS_UNIT)
    return [s["Y"], s["state"]]


def _own_product(s):
    L = s["L"]
    L.ssd_matmul(s["a"], s["w"], s["bias"], s["out"], act=getattr(L, "SSD_ACT_" + s["case"]["act"].upper()),
                 residual=s["residual"], workspace=s["workspace"])
    return s["out"]


def _own_block_norm(s):
    L, c = s["L"], s["case"]
    L.ssd_block_norm(s["x"], s["post"], s["residual"], s["sum"], s["weight"], EPS, s["out"], s["q"], s["step"],
                     gate=s["gate"], gate_act=getattr(L, "SSD_ACT_" + c["act"].upper()),
                     rows_per_gate=c["rows"] if c["gate"] == "channel" else 1, res_scale=s["res_scale"])
    return [s["out"], s["step"], s["sum"]] if c["codes"] else [s["out"], s["sum"]]


_own = {"delta": _own_delta, "delta_step": _own_delta_step, "product": _own_product, "block_norm": _own_block_norm}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] in ("delta", "delta_step"):
        B, H, P, N, G = (c[k] for k in "BHPNG")
        n = B * c.get("L", 1)
        states = 4 * B * H * P * N * (2 if c.get("history", True) else 1)
        # a position's decay, product with the key, update and product with the query
        return {"bytes": e * n * (2 * H * P + 2 * G * N + 2 * H) + 4 * H + states, "flops": 7 * n * H * P * N}
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        eo = 4 if c["out"] == "fp32" else e
        return {"bytes": e * (M * K + N * K) + eo * M * N * (2 if c["residual"] else 1) + (4 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    n = c["rows"] * c["cols"]
    er = {"none": 0, "same": e, "fp32": 4}[c["residual"]]
    gate = {"none": 0, "channel": e * c["cols"], "token": e * n}[c["gate"]]
    codes = n + 4 * c["rows"] if c["codes"] else 0
    return {"bytes": n * (2 * e + er + (er or e)) + gate + codes + 8 * c["cols"], "flops": 14 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "delta_step": _exact_delta, "product": _exact_product,
            "block_norm": _exact_block_norm}[case["op"]](s, case)


def _exact_delta(s, c):
    """The recurrence, one position after the other."""
    B, H, P, N, G = (c[k] for k in "BHPNG")
    n = c.get("L", 1)
    x, k, q = (s[v].double().reshape(B, n, -1, s[v].shape[-1]) for v in "XKQ")
    if c["unit"]:
        k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + EPS_UNIT)
        q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + EPS_UNIT)
    q = q * s["scale"]
    beta = s["beta"].double().reshape(B, n, H)
    beta = torch.sigmoid(beta) if c["logit"] else beta
    decay = torch.exp(s["dt"].double().reshape(B, n, H) * s["A"].double())
    h = torch.zeros((B * G, H // G * P, N), dtype=torch.float64, device=DEVICE)
    if s["state"] is not None:
        h += s["state"].double().reshape(h.shape)
    y = torch.empty((B, n, H, P), dtype=torch.float64, device=DEVICE)
    for t in range(n):
        h *= decay[:, t].repeat_interleave(P, -1).reshape(B * G, -1, 1)
        kt = k[:, t].reshape(B * G, N, 1)
        u = beta[:, t].repeat_interleave(P, -1).reshape(B * G, -1, 1) * (
            x[:, t].reshape(B * G, -1, 1) - torch.matmul(h, kt))
        h += u * kt.reshape(B * G, 1, N)
        y[:, t] = torch.matmul(h, q[:, t].reshape(B * G, N, 1)).reshape(B, H, P)
    return [y.reshape(s["X"].shape), h.reshape(B, H, P, N)]


def _exact_act(v, act):
    if act in ("relu", "relu2"):
        return torch.where(v > 0, v if act == "relu" else v.square(), 0.0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "sigmoid":
        return torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def _exact_product(s, c):
    y = torch.matmul(s["a"].double(), s["w"].double().t().contiguous())
    if s["bias"] is not None:
        y += s["bias"].double()
    y = _exact_act(y, c["act"])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rms(v, w):
    return v * torch.rsqrt(v.square().sum(-1) / v.shape[-1] + EPS)[:, None] * w.double()


def _exact_block_norm(s, c):
    r = _exact_rms(s["x"].double(), s["post"])
    if s["gate"] is not None:
        r *= _exact_act(s["gate"].double(), c["act"])
    if s["residual"] is not None:
        r += s["residual"].double() * s["res_scale"]
    y = _exact_rms(r, s["weight"])
    if not c["codes"]:
        return [y, r]
    step = y.abs().max(-1).values / 127
    step[step == 0] = 1
    v = y / step[:, None]
    return [torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)) * step[:, None], step, r]
