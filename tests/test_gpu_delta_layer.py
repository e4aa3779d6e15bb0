"""A layer around the gated delta rule from its prompts on token by token."""
import numpy as np
import pytest

from tests import test_gpu_delta as D
from tests import test_gpu_operators as T

pytestmark = pytest.mark.gpu

_np = T._np


def test_delta_layer_token_by_token(gpu_lib):
    """A layer's prompts, and then its single tokens: the convolution's ring and the state that
    the prompts leave, each token through every call of the layer, against the whole sequences."""
    import torch
    L = gpu_lib
    for dims in ((3, 40, 4, 64, 128, 1, "bf16"), (2, 21, 6, 32, 64, 2, "fp16"), (2, 12, 3, 128, 32, 1, "fp32")):
        B, Ln, H_, P, N, G, dtype = dims
        print("layer", dims, flush=True)
        more, w = 9, T.layer(torch, 3, dtype, 96, H_, P, N, G)
        td, d, cd = getattr(torch, D.DT[dtype]), w["d"], w["cd"]
        g = torch.Generator(device="cuda").manual_seed(6)
        full = torch.randn(B, Ln + more, 96, generator=g, device="cuda").to(td)
        ends = [Ln, 1, Ln // 2][:B]
        prompt = torch.zeros(B, Ln, 96, dtype=td, device="cuda")
        for b, n in enumerate(ends):
            prompt[b, :n] = full[b, :n]
        o = T.layer_prompts(L, torch, w, prompt, dims, torch.tensor(ends, dtype=torch.int32, device="cuda"))
        pos = torch.tensor(ends, dtype=torch.int32, device="cuda")
        got = {"r2": [], "x2": []}
        sh = L.make_shape(B, 1, H_, P, N, G, 64, dtype)
        conv = L.ConvParams(w["conv"], w["conv_b"], w["dt_b"])
        e = lambda *s: torch.empty(*s, dtype=td, device="cuda")  # noqa: E731
        for i in range(more):
            res = torch.stack([full[b, n + i] for b, n in enumerate(ends)])
            x, r, p, m, r2, x2 = e(B, 96), e(B, 96), e(B, w["rows"]), e(B, 96), e(B, 96), e(B, 96)
            X, K, Q, dt, Y, gn = e(B, 1, H_, P), e(B, 1, G, N), e(B, 1, G, N), e(B, 1, H_), e(B, 1, H_, P), e(B, d)
            L.ssd_add_norm(res, None, r, w["norm"], 1e-5, x)
            L.ssd_matmul(x, w["in"], w["bias"], p)
            row = p.view(B, 1, -1)
            L.ssd_conv_forward(sh, conv, row[..., d:d + cd], row[..., d + cd:d + cd + H_], X, K, Q, dt, o["ring"], pos)
            L.ssd_delta_step(sh, X, dt, w["A"], K, Q, row[..., d + cd + H_:], o["S"], Y, scale=N ** -0.5, logit=True)
            L.ssd_gated_norm(Y.view(B, d), p[..., :d], 1, w["gate"], 1e-5, gn)
            L.ssd_matmul(gn, w["out"], None, m)
            L.ssd_block_norm(m, w["post"], r, r2, w["next"], 1e-5, x2)
            pos += 1
            got["r2"].append(r2)
            got["x2"].append(x2)
        torch.cuda.synchronize()
        for b, n in enumerate(ends):
            whole = (1, n + more) + dims[2:]
            s, r2, x2 = T.layer_reference(w, full[b:b + 1, :n + more], whole, [n + more])
            have = {"state": _np(o["S"][b]), "r2": _np(torch.stack([t[b] for t in got["r2"]])),
                    "x2": _np(torch.stack([t[b] for t in got["x2"]]))}
            for what, ref in (("state", s[0]), ("r2", r2[0, n:]), ("x2", x2[0, n:])):
                rel = np.linalg.norm(have[what] - ref) / np.linalg.norm(ref)
                assert rel <= T.LAYER[dtype], f"{what} of sequence {b}: {rel:.3g}"
