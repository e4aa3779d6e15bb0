"""Refusals of the gated delta rule, the product with an epilogue and the block norm (no GPU
needed): every call here fails validation, is empty, or is host-only."""
import ctypes

import pytest
import torch

L = pytest.importorskip("mamba_ssd_chunked_amd._lib")

A16, MIS, ODD, BIG = 0x10000, 0x10004, 0x10001, 1 << 62
NAN, INF = float("nan"), float("inf")


def shape(**kw):
    base = dict(batch=2, seqlen=64, nheads=4, headdim=16, dstate=16, ngroups=1, chunk=64, dtype="fp16")
    base.update(kw)
    return L.make_shape(**base)


def fwd(sh=None, flags=0, scale=1.0, eps=1e-6, init=None, fin=None, ws=None, wsb=0, **p):
    sh = shape(batch=0) if sh is None else sh
    v = dict(X=A16, dt=A16, A=A16, B=A16, C=A16, beta=A16, ld=4, Y=A16)
    v.update(p)
    return L.LIB.ssd_delta_forward(ctypes.byref(sh), flags, v["X"], v["dt"], v["A"], v["B"], v["C"], v["beta"], v["ld"],
                                   scale, eps, v["Y"], init, fin, ws, wsb, None)


def step(sh=None, flags=0, scale=1.0, eps=1e-6, **p):
    sh = shape(batch=0, seqlen=1) if sh is None else sh
    v = dict(X=A16, dt=A16, A=A16, B=A16, C=A16, beta=A16, ld=4, Y=A16, state=A16)
    v.update(p)
    return L.LIB.ssd_delta_step(ctypes.byref(sh), flags, v["X"], v["dt"], v["A"], v["B"], v["C"], v["beta"], v["ld"],
                                scale, eps, v["state"], v["Y"], None)


def test_delta_refusals():
    for call in (fwd, step):
        assert call() == L.SSD_OK
        assert call(flags=3) == L.SSD_OK
        assert call(flags=4) == L.SSD_E_UNSUPPORTED and call(flags=-1) == L.SSD_E_UNSUPPORTED
        for k in ("X", "dt", "A", "B", "C", "beta", "Y"):
            assert call(**{k: None}) == L.SSD_E_NULL, k
            assert call(**{k: ODD}) == L.SSD_E_ALIGN, k
        for k in ("X", "dt", "A", "B", "C", "Y"):
            assert call(**{k: MIS}) == L.SSD_E_ALIGN, k
        assert call(beta=MIS + 2) == L.SSD_OK  # a slice needs its element's alignment only
        assert call(ld=3) == L.SSD_E_SHAPE and call(ld=1 << 28) == L.SSD_E_SHAPE
        for bad in (NAN, INF, -INF):
            assert call(scale=bad) == L.SSD_E_SHAPE and call(eps=bad) == L.SSD_E_SHAPE
        assert call(eps=-1e-6) == L.SSD_E_SHAPE and call(eps=0.0) == L.SSD_OK
    one = dict(batch=0, seqlen=1)
    for call in (fwd, step):
        for kw in (dict(headdim=8), dict(headdim=256), dict(dstate=256), dict(dstate=8), dict(dtype=7), dict(chunk=32)):
            assert call(sh=shape(**one, **kw)) == L.SSD_E_UNSUPPORTED, kw
        for kw in (dict(nheads=5, ngroups=2), dict(nheads=0), dict(batch=-1), dict(batch=65536)):
            assert call(sh=shape(**{**one, **kw})) == L.SSD_E_SHAPE, kw
        assert call(sh=shape(**one, headdim=128)) == L.SSD_OK
        assert call(sh=shape(batch=65535, seqlen=1, nheads=129), ld=129) == L.SSD_E_SHAPE  # over 2^23
    assert step(sh=shape(seqlen=2)) == L.SSD_E_SHAPE and step(sh=shape(seqlen=0)) == L.SSD_E_SHAPE
    assert step(state=None) == L.SSD_E_NULL and step(state=MIS) == L.SSD_E_ALIGN
    assert fwd(init=MIS) == L.SSD_E_ALIGN and fwd(fin=MIS) == L.SSD_E_ALIGN and fwd(ws=MIS) == L.SSD_E_ALIGN
    # no positions and no state wanted: nothing is enqueued, and nothing but A is looked at
    assert fwd(sh=shape(seqlen=0), X=None, dt=None, B=None, C=None, beta=None, Y=None, ld=0) == L.SSD_OK
    assert fwd(sh=shape(seqlen=0), A=None) == L.SSD_E_NULL
    # a workspace that is missing or too small
    sh = shape(seqlen=300)
    need = L.ssd_delta_workspace_bytes(sh)
    assert need > 0
    assert fwd(sh=sh) == L.SSD_E_WORKSPACE
    assert fwd(sh=sh, ws=A16, wsb=need - 1) == L.SSD_E_WORKSPACE
    assert fwd(sh=sh, ws=None, wsb=need) == L.SSD_E_NULL
    assert L.LIB.ssd_delta_forward(None, 0, *([A16] * 6), 4, 1.0, 0.0, A16, None, None, None, 0, None) == L.SSD_E_NULL


def test_delta_workspace_bytes():
    def ws(**kw):
        return L.ssd_delta_workspace_bytes(shape(**kw))

    assert ws(seqlen=1) == 0 and ws(seqlen=0) == 0 and ws(batch=0) == 0 and ws(headdim=8) == 0
    assert ws(seqlen=65) == ws(seqlen=128) == 2 * ws(seqlen=64) > 0
    assert ws(seqlen=65, chunk=256) == ws(seqlen=65)  # the shape's chunk has no influence
    assert ws(seqlen=640, headdim=128) == ws(seqlen=640)
    # fp16 keeps what its weights' rounding leaves, 3 KB a chunk and head
    assert ws(seqlen=640, dtype="fp32") > ws(seqlen=640, dtype="fp16") > ws(seqlen=640, dtype="bf16")
    assert L.LIB.ssd_delta_workspace_bytes(None) == 0


def mm(m=0, n=16, k=64, dtype=1, a=A16, ld=None, w=A16, bias=None, act=0, res=None, od=1, out=A16, ws=None, wsb=0):
    return L.LIB.ssd_matmul(m, n, k, dtype, a, k if ld is None else ld, w, bias, act, res, od, out, ws, wsb, None)


def test_matmul_refusals():
    assert mm() == L.SSD_OK and mm(bias=MIS, res=A16) == L.SSD_OK
    assert mm(m=-1) == L.SSD_E_SHAPE and mm(m=1 << 26) == L.SSD_E_SHAPE
    assert mm(n=0) == L.SSD_E_SHAPE and mm(n=1 << 26) == L.SSD_E_SHAPE and mm(k=0) == L.SSD_E_SHAPE
    assert mm(m=1 << 20, n=1 << 20) == L.SSD_E_SHAPE
    assert mm(k=1 << 22) == L.SSD_E_SHAPE and mm(ld=63) == L.SSD_E_SHAPE and mm(ld=1 << 22) == L.SSD_E_SHAPE
    assert mm(ld=(1 << 22) - 1) == L.SSD_OK and mm(k=1) == L.SSD_OK
    for dt in (-1, 3):
        assert mm(dtype=dt, od=0) == L.SSD_E_UNSUPPORTED and mm(od=dt) == L.SSD_E_UNSUPPORTED
    assert mm(dtype=1, od=2) == L.SSD_E_UNSUPPORTED and mm(dtype=0, od=1) == L.SSD_E_UNSUPPORTED
    for dt in (0, 1, 2):
        assert mm(dtype=dt, od=dt) == L.SSD_OK and mm(dtype=dt, od=0) == L.SSD_OK
    assert mm(act=-1) == L.SSD_E_UNSUPPORTED and mm(act=7) == L.SSD_E_UNSUPPORTED
    for act in range(7):
        assert mm(act=act) == L.SSD_OK
    for p in ("a", "w", "out"):
        assert mm(**{p: None}) == L.SSD_E_NULL and mm(**{p: ODD}) == L.SSD_E_ALIGN, p
    for p in ("w", "out", "res", "ws"):
        assert mm(**{p: MIS}) == L.SSD_E_ALIGN, p
    assert mm(a=MIS + 2) == L.SSD_OK and mm(a=A16 + 2, dtype=0, od=0) == L.SSD_E_ALIGN
    assert mm(bias=A16 + 2) == L.SSD_E_ALIGN
    # a workspace is optional, but not too small where the rows need one
    need = L.ssd_matmul_workspace_bytes(100, 16, 65, torch.float16)
    assert need == (100 + 16) * 128 * 2
    assert mm(m=100, k=65, ws=A16, wsb=need - 1) == L.SSD_E_WORKSPACE
    assert L.ssd_matmul_workspace_bytes(100, 16, 64, torch.float16) == 100 * 64 * 2  # w's rows are aligned
    assert L.ssd_matmul_workspace_bytes(3, 16, 65, torch.float16) == 0
    assert L.ssd_matmul_workspace_bytes(100, 16, 65, torch.float32) == 0
    assert L.LIB.ssd_matmul_workspace_bytes(100, 0, 65, 1) == 0 and L.LIB.ssd_matmul_workspace_bytes(100, 8, 65, 9) == 0


def bn(rows=0, cols=64, dtype=1, x=A16, ld=64, post=A16, gate=None, ldg=64, per=1, act=0, res=None, rs=1.0, rt=1,
       res_out=A16, w=A16, eps=1e-5, out=A16, q=None, s=None):
    return L.LIB.ssd_block_norm(rows, cols, dtype, x, ld, post, gate, ldg, per, act, res, rs, rt, res_out, w, eps, out, q,
                                s, None)


def test_block_norm_refusals():
    assert bn() == L.SSD_OK and bn(gate=A16, res=A16) == L.SSD_OK
    assert bn(out=None, w=None) == L.SSD_OK and bn(res_out=None) == L.SSD_OK
    assert bn(q=A16, s=A16, out=None) == L.SSD_OK
    assert bn(out=None, res_out=None) == L.SSD_E_NULL
    assert bn(w=None) == L.SSD_E_NULL and bn(out=None, q=A16, s=A16, w=None) == L.SSD_E_NULL
    assert bn(q=A16) == L.SSD_E_NULL and bn(s=A16) == L.SSD_E_NULL
    assert bn(x=None) == L.SSD_E_NULL and bn(post=None) == L.SSD_E_NULL
    assert bn(dtype=3) == L.SSD_E_UNSUPPORTED and bn(rt=2) == L.SSD_E_UNSUPPORTED and bn(rt=0) == L.SSD_OK
    assert bn(rt=2, res_out=None) == L.SSD_OK  # not looked at without a residual
    assert bn(rows=-1) == L.SSD_E_SHAPE and bn(rows=1 << 31) == L.SSD_E_SHAPE
    for cols in (0, -8, 16385):
        assert bn(cols=cols, ld=20000) == L.SSD_E_SHAPE
    assert bn(ld=63) == L.SSD_E_SHAPE and bn(rows=1 << 20, ld=BIG) == L.SSD_E_SHAPE
    for bad in (NAN, INF):
        assert bn(eps=bad) == L.SSD_E_SHAPE and bn(rs=bad) == L.SSD_E_SHAPE
    assert bn(eps=-1.0) == L.SSD_E_SHAPE
    for act in (1, 2, 5, 6, 7, -1):
        assert bn(gate=A16, act=act) == L.SSD_E_UNSUPPORTED and bn(act=act) == L.SSD_OK
    for act in (0, 3, 4):
        assert bn(gate=A16, act=act) == L.SSD_OK
    assert bn(gate=A16, per=0) == L.SSD_E_SHAPE and bn(gate=A16, per=-1) == L.SSD_E_SHAPE
    assert bn(gate=A16, per=BIG) == L.SSD_OK and bn(gate=A16, ldg=63) == L.SSD_E_SHAPE
    assert bn(gate=A16, rows=1 << 20, ldg=BIG) == L.SSD_E_SHAPE
    assert bn(x=ODD) == L.SSD_E_ALIGN and bn(gate=ODD) == L.SSD_E_ALIGN
    assert bn(x=MIS) == L.SSD_OK and bn(gate=MIS) == L.SSD_OK
    for k in ("post", "w", "out", "res", "res_out"):
        assert bn(**{k: MIS}) == L.SSD_E_ALIGN, k
    assert bn(q=MIS, s=A16) == L.SSD_E_ALIGN and bn(q=A16, s=A16 + 2) == L.SSD_E_ALIGN


def test_conv_takes_the_delta_rules_heads():
    """Heads of 128 channels, which the SSD itself refuses, come from the same convolution."""
    cd = 4 * 128 + 2 * 16
    sh = shape(seqlen=0, headdim=128)
    cv = ctypes.byref(L.SsdConv(A16, A16, A16, 4))
    assert L.LIB.ssd_conv_forward(ctypes.byref(sh), cv, A16, cd, A16, 4, None, None, None, A16, A16, A16, A16,
                                  None) == L.SSD_OK
    one = shape(batch=0, seqlen=1, headdim=128)
    assert L.LIB.ssd_conv_decode_step(ctypes.byref(one), 0, cv, A16, cd, A16, 4, A16, A16, None, A16, A16, A16, A16,
                                      None) == L.SSD_E_UNSUPPORTED


def test_binding_refuses_what_the_library_cannot_see():
    h = torch.float16
    with pytest.raises(ValueError, match="no columns"):
        L.ssd_matmul(torch.empty(4, 0, dtype=h), torch.empty(16, 0, dtype=h), None, torch.empty(4, 16, dtype=h))
    with pytest.raises(ValueError, match="last dimension"):
        L.ssd_matmul(torch.empty(4, 8, dtype=h), torch.empty(16, 9, dtype=h), None, torch.empty(4, 16, dtype=h))
    with pytest.raises(ValueError, match="no channels"):
        L.ssd_block_norm(torch.empty(4, 0), torch.ones(0), None, None, torch.ones(0), 1e-5, torch.empty(4, 0))
    # empty problems pass
    L.ssd_matmul(torch.empty(0, 8, dtype=h), torch.empty(16, 8, dtype=h), None, torch.empty(0, 16, dtype=h))
    L.ssd_block_norm(torch.empty(0, 8), torch.ones(8), None, None, torch.ones(8), 1e-5, torch.empty(0, 8))
    e = torch.empty
    sh = shape(batch=0)
    assert L.ssd_delta_forward(sh, e(0), e(0), e(4), e(0), e(0), e(0, 4), e(0)) is None
    L.ssd_delta_step(shape(batch=0, seqlen=1), e(0), e(0), e(4), e(0), e(0), e(0, 4), e(0), e(0))
    # rows of a's slices that lie aligned need no workspace; others say how much
    wide = torch.zeros(100, 200, dtype=h)
    w, out = torch.zeros(16, 64, dtype=h), torch.zeros(100, 16, dtype=h)
    assert L.ssd_matmul_workspace(wide[:, 8:72], w, out) is None
    assert L.ssd_matmul_workspace(wide[:, 3:67], w, out).numel() == 100 * 64 * 2
    assert L.ssd_matmul_workspace(wide[:3, 3:67], w, out[:3]) is None
