"""Refusals and host calls of the layer entry points (no GPU needed): every call
here fails validation, is empty, or is host-only, so nothing is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import layer_oracle as LO

L = pytest.importorskip("mamba_ssd_chunked_amd._lib")

A16 = 0x10000
MIS = 0x10004
ODD = 0x10001
BIG = 1 << 62


def shape(**kw):
    base = dict(batch=2, seqlen=64, nheads=4, headdim=16, dstate=16, ngroups=1, chunk=64, dtype="fp16")
    base.update(kw)
    return L.make_shape(**base)


CD = 4 * 16 + 2 * 16


def conv_struct(weight=A16, bias=A16, dt_bias=A16, width=4):
    return ctypes.byref(L.SsdConv(weight, bias, dt_bias, width))


def conv_fwd(sh=None, cv=None, xbc=A16, ldx=CD, raw=A16, ldt=4, lengths=None, pos=None, ring=None, X=A16, B=A16,
             C=A16, dt=A16):
    sh = shape(seqlen=0) if sh is None else sh
    return L.LIB.ssd_conv_forward(ctypes.byref(sh), conv_struct() if cv is None else cv, xbc, ldx, raw, ldt,
                                  lengths, pos, ring, X, B, C, dt, None)


def test_conv_forward_refusals():
    # with no positions a valid call enqueues nothing: the base of every case
    assert conv_fwd() == L.SSD_OK
    assert L.LIB.ssd_conv_forward(None, conv_struct(), A16, CD, A16, 4, None, None, None, A16, A16, A16, A16,
                                  None) == L.SSD_E_NULL
    assert conv_fwd(sh=shape(seqlen=0, headdim=8)) == L.SSD_E_UNSUPPORTED
    assert conv_fwd(sh=shape(seqlen=0, dtype=9)) == L.SSD_E_UNSUPPORTED
    assert conv_fwd(cv=ctypes.POINTER(L.SsdConv)()) == L.SSD_E_NULL
    assert conv_fwd(cv=conv_struct(weight=None)) == L.SSD_E_NULL
    for w in (-1, 0, 1, 5):
        assert conv_fwd(cv=conv_struct(width=w)) == L.SSD_E_UNSUPPORTED
    for w in (2, 3, 4):
        assert conv_fwd(cv=conv_struct(bias=None, dt_bias=None, width=w)) == L.SSD_OK
    assert conv_fwd(cv=conv_struct(weight=MIS)) == L.SSD_E_ALIGN
    assert conv_fwd(cv=conv_struct(bias=MIS)) == L.SSD_E_ALIGN
    assert conv_fwd(cv=conv_struct(dt_bias=MIS)) == L.SSD_OK
    assert conv_fwd(cv=conv_struct(dt_bias=ODD)) == L.SSD_E_ALIGN
    for k in ("xbc", "raw", "X", "B", "C", "dt"):
        assert conv_fwd(**{k: None}) == L.SSD_E_NULL, k
        assert conv_fwd(**{k: ODD}) == L.SSD_E_ALIGN, k
    assert conv_fwd(xbc=MIS + 2, raw=MIS + 2) == L.SSD_OK  # slices need their element's alignment only
    assert conv_fwd(X=MIS) == L.SSD_E_ALIGN
    assert conv_fwd(ldx=CD - 1) == L.SSD_E_SHAPE
    assert conv_fwd(ldt=3) == L.SSD_E_SHAPE
    assert conv_fwd(sh=shape(), ldx=BIG) == L.SSD_E_SHAPE
    assert conv_fwd(sh=shape(), ldt=BIG) == L.SSD_E_SHAPE
    # a row's bytes are counted in 32 bits
    assert conv_fwd(ldx=1 << 28) == L.SSD_E_SHAPE and conv_fwd(ldt=1 << 28) == L.SSD_E_SHAPE
    assert conv_fwd(ldx=(1 << 28) - 1, ldt=(1 << 28) - 1) == L.SSD_OK
    assert conv_fwd(sh=shape(seqlen=0, batch=65535, nheads=4096), ldx=1 << 20, ldt=4096) == L.SSD_E_SHAPE
    assert conv_fwd(pos=A16) == L.SSD_E_NULL  # a position without the ring it speaks of
    assert conv_fwd(pos=A16, ring=A16) == L.SSD_OK
    assert conv_fwd(ring=MIS) == L.SSD_E_ALIGN
    assert conv_fwd(pos=A16 + 2, ring=A16) == L.SSD_E_ALIGN
    assert conv_fwd(lengths=A16 + 2) == L.SSD_E_ALIGN


def step(sh=None, path=0, cv=None, scales=None, **p):
    sh = shape(batch=0, seqlen=1) if sh is None else sh
    v = dict(xbc=A16, ldx=CD, raw=A16, ldt=4, A=A16, D=A16, ring=A16, pos=A16, state=A16, Y=A16)
    v.update(p)
    return L.LIB.ssd_conv_decode_step(ctypes.byref(sh), path, conv_struct() if cv is None else cv, v["xbc"], v["ldx"],
                                      v["raw"], v["ldt"], v["A"], v["D"], scales, v["ring"], v["pos"], v["state"],
                                      v["Y"], None)


def test_conv_decode_step_refusals():
    sc = ctypes.byref(L.SsdScales(*([A16] * 7)))
    assert step() == L.SSD_OK and step(path=1, scales=sc) == L.SSD_OK
    assert step(path=1) == L.SSD_E_NULL
    assert step(path=2) == L.SSD_E_UNSUPPORTED and step(path=-1) == L.SSD_E_UNSUPPORTED
    assert step(sh=shape(seqlen=2)) == L.SSD_E_SHAPE
    assert step(sh=shape(seqlen=0)) == L.SSD_E_SHAPE
    assert step(sh=shape(seqlen=1, batch=65535, nheads=512), ldx=1 << 20, ldt=512) == L.SSD_E_SHAPE
    # 2^24 workgroups of 256 threads are one more than a grid holds
    assert step(sh=shape(seqlen=1, batch=32768, nheads=512), ldx=1 << 20, ldt=512) == L.SSD_E_SHAPE
    for k in ("xbc", "raw", "A", "D", "ring", "pos", "state", "Y"):
        assert step(**{k: None}) == L.SSD_E_NULL, k
        assert step(**{k: ODD}) == L.SSD_E_ALIGN, k
    for k in ("A", "D", "ring", "state", "Y"):
        assert step(**{k: MIS}) == L.SSD_E_ALIGN, k
    assert step(cv=conv_struct(width=5)) == L.SSD_E_UNSUPPORTED
    assert step(ldx=CD - 1) == L.SSD_E_SHAPE


def norm(gated=False, rows=0, cols=64, dtype=1, x=A16, ld=64, res=None, rt=1, res_out=None, w=A16, eps=1e-5, out=A16,
         q=None, s=None, groups=1):
    if gated:
        return L.LIB.ssd_gated_norm(rows, cols, groups, dtype, x, res, ld, w, eps, out, q, s, None)
    return L.LIB.ssd_add_norm(rows, cols, dtype, x, ld, res, rt, res_out, w, eps, out, q, s, None)


def test_norm_refusals():
    for gated in (False, True):
        kw = {"gated": gated, **({"res": A16} if gated else {})}
        assert norm(**kw) == L.SSD_OK
        assert norm(**kw, q=A16, s=A16, out=None) == L.SSD_OK
        assert norm(**kw, out=None) == L.SSD_E_NULL
        assert norm(**kw, q=A16) == L.SSD_E_NULL
        assert norm(**kw, s=A16) == L.SSD_E_NULL
        assert norm(**kw, x=None) == L.SSD_E_NULL
        assert norm(**kw, w=None) == L.SSD_E_NULL
        assert norm(**kw, dtype=3) == L.SSD_E_UNSUPPORTED and norm(**kw, dtype=-1) == L.SSD_E_UNSUPPORTED
        assert norm(**kw, rows=-1) == L.SSD_E_SHAPE and norm(**kw, rows=1 << 31) == L.SSD_E_SHAPE
        for cols in (0, -8, 16385):
            assert norm(**kw, cols=cols, ld=20000) == L.SSD_E_SHAPE
        assert norm(**kw, ld=63) == L.SSD_E_SHAPE
        assert norm(**kw, rows=1 << 20, ld=BIG) == L.SSD_E_SHAPE
        for eps in (-1e-6, float("nan"), float("inf")):
            assert norm(**kw, eps=eps) == L.SSD_E_SHAPE
        assert norm(**kw, x=ODD) == L.SSD_E_ALIGN
        assert norm(**kw, w=MIS) == L.SSD_E_ALIGN and norm(**kw, out=MIS) == L.SSD_E_ALIGN
        assert norm(**kw, q=MIS, s=A16) == L.SSD_E_ALIGN and norm(**kw, q=A16, s=A16 + 2) == L.SSD_E_ALIGN
    assert norm(x=MIS) == L.SSD_OK  # a slice
    assert norm(gated=True, res=A16, x=MIS) == L.SSD_E_ALIGN and norm(gated=True, res=MIS) == L.SSD_OK
    assert norm(gated=True, res=None) == L.SSD_E_NULL
    assert norm(gated=True, res=A16, groups=0) == L.SSD_E_SHAPE
    assert norm(gated=True, res=A16, groups=5) == L.SSD_E_SHAPE
    assert norm(res=A16, rt=0) == L.SSD_OK and norm(res_out=A16, rt=0) == L.SSD_OK
    assert norm(res=A16, rt=2) == L.SSD_E_UNSUPPORTED and norm(res_out=A16, rt=7) == L.SSD_E_UNSUPPORTED
    assert norm(res=MIS) == L.SSD_E_ALIGN and norm(res_out=MIS) == L.SSD_E_ALIGN
    assert norm(rt=7) == L.SSD_OK  # not looked at without a residual


def mm(m=0, n=16, k=64, a=A16, sa=A16, w=A16, sw=A16, bias=None, dtype=1, out=A16, ws=None, wsb=0):
    return L.LIB.ssd_matmul_i8(m, n, k, a, sa, w, sw, bias, dtype, out, ws, wsb, None)


def test_matmul_refusals():
    assert mm() == L.SSD_OK and mm(bias=MIS) == L.SSD_OK
    assert mm(m=-1) == L.SSD_E_SHAPE and mm(m=1 << 26) == L.SSD_E_SHAPE
    assert mm(n=0) == L.SSD_E_SHAPE and mm(n=1 << 26) == L.SSD_E_SHAPE
    assert mm(m=1 << 20, n=1 << 20) == L.SSD_E_SHAPE
    assert mm(k=0) == L.SSD_E_SHAPE and mm(k=131072) == L.SSD_E_SHAPE and mm(k=131056) == L.SSD_OK
    for k in (1, 8, 24, 100):
        assert mm(k=k) == L.SSD_E_UNSUPPORTED
    assert mm(dtype=3) == L.SSD_E_UNSUPPORTED and mm(dtype=-1) == L.SSD_E_UNSUPPORTED
    for p in ("a", "sa", "w", "sw", "out"):
        assert mm(**{p: None}) == L.SSD_E_NULL, p
        assert mm(**{p: ODD}) == L.SSD_E_ALIGN, p
    assert mm(a=MIS) == L.SSD_E_ALIGN and mm(out=MIS) == L.SSD_E_ALIGN and mm(ws=MIS) == L.SSD_E_ALIGN
    assert mm(bias=A16 + 2) == L.SSD_E_ALIGN
    assert L.ssd_matmul_i8_workspace_bytes(0, 16, 64) == 0
    assert L.ssd_matmul_i8_workspace_bytes(8, 16, 100) == 0
    # where a workspace is needed, a smaller one is refused
    for m, n, k in ((1, 64, 8192), (64, 2560, 5120), (333, 512, 4096), (16384, 2560, 5120)):
        need = L.ssd_matmul_i8_workspace_bytes(m, n, k)
        if need:
            assert mm(m=m, n=n, k=k) == L.SSD_E_WORKSPACE
            assert mm(m=m, n=n, k=k, ws=A16, wsb=need - 1) == L.SSD_E_WORKSPACE


def test_pack_weight():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((5, 37)).astype(np.float32) * np.array([[1], [1e-3], [0], [1e30], [7]], np.float32)
    q, s = L.ssd_pack_weight_i8(w)
    codes, steps = LO.row_codes(w.astype(np.float64))
    assert np.array_equal(s, steps.astype(np.float32))
    # the codes go by the float32 step that is handed out
    assert np.array_equal(q, np.clip(LO.rhaz(w.astype(np.float64) / s[:, None].astype(np.float64)), -127, 127))
    assert np.abs(q - codes).max() <= 1
    for bad in (np.nan, np.inf, -np.inf):
        v = w.copy()
        v[3, 5] = bad
        with pytest.raises(L.SSDError) as e:
            L.ssd_pack_weight_i8(v)
        assert e.value.status == L.SSD_E_VALUE
    with pytest.raises(ValueError):
        L.ssd_pack_weight_i8(w[0])
    assert L.LIB.ssd_pack_weight_i8(0, 4, w.ctypes.data, q.ctypes.data, s.ctypes.data) == L.SSD_E_SHAPE
    assert L.LIB.ssd_pack_weight_i8(4, 4, None, q.ctypes.data, s.ctypes.data) == L.SSD_E_NULL
    assert L.LIB.ssd_pack_weight_i8(BIG, BIG, w.ctypes.data, q.ctypes.data, s.ctypes.data) == L.SSD_E_SHAPE


def test_binding_refuses_what_the_library_cannot_see():
    """Host tensors, wrong sizes and types, rows at unequal distances or that overlap.
    (-1 stands for a host tensor's device, so that the other checks are met here.)"""
    x = torch.zeros(4, 64, dtype=torch.float16)
    w = torch.ones(64)
    with pytest.raises(ValueError):
        L.ssd_add_norm(x, None, None, w, 1e-5, torch.zeros_like(x))  # not on a GPU
    f = torch.float32
    assert L._rows(w.view(1, 64), "x", 64, f, -1) == (w.data_ptr(), 64)
    wide = torch.zeros(4, 6, 100)
    assert L._rows(wide[:, :, 3:67], "x", 64, f, -1) == (wide.data_ptr() + 12, 100)
    assert L._rows(wide[:, 0, 3:67], "x", 64, f, -1) == (wide.data_ptr() + 12, 600)
    assert L._rows(wide[2:3, 1:2, 3:67], "x", 64, f, -1) == (wide[2, 1, 3:].data_ptr(), 64)
    for t, n, dt, dev, words in ((torch.zeros(4, 64).t(), 4, f, -1, "consecutive"),
                                 (wide[:, :5, 3:67], 64, f, -1, "equal distances"),
                                 (w.expand(4, 64), 64, f, -1, "overlap"),
                                 (wide, 64, f, -1, "rows of 64"), (wide, 100, torch.float16, -1, "float16"),
                                 (wide, 100, f, 0, "current GPU")):
        with pytest.raises(ValueError, match=words):
            L._rows(t, "x", n, dt, dev)
    assert L._dense(None, "w", 64, f, -1) is None
    assert L._dense(w, "w", 64, f, -1) == w.data_ptr()
    for t, n, dt, dev in ((w, 63, f, -1), (w, 64, torch.int8, -1), (w, 64, f, 0), (wide.transpose(0, 1), 2400, f, -1)):
        with pytest.raises(ValueError, match="contiguous"):
            L._dense(t, "w", n, dt, dev)
    other = type("S", (), {"device_index": 1, "cuda_stream": 7})()
    assert L._stream_on(5, 0) == 5 and L._stream_on(other, 1) == 7
    with pytest.raises(ValueError, match="GPU 1"):
        L._stream_on(other, 0)
    assert L._code(torch.bfloat16) == L.DTYPE_CODE[torch.bfloat16]
    for dt in (torch.float64, torch.int32):
        with pytest.raises(ValueError, match=str(dt)):
            L._code(dt)
    for bad in (torch.zeros(96, 4, dtype=torch.float16), torch.zeros(96, 4)):
        with pytest.raises(ValueError, match="float32 tensors on one GPU"):
            L.ConvParams(bad)


def test_step_refuses_scales_of_another_shape():
    """The kernel reads G and H*P steps: a pack of fewer would be read behind its end."""
    def pack(g, hp):
        return L.ScalePack({k: np.ones(g if k in ("s_B", "s_C", "inv_B", "inv_C") else hp, np.float32)
                            for k in L.ScalePack.ORDER}, "cpu")

    sh = shape(batch=0, seqlen=1, nheads=4, headdim=16, ngroups=2)
    assert L._pack(None, sh, -1) is None
    L._pack(pack(2, 64), sh, -1)
    for g, hp, name in ((1, 64, "s_B"), (4, 64, "s_B"), (2, 48, "s_X"), (2, 16, "s_X")):
        with pytest.raises(ValueError, match=name):
            L._pack(pack(g, hp), sh, -1)
    with pytest.raises(ValueError, match="current GPU"):
        L._pack(pack(2, 64), sh, 0)


def test_rows_of_no_columns_are_refused():
    """Sums over nothing are refused, as in the C calls, instead of leaving the outputs
    as they were; no rows are a valid empty problem."""
    e = torch.empty
    w, s, out = torch.ones(0), torch.zeros(4), torch.zeros(4, 16)
    with pytest.raises(ValueError, match="no columns"):
        L.ssd_matmul_i8(e(4, 0, dtype=torch.int8), s, e(16, 0, dtype=torch.int8), torch.zeros(16), None, out)
    with pytest.raises(ValueError, match="no channels"):
        L.ssd_add_norm(e(4, 0), None, None, w, 1e-5, None, e(4, 0, dtype=torch.int8), s)
    with pytest.raises(ValueError, match="no channels"):
        L.ssd_gated_norm(e(4, 0), e(4, 0), 1, w, 1e-5, None, e(4, 0, dtype=torch.int8), s)
    L.ssd_matmul_i8(e(0, 64, dtype=torch.int8), e(0), e(16, 64, dtype=torch.int8), torch.zeros(16), None, e(0, 16))
    L.ssd_add_norm(e(0, 64), None, None, torch.ones(64), 1e-5, e(0, 64))
    L.ssd_gated_norm(e(0, 64), e(0, 64), 1, torch.ones(64), 1e-5, e(0, 64))


def test_alignment_error_names_both_alignments():
    """A float array at an odd address and a strided row at half an element are refused
    with the same status as a dense buffer at 4 bytes: its text says so."""
    assert mm(sa=ODD) == norm(x=ODD) == norm(out=MIS) == L.SSD_E_ALIGN
    assert "16 bytes" in L.status_string(L.SSD_E_ALIGN) and "element" in L.status_string(L.SSD_E_ALIGN)
