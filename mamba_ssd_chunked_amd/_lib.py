"""Python binding of libssd.so (the SSD C ABI declared in include/ssd.h).

Argument marshalling only: every step of the SSD forward runs in the HIP
kernels behind the C ABI. torch tensors supply device memory and the current
stream. The functions keep the C names and argument order; device buffers are
passed as torch tensors (or None for optional ones), the shape as an
``SsdShape`` and the INT8 scales as a ``ScalePack``.

Importing this module loads libssd.so and raises if it is missing: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssd.so")

SSD_OK = 0
SSD_E_NULL = 1
SSD_E_SHAPE = 2
SSD_E_UNSUPPORTED = 3
SSD_E_ALIGN = 4
SSD_E_WORKSPACE = 5
SSD_E_HIP = 6
SSD_E_INTERNAL = 7
SSD_E_VALUE = 8
SSD_E_TOO_LARGE = 9
NOALLOC_SCRATCH_BYTES = 128 << 20

SSD_DTYPE_F32 = 0
SSD_DTYPE_F16 = 1
SSD_DTYPE_BF16 = 2
SSD_PATH_FLOAT = 0
SSD_PATH_INT8 = 1
SSD_PATH_ABL_QX = 2
SSD_PATH_ABL_RECON = 3
SSD_DELTA_UNIT = 1
SSD_DELTA_LOGIT = 2
SSD_ACT_NONE = 0
SSD_ACT_RELU = 1
SSD_ACT_RELU2 = 2
SSD_ACT_SILU = 3
SSD_ACT_SIGMOID = 4
SSD_ACT_GELU = 5
SSD_ACT_GELU_TANH = 6
SSD_SCHED_AUTO = 0
SSD_SCHED_HEAD = 1
SSD_SCHED_CHUNK = 2

DTYPE_CODE = {torch.float32: SSD_DTYPE_F32, torch.float16: SSD_DTYPE_F16,
              torch.bfloat16: SSD_DTYPE_BF16}
DTYPE_NAME = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


class SsdShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("schedule", ctypes.c_int32)]

    @property
    def nchunks(self) -> int:
        return -(-self.seqlen // self.chunk)


class SsdScales(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("s_B", "s_C", "inv_B", "inv_C", "inv_X", "s_S", "M_req", "s_X", "s_Xq", "inv_Xq")]


class SsdTaps(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q_xs", "s32", "s8_local", "passed")]


class SsdConv(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("width", ctypes.c_int32)]


class SSDError(RuntimeError):
    def __init__(self, name: str, rc: int):
        super().__init__(f"{name} failed: {status_string(rc)} (status {rc})")
        self.status = rc


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build the HIP library first "
                           "(python -m mamba_ssd_chunked_amd.csrc.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    SP = ctypes.POINTER(SsdShape)
    CP = ctypes.POINTER(SsdConv)
    I64 = ctypes.c_int64
    sig = {
        "ssd_quantize_bc": [SP, P, P, ctypes.POINTER(SsdScales), P, P, P],
        "ssd_chunk_cumsum": [SP, P, P, P, P, P, P],
        "ssd_chunk_state": [SP, ctypes.c_int, P, P, P, ctypes.POINTER(SsdScales), P,
                            ctypes.POINTER(SsdTaps), P],
        "ssd_state_passing": [SP, ctypes.c_int, P, P, P, P, P, P],
        "ssd_chunk_bmm": [SP, ctypes.c_int, P, P, P, P],
        "ssd_chunk_scan": [SP, ctypes.c_int, P, P, P, P, P, P, P, P, ctypes.POINTER(SsdScales), P, P],
        "ssd_forward": [SP, ctypes.c_int, P, P, P, P, P, P, ctypes.POINTER(SsdScales), P, P, P, P,
                        ctypes.c_size_t, ctypes.POINTER(SsdTaps), P],
        "ssd_forward_noalloc": [SP, ctypes.c_int, P, P, P, P, P, P, ctypes.POINTER(SsdScales), P, P, P,
                                ctypes.POINTER(SsdTaps), P],
        "ssd_decode_step": [SP, ctypes.c_int, P, P, P, P, P, P, ctypes.POINTER(SsdScales), P, P,
                            P],
        "ssd_epilogue": [SP, P, P, ctypes.c_float, P, ctypes.c_float, P, P],
        "ssd_mean_correction": [SP, P, P, P, P],
        "ssd_calibrate_amax": [SP, P, P, P, P, P, P, P, ctypes.c_size_t, P],
        "ssd_scales_from_amax": [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, P, P],
        "ssd_conv_forward": [SP, CP, P, I64, P, I64, P, P, P, P, P, P, P, P],
        "ssd_conv_decode_step": [SP, ctypes.c_int, CP, P, I64, P, I64, P, P, ctypes.POINTER(SsdScales), P, P,
                                 P, P, P],
        "ssd_add_norm": [I64, I64, ctypes.c_int, P, I64, P, ctypes.c_int, P, P, ctypes.c_float, P, P, P, P],
        "ssd_gated_norm": [I64, I64, I64, ctypes.c_int, P, P, I64, P, ctypes.c_float, P, P, P, P],
        "ssd_matmul_i8": [I64, I64, I64, P, P, P, P, P, ctypes.c_int, P, P, ctypes.c_size_t, P],
        "ssd_pack_weight_i8": [I64, I64, P, P, P],
        "ssd_delta_forward": [SP, ctypes.c_int, P, P, P, P, P, P, I64, ctypes.c_float, ctypes.c_float, P, P, P, P,
                              ctypes.c_size_t, P],
        "ssd_matmul": [I64, I64, I64, ctypes.c_int, P, I64, P, P, ctypes.c_int, P, ctypes.c_int, P, P, ctypes.c_size_t,
                       P],
        "ssd_block_norm": [I64, I64, ctypes.c_int, P, I64, P, P, I64, I64, ctypes.c_int, P, ctypes.c_float, ctypes.c_int,
                           P, P, ctypes.c_float, P, P, P, P],
        "ssd_delta_step": [SP, ctypes.c_int, P, P, P, P, P, P, I64, ctypes.c_float, ctypes.c_float, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    for name in ("ssd_workspace_bytes",):
        f = getattr(lib, name)
        f.argtypes = [SP, ctypes.c_int]
        f.restype = ctypes.c_size_t
    lib.ssd_matmul_i8_workspace_bytes.argtypes = [I64, I64, I64]
    lib.ssd_matmul_i8_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_calibrate_workspace_bytes.argtypes = [SP]
    lib.ssd_calibrate_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_matmul_workspace_bytes.argtypes = [I64, I64, I64, ctypes.c_int]
    lib.ssd_matmul_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_delta_workspace_bytes.argtypes = [SP]
    lib.ssd_delta_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_status_string.restype = ctypes.c_char_p
    return lib


LIB = _load()

EXPORTED = ("ssd_quantize_bc", "ssd_chunk_cumsum", "ssd_chunk_state", "ssd_state_passing",
            "ssd_chunk_bmm", "ssd_chunk_scan", "ssd_forward", "ssd_forward_noalloc", "ssd_decode_step",
            "ssd_epilogue", "ssd_mean_correction",
            "ssd_workspace_bytes",
            "ssd_calibrate_amax", "ssd_calibrate_workspace_bytes", "ssd_scales_from_amax",
            "ssd_conv_forward", "ssd_conv_decode_step", "ssd_add_norm", "ssd_gated_norm", "ssd_matmul_i8",
            "ssd_matmul_i8_workspace_bytes", "ssd_pack_weight_i8",
            "ssd_delta_forward", "ssd_delta_workspace_bytes", "ssd_delta_step",
            "ssd_matmul", "ssd_matmul_workspace_bytes", "ssd_block_norm",
            "ssd_status_string")


def status_string(rc: int) -> str:
    return LIB.ssd_status_string(rc).decode()


def _check(name: str, rc: int) -> None:
    if rc != SSD_OK:
        raise SSDError(name, rc)


def _p(t):
    """Device address of a tensor; the C ABI takes dense row-major buffers only."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("SSD buffers must be contiguous (row-major, no strides)")
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if torch.cuda.is_available():
        return torch.cuda.current_stream().cuda_stream
    return None


def make_shape(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, dtype,
               schedule=0) -> SsdShape:
    code = dtype if isinstance(dtype, int) else DTYPE_CODE[DTYPE_NAME.get(dtype, dtype)]
    return SsdShape(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, code, schedule)


class ScalePack:
    """Device copy of the static scale pack, each array 256-byte aligned.

    ``arrays`` holds float32 numpy arrays s_B, s_C, inv_B, inv_C ([G]) and
    s_X, inv_X, s_S, M_req ([H, P] or [H*P]); optionally s_Xq, inv_Xq ([H, P],
    the step of X itself, read only by the "Q(X) only" ablation path).
    """

    ORDER = ("s_B", "s_C", "inv_B", "inv_C", "s_X", "inv_X", "s_S", "M_req")
    OPTIONAL = ("s_Xq", "inv_Xq")
    PER_GROUP = ("s_B", "s_C", "inv_B", "inv_C")

    def __init__(self, arrays: dict, device="cuda"):
        names = [k for k in self.ORDER if k in arrays] + [k for k in self.OPTIONAL if k in arrays]
        flat = [np.ascontiguousarray(arrays[k], dtype=np.float32).reshape(-1) for k in names]
        offs, cur = [], 0
        for a in flat:
            offs.append(cur)
            cur += -(-a.size // 64) * 64
        host = np.zeros(max(cur, 64), dtype=np.float32)
        for o, a in zip(offs, flat):
            host[o:o + a.size] = a
        self.host = {k: a for k, a in zip(names, flat)}
        self.tensor = torch.from_numpy(host).to(device)
        self.device_index = self.tensor.get_device()
        # (G, H*P) that all arrays agree on, or None
        sizes = [{a.size for k, a in self.host.items() if (k in self.PER_GROUP) == g} for g in (True, False)]
        self.fits = (sizes[0].pop(), sizes[1].pop()) if all(len(v) == 1 for v in sizes) else None
        base = self.tensor.data_ptr()
        ptr = {k: base + 4 * o for k, o in zip(names, offs)}
        self.struct = SsdScales(*[ptr.get(k) for k in ("s_B", "s_C", "inv_B", "inv_C", "inv_X",
                                                       "s_S", "M_req", "s_X", "s_Xq", "inv_Xq")])


def _scales(sc):
    if sc is None:
        return None
    if isinstance(sc, ScalePack):
        return ctypes.byref(sc.struct)
    return ctypes.byref(sc)


def _taps(taps):
    if taps is None:
        return None
    return ctypes.byref(SsdTaps(_p(taps.get("q_xs")), _p(taps.get("s32")),
                                _p(taps.get("s8_local")), _p(taps.get("passed"))))


# ---------------------------------------------------------------------------
# the C calls, same names and argument order
# ---------------------------------------------------------------------------

def ssd_quantize_bc(shape, B, C, scales, qB, qC, stream=None):
    _check("ssd_quantize_bc", LIB.ssd_quantize_bc(ctypes.byref(shape), _p(B), _p(C),
                                                  _scales(scales), _p(qB), _p(qC),
                                                  _stream(stream)))


def ssd_chunk_cumsum(shape, dt, A, dAcs, lut=None, qdecay=None, stream=None):
    _check("ssd_chunk_cumsum", LIB.ssd_chunk_cumsum(ctypes.byref(shape), _p(dt), _p(A),
                                                    _p(dAcs), _p(lut), _p(qdecay),
                                                    _stream(stream)))


def ssd_chunk_state(shape, path, X, lut, Bq, scales, states, taps=None, stream=None):
    _check("ssd_chunk_state", LIB.ssd_chunk_state(ctypes.byref(shape), path, _p(X), _p(lut),
                                                  _p(Bq), _scales(scales), _p(states),
                                                  _taps(taps), _stream(stream)))


def ssd_state_passing(shape, path, states, dAcs=None, qdecay=None, final_state=None,
                      stream=None, initial_state=None):
    _check("ssd_state_passing", LIB.ssd_state_passing(ctypes.byref(shape), path, _p(states),
                                                      _p(dAcs), _p(qdecay), _p(initial_state),
                                                      _p(final_state), _stream(stream)))


def ssd_chunk_bmm(shape, path, Cq, Bq, CB, stream=None):
    _check("ssd_chunk_bmm", LIB.ssd_chunk_bmm(ctypes.byref(shape), path, _p(Cq), _p(Bq), _p(CB),
                                              _stream(stream)))


def ssd_chunk_scan(shape, path, X, dt, dAcs, Cq, CB, states, D, scales, Y, stream=None,
                   initial_state=None):
    _check("ssd_chunk_scan", LIB.ssd_chunk_scan(ctypes.byref(shape), path, _p(X), _p(dt),
                                                _p(dAcs), _p(Cq), _p(CB), _p(states),
                                                _p(initial_state), _p(D), _scales(scales), _p(Y),
                                                _stream(stream)))


def ssd_workspace_bytes(shape, path) -> int:
    return int(LIB.ssd_workspace_bytes(ctypes.byref(shape), path))


def ssd_forward(shape, path, X, dt, A, B, C, D, scales, Y, final_state=None, workspace=None,
                taps=None, stream=None, initial_state=None):
    """Whole forward. ``workspace`` (a uint8 device tensor) is allocated here if None.
    ``initial_state`` continues a sequence from a previous call's final state."""
    need = ssd_workspace_bytes(shape, path)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ssd_forward", LIB.ssd_forward(ctypes.byref(shape), path, _p(X), _p(dt), _p(A), _p(B),
                                          _p(C), _p(D), _scales(scales), _p(Y),
                                          _p(initial_state), _p(final_state), _p(workspace), wsb,
                                          _taps(taps),
                                          _stream(stream)))
    return workspace


def ssd_forward_noalloc(shape, path, X, dt, A, B, C, D, scales, Y, final_state=None, taps=None,
                        stream=None, initial_state=None):
    """Whole forward on the library's fixed device workspace (allocates nothing;
    calls that may overlap on one device race)."""
    _check("ssd_forward_noalloc",
           LIB.ssd_forward_noalloc(ctypes.byref(shape), path, _p(X), _p(dt), _p(A), _p(B), _p(C), _p(D),
                                   _scales(scales), _p(Y), _p(initial_state), _p(final_state),
                                   _taps(taps), _stream(stream)))


def ssd_decode_step(shape, path, X, dt, A, B, C, D, scales, state, Y, stream=None):
    """One position: ``state`` [B,H,P,N] (int8 or fp32) is updated in place,
    Y [B,H,P] receives the output. ``shape.seqlen`` must be 1."""
    _check("ssd_decode_step", LIB.ssd_decode_step(ctypes.byref(shape), path, _p(X), _p(dt), _p(A),
                                                  _p(B), _p(C), _p(D), _scales(scales),
                                                  _p(state), _p(Y), _stream(stream)))


# "Key design 4": the mean correction's coefficient fixed by "Training strategy"
MEAN_CORRECTION_ALPHA = 0.15


def ssd_epilogue(shape, Y, corr, alpha, weight, eps, out, stream=None):
    """RMSNorm over the H*P channels of every position of Y, after adding
    alpha * corr (corr may be None)."""
    _check("ssd_epilogue", LIB.ssd_epilogue(ctypes.byref(shape), _p(Y), _p(corr), float(alpha),
                                            _p(weight), float(eps), _p(out), _stream(stream)))


def ssd_mean_correction(shape, Y_ref, Y_q, c, stream=None):
    """c = per-channel mean of Y_ref - Y_q over all positions."""
    _check("ssd_mean_correction", LIB.ssd_mean_correction(ctypes.byref(shape), _p(Y_ref), _p(Y_q),
                                                          _p(c), _stream(stream)))


def ssd_calibrate_workspace_bytes(shape) -> int:
    return int(LIB.ssd_calibrate_workspace_bytes(ctypes.byref(shape)))


def ssd_calibrate_amax(shape, X, dt, A, B, C, amax, workspace=None, stream=None):
    need = ssd_calibrate_workspace_bytes(shape)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("ssd_calibrate_amax", LIB.ssd_calibrate_amax(ctypes.byref(shape), _p(X), _p(dt), _p(A),
                                                        _p(B), _p(C), _p(amax), _p(workspace),
                                                        wsb, _stream(stream)))


def ssd_scales_from_amax(ngroups: int, nheads: int, headdim: int, amax: np.ndarray) -> dict:
    """Host call: the static scale pack from calibration maxima (numpy in, numpy out)."""
    G, HP = ngroups, nheads * headdim
    a = np.ascontiguousarray(amax, dtype=np.float32).reshape(-1)
    if a.size != 2 * G + 2 * HP:
        raise ValueError("amax must hold 2*G + 2*H*P values")
    pack = np.zeros(4 * G + 4 * HP, dtype=np.float32)
    _check("ssd_scales_from_amax", LIB.ssd_scales_from_amax(
        ngroups, nheads, headdim, a.ctypes.data, pack.ctypes.data))
    out, o = {}, 0
    for k, n in (("s_B", G), ("s_C", G), ("inv_B", G), ("inv_C", G),
                 ("s_X", HP), ("inv_X", HP), ("s_S", HP), ("M_req", HP)):
        out[k] = pack[o:o + n].copy()
        o += n
    return out


def calibrate(shape_of, seqs, A, device="cuda") -> ScalePack:
    """Static scales from calibration sequences, on the GPU.

    ``seqs``: iterable of dicts of device tensors x, dt, B, C (one batch each);
    ``shape_of(seq)`` returns the SsdShape of a sequence.
    """
    seqs = list(seqs)
    s0 = shape_of(seqs[0])
    G, H, P = s0.ngroups, s0.nheads, s0.headdim
    amax = torch.zeros(2 * G + 2 * H * P, dtype=torch.float32, device=device)
    for sq in seqs:
        ssd_calibrate_amax(shape_of(sq), sq["x"], sq["dt"], A, sq["B"], sq["C"], amax)
    host = amax.cpu().numpy()
    return ScalePack(ssd_scales_from_amax(G, H, P, host), device)


# ---------------------------------------------------------------------------
# the steps around the SSD in a layer
# ---------------------------------------------------------------------------

class ConvParams:
    """The causal convolution's parameters on a GPU: weight [Cd, width] (or
    [Cd, 1, width]), bias [Cd] and dt_bias [H] (either may be None), float32."""

    def __init__(self, weight, bias=None, dt_bias=None):
        self.weight = weight.reshape(weight.shape[0], -1)
        self.bias, self.dt_bias = bias, dt_bias
        self.channels, self.width = self.weight.shape
        self.heads = None if dt_bias is None else dt_bias.numel()
        if bias is not None and bias.numel() != self.channels:
            raise ValueError("bias must hold one value for each channel")
        for t in (self.weight, bias, dt_bias):
            if t is not None and (t.dtype is not torch.float32 or not t.is_cuda or t.device != weight.device):
                raise ValueError("convolution parameters are float32 tensors on one GPU")
        self.device_index = weight.get_device()
        self.struct = SsdConv(_p(self.weight), _p(bias), _p(dt_bias), self.width)


def _current_device() -> int:
    """The device that kernels are launched on. The checks below run once per call and
    tensor, in front of launches of a few microseconds: they use the cheap queries."""
    try:
        return torch._C._cuda_getDevice()
    except (RuntimeError, AttributeError) as e:
        raise ValueError(f"the buffers must be on a GPU: {e}") from None


def _stream_on(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, int):
        return stream
    if stream.device_index != dev:
        raise ValueError(f"the stream belongs to GPU {stream.device_index}, the current GPU is {dev}")
    return stream.cuda_stream


def _code(dtype):
    try:
        return DTYPE_CODE[dtype]
    except KeyError:
        raise ValueError(f"no such type here: {dtype}") from None


def _dense(t, name, numel, dtype, dev):
    """Address of a dense buffer of a given size and type on device ``dev`` (None passes:
    the C call decides)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} values on the current GPU, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _rows(t, name, n, dtype, dev):
    """Address and row distance of a tensor whose rows of n values lie at equal
    distances (a contiguous tensor, or a slice of the columns of one)."""
    sh = t.shape
    if sh[-1] != n or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must hold rows of {n} values of {dtype} on the current GPU, got {tuple(sh)} "
                         f"{t.dtype} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), n
    st = t.stride()
    if n > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the values of a row must be consecutive")
    ld, rows = None, 1
    for size, step in zip(reversed(sh[:-1]), reversed(st[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = step
        elif step != ld * rows:
            raise ValueError(f"{name}: rows must lie at equal distances")
        rows *= size
    # a row on its own, or rows that overlap (an expanded tensor), have no distance of their own
    if ld is None:
        ld = n
    elif ld < n:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld


def _pack(scales, shape, dev):
    """A scale pack for the INT8 step, whose arrays must fit the shape (None and bare
    structs pass: the C call decides)."""
    if isinstance(scales, ScalePack):
        if scales.device_index != dev:
            raise ValueError(f"the scales must be on the current GPU, they are on {scales.tensor.device}")
        if scales.fits != (shape.ngroups, shape.nheads * shape.headdim):
            for k, v in scales.host.items():
                n = shape.ngroups if k in ScalePack.PER_GROUP else shape.nheads * shape.headdim
                if v.size != n:
                    raise ValueError(f"the scales' {k} holds {v.size} values, the shape has {n}")
    return _scales(scales)


_TORCH_DTYPE = {v: k for k, v in DTYPE_CODE.items()}


def _conv_dims(shape, conv, xbc, dt_raw):
    """Channels, type and rows of the convolution's inputs, which must fit the shape."""
    cd = shape.nheads * shape.headdim + 2 * shape.ngroups * shape.dstate
    n = shape.batch * shape.seqlen
    if conv.channels != cd or (conv.heads is not None and conv.heads != shape.nheads):
        raise ValueError(f"the shape has {cd} channels and {shape.nheads} heads, the parameters {conv.channels} and "
                         f"{conv.heads}")
    if xbc.numel() != n * cd or dt_raw.numel() != n * shape.nheads:
        raise ValueError(f"xbc and dt_raw must hold {n} rows, got {tuple(xbc.shape)} and {tuple(dt_raw.shape)}")
    return cd, _TORCH_DTYPE.get(shape.dtype), n


def ssd_conv_forward(shape, conv, xbc, dt_raw, X, B, C, dt, conv_state=None, pos=None, lengths=None,
                     stream=None):
    """Causal convolution, SiLU and softplus of prompts. ``xbc`` and ``dt_raw`` may be
    column slices of In Proj's output; ``pos`` and ``lengths`` are int32 [B]."""
    cd, td, n = _conv_dims(shape, conv, xbc, dt_raw)
    if n == 0:
        return  # empty tensors have no addresses
    dev = _current_device()
    if conv.device_index != dev:
        raise ValueError("the convolution's parameters must be on the current GPU")
    px, ldx = _rows(xbc, "xbc", cd, td, dev)
    pt, ldt = _rows(dt_raw, "dt_raw", shape.nheads, td, dev)
    b, bc = shape.batch, n * shape.ngroups * shape.dstate
    _check("ssd_conv_forward", LIB.ssd_conv_forward(
        ctypes.byref(shape), ctypes.byref(conv.struct), px, ldx, pt, ldt,
        _dense(lengths, "lengths", b, torch.int32, dev), _dense(pos, "pos", b, torch.int32, dev),
        _dense(conv_state, "conv_state", b * conv.width * cd, td, dev),
        _dense(X, "X", n * shape.nheads * shape.headdim, td, dev), _dense(B, "B", bc, td, dev),
        _dense(C, "C", bc, td, dev), _dense(dt, "dt", n * shape.nheads, td, dev), _stream_on(stream, dev)))


def ssd_conv_decode_step(shape, path, conv, xbc, dt_raw, A, D, scales, conv_state, pos, state, Y,
                         stream=None):
    """One position of the convolution and the SSD: ``conv_state`` and ``state`` are
    updated in place, ``pos`` (int32 [B]) is left for the caller to advance."""
    cd, td, b = _conv_dims(shape, conv, xbc, dt_raw)
    if b == 0:
        return
    dev = _current_device()
    if conv.device_index != dev:
        raise ValueError("the convolution's parameters must be on the current GPU")
    h = shape.nheads
    px, ldx = _rows(xbc, "xbc", cd, td, dev)
    pt, ldt = _rows(dt_raw, "dt_raw", h, td, dev)
    hp = b * h * shape.headdim
    _check("ssd_conv_decode_step", LIB.ssd_conv_decode_step(
        ctypes.byref(shape), path, ctypes.byref(conv.struct), px, ldx, pt, ldt,
        _dense(A, "A", h, torch.float32, dev), _dense(D, "D", h, torch.float32, dev), _pack(scales, shape, dev),
        _dense(conv_state, "conv_state", b * conv.width * cd, td, dev), _dense(pos, "pos", b, torch.int32, dev),
        _dense(state, "state", hp * shape.dstate, torch.int8 if path == SSD_PATH_INT8 else torch.float32, dev),
        _dense(Y, "Y", hp, td, dev), _stream_on(stream, dev)))


def ssd_add_norm(x, residual, residual_out, weight, eps, out=None, q=None, scale=None, stream=None):
    """r = x + residual, RMSNorm of r's rows; the rows in ``out`` and as codes ``q`` with
    a step ``scale`` each. ``x`` may be a column slice; ``residual`` and
    ``residual_out`` share a type, x's or float32 (either may be None)."""
    cols, td, n = x.shape[-1], x.dtype, x.numel()
    if cols == 0:
        raise ValueError("the rows hold no channels")
    if n == 0:
        return
    dev = _current_device()
    rows = n // cols
    px, ldx = _rows(x, "x", cols, td, dev)
    rt = td if residual is None and residual_out is None else (residual_out if residual is None else residual).dtype
    _check("ssd_add_norm", LIB.ssd_add_norm(
        rows, cols, _code(td), px, ldx, _dense(residual, "residual", n, rt, dev), _code(rt),
        _dense(residual_out, "residual_out", n, rt, dev), _dense(weight, "weight", cols, torch.float32, dev), eps,
        _dense(out, "out", n, td, dev), _dense(q, "q", n, torch.int8, dev),
        _dense(scale, "scale", rows, torch.float32, dev), _stream_on(stream, dev)))


def ssd_gated_norm(y, z, groups, weight, eps, out=None, q=None, scale=None, stream=None):
    """RMSNorm over each of ``groups`` runs of channels of y * silu(z); outputs as
    ``ssd_add_norm``. ``z`` may be a column slice of In Proj's output. The row
    length is z's last dimension."""
    cols, td, n = z.shape[-1], y.dtype, z.numel()
    if cols == 0:
        raise ValueError("the rows hold no channels")
    if n == 0:
        return
    dev = _current_device()
    rows = n // cols
    pz, ldz = _rows(z, "z", cols, td, dev)
    _check("ssd_gated_norm", LIB.ssd_gated_norm(
        rows, cols, groups, _code(td), _dense(y, "y", n, td, dev), pz, ldz,
        _dense(weight, "weight", cols, torch.float32, dev), eps, _dense(out, "out", n, td, dev),
        _dense(q, "q", n, torch.int8, dev), _dense(scale, "scale", rows, torch.float32, dev),
        _stream_on(stream, dev)))


def ssd_matmul_i8_workspace_bytes(m, n, k) -> int:
    return int(LIB.ssd_matmul_i8_workspace_bytes(m, n, k))


def ssd_matmul_i8_workspace(m, n, k, device="cuda"):
    """A workspace for products of this size on ``device`` (None where none is needed)."""
    need = ssd_matmul_i8_workspace_bytes(m, n, k)
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def ssd_matmul_i8(a, a_scale, w, w_scale, bias, out, workspace=None, stream=None):
    """out = a_scale * w_scale * (a @ w.T) + bias for int8 a [..., K], w [N, K]; bias may
    be None. ``workspace``: see the C call (None will do)."""
    n, k = w.shape
    if a.shape[-1] != k:
        raise ValueError("a and w must agree in their last dimension")
    if k == 0:
        raise ValueError("a and w hold no columns")
    m = a.numel() // k
    if m == 0:
        return
    dev = _current_device()
    wsb = 0 if workspace is None else workspace.numel()
    pw = _dense(workspace, "workspace", wsb, torch.uint8, dev)
    _check("ssd_matmul_i8", LIB.ssd_matmul_i8(
        m, n, k, _dense(a, "a", m * k, torch.int8, dev), _dense(a_scale, "a_scale", m, torch.float32, dev),
        _dense(w, "w", n * k, torch.int8, dev), _dense(w_scale, "w_scale", n, torch.float32, dev),
        _dense(bias, "bias", n, torch.float32, dev), _code(out.dtype),
        _dense(out, "out", m * n, out.dtype, dev), pw, wsb, _stream_on(stream, dev)))


def ssd_pack_weight_i8(w: np.ndarray):
    """Host call: a float32 weight matrix [N, K] as int8 codes [N, K] and steps [N]."""
    a = np.ascontiguousarray(w, dtype=np.float32)
    if a.ndim != 2:
        raise ValueError("the weight must be a matrix [N, K]")
    q = np.zeros(a.shape, dtype=np.int8)
    s = np.zeros(a.shape[0], dtype=np.float32)
    _check("ssd_pack_weight_i8", LIB.ssd_pack_weight_i8(a.shape[0], a.shape[1], a.ctypes.data, q.ctypes.data,
                                                        s.ctypes.data))
    return q, s


# ---------------------------------------------------------------------------
# operators that stand beside the SSD in a layer
# ---------------------------------------------------------------------------

def ssd_delta_workspace_bytes(shape) -> int:
    return int(LIB.ssd_delta_workspace_bytes(ctypes.byref(shape)))


def ssd_delta_workspace(shape, device="cuda"):
    """A workspace for ``ssd_delta_forward`` on ``device`` (None where none is needed)."""
    need = ssd_delta_workspace_bytes(shape)
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def _delta_inputs(shape, X, dt, A, B, C, beta, Y, dev):
    """Addresses of the gated delta rule's inputs and output, which must fit the shape."""
    td = _TORCH_DTYPE.get(shape.dtype)
    n = shape.batch * shape.seqlen
    hp, gn = n * shape.nheads * shape.headdim, n * shape.ngroups * shape.dstate
    if beta.numel() != n * shape.nheads:
        raise ValueError(f"beta must hold {n} rows of {shape.nheads} values, got {tuple(beta.shape)}")
    pb, ldb = _rows(beta, "beta", shape.nheads, td, dev)
    return (_dense(X, "X", hp, td, dev), _dense(dt, "dt", n * shape.nheads, td, dev),
            _dense(A, "A", shape.nheads, torch.float32, dev), _dense(B, "B", gn, td, dev), _dense(C, "C", gn, td, dev),
            pb, ldb), _dense(Y, "Y", hp, td, dev)


def _delta_flags(unit, logit) -> int:
    return (SSD_DELTA_UNIT if unit else 0) | (SSD_DELTA_LOGIT if logit else 0)


def ssd_delta_forward(shape, X, dt, A, B, C, beta, Y, final_state=None, initial_state=None, workspace=None, scale=1.0,
                      unit=True, logit=False, eps=1e-6, stream=None):
    """The gated delta rule over prompts: values ``X``, keys ``B``, queries ``C``, write
    strengths ``beta`` [..., H] (may be a column slice of In Proj's output; ``logit``: before
    their logistic function). ``unit`` takes keys and queries to length 1. A ``workspace`` (uint8)
    is allocated here if None, and returned."""
    if shape.batch == 0:
        return workspace
    dev = _current_device()
    ns = shape.batch * shape.nheads * shape.headdim * shape.dstate
    inputs, py = _delta_inputs(shape, X, dt, A, B, C, beta, Y, dev)
    need = ssd_delta_workspace_bytes(shape)
    on = _stream_on(stream, dev)
    if workspace is None and need > 0:
        # from the stream that uses it: memory of the current stream may be in use there still, or again
        own = torch.cuda.ExternalStream(on, device=X.device) if on else torch.cuda.default_stream(dev)
        with torch.cuda.stream(None if stream is None else own):
            workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    wsb = 0 if workspace is None else workspace.numel()
    _check("ssd_delta_forward", LIB.ssd_delta_forward(
        ctypes.byref(shape), _delta_flags(unit, logit), *inputs, scale, eps, py,
        _dense(initial_state, "initial_state", ns, torch.float32, dev),
        _dense(final_state, "final_state", ns, torch.float32, dev), _dense(workspace, "workspace", wsb, torch.uint8, dev),
        wsb, on))
    return workspace


def ssd_delta_step(shape, X, dt, A, B, C, beta, state, Y, scale=1.0, unit=True, logit=False, eps=1e-6, stream=None):
    """One position of the gated delta rule: ``state`` [B,H,P,N] float32 is updated in place.
    ``shape.seqlen`` must be 1."""
    if shape.batch == 0:
        return
    dev = _current_device()
    inputs, py = _delta_inputs(shape, X, dt, A, B, C, beta, Y, dev)
    ns = shape.batch * shape.nheads * shape.headdim * shape.dstate
    _check("ssd_delta_step", LIB.ssd_delta_step(
        ctypes.byref(shape), _delta_flags(unit, logit), *inputs, scale, eps,
        _dense(state, "state", ns, torch.float32, dev), py, _stream_on(stream, dev)))


def ssd_matmul_workspace_bytes(m, n, k, dtype) -> int:
    return int(LIB.ssd_matmul_workspace_bytes(m, n, k, _code(dtype)))


def ssd_matmul_workspace(a, w, out):
    """A workspace for ``ssd_matmul`` on tensors like these (None where it has no use for one: rows that are
    16-byte aligned, few, or fp32)."""
    n, k = w.shape
    m = a.numel() // max(1, k)
    _, lda = _rows(a, "a", k, a.dtype, a.get_device())
    if (a.data_ptr() | w.data_ptr() | lda * a.element_size() | k * a.element_size()) % 16 == 0:
        return None
    need = ssd_matmul_workspace_bytes(m, n, k, a.dtype)
    return torch.empty(need, dtype=torch.uint8, device=out.device) if need else None


def ssd_matmul(a, w, bias, out, act=SSD_ACT_NONE, residual=None, workspace=None, stream=None):
    """out = act(a @ w.T + bias) + residual for a [..., K] (may be a column slice), w [N, K] of a's
    type; ``out`` and ``residual`` (which may be the same tensor) in that type or float32; bias float32 or
    None. ``workspace``: from ``ssd_matmul_workspace``, for rows that are not 16-byte aligned (None will do)."""
    n, k = w.shape
    if a.shape[-1] != k:
        raise ValueError("a and w must agree in their last dimension")
    if k == 0:
        raise ValueError("a and w hold no columns")
    m = a.numel() // k
    if m == 0:
        return
    dev = _current_device()
    td, to = a.dtype, out.dtype
    pa, lda = _rows(a, "a", k, td, dev)
    wsb = 0 if workspace is None else workspace.numel()
    pw = _dense(workspace, "workspace", wsb, torch.uint8, dev)
    _check("ssd_matmul", LIB.ssd_matmul(
        m, n, k, _code(td), pa, lda, _dense(w, "w", n * k, td, dev), _dense(bias, "bias", n, torch.float32, dev), act,
        _dense(residual, "residual", m * n, to, dev), _code(to), _dense(out, "out", m * n, to, dev), pw, wsb,
        _stream_on(stream, dev)))


def ssd_block_norm(x, post_weight, residual, residual_out, weight, eps, out=None, q=None, scale=None, gate=None,
                   gate_act=SSD_ACT_NONE, rows_per_gate=1, res_scale=1.0, stream=None):
    """u = RMSNorm of x's rows, r = act(gate) * u + res_scale * residual, and RMSNorm of r's rows
    in ``out`` and as codes ``q`` with a step ``scale`` each. Row i reads row i // rows_per_gate of
    ``gate``. ``x`` and ``gate`` may be column slices; ``residual`` and ``residual_out`` share a type,
    x's or float32 (either may be None)."""
    cols, td, n = x.shape[-1], x.dtype, x.numel()
    if cols == 0:
        raise ValueError("the rows hold no channels")
    if n == 0:
        return
    dev = _current_device()
    rows = n // cols
    px, ldx = _rows(x, "x", cols, td, dev)
    pg, ldg = None, 0
    if gate is not None:
        pg, ldg = _rows(gate, "gate", cols, td, dev)
        if rows_per_gate <= 0 or gate.numel() // cols < -(-rows // rows_per_gate):
            raise ValueError(f"{rows} rows need a gate for each {rows_per_gate}, got {tuple(gate.shape)}")
    rt = td if residual is None and residual_out is None else (residual_out if residual is None else residual).dtype
    _check("ssd_block_norm", LIB.ssd_block_norm(
        rows, cols, _code(td), px, ldx, _dense(post_weight, "post_weight", cols, torch.float32, dev), pg, ldg,
        rows_per_gate, gate_act, _dense(residual, "residual", n, rt, dev), res_scale, _code(rt),
        _dense(residual_out, "residual_out", n, rt, dev), _dense(weight, "weight", cols, torch.float32, dev), eps,
        _dense(out, "out", n, td, dev), _dense(q, "q", n, torch.int8, dev),
        _dense(scale, "scale", rows, torch.float32, dev), _stream_on(stream, dev)))
