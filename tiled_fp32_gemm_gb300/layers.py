"""Binding of the feed-forward operators (include/mt_layers.h).

``rms_norm``, ``linear`` and their gradients on torch CUDA tensors, and the C
entry points under their own names taking a filled argument structure.
Marshalling only, as in the package's ``__init__``, which re-exports
everything here.  A call that allocates its outputs and runs on the current
stream of the current device is marshalled natively (csrc/torch_binding.cpp,
built beside the library): 6 us of the host's time for an rms_norm with a
residual, 16 us here.  ``stream`` (a handle; None: the current stream) runs a
call elsewhere, its outputs in that stream's memory; operands have to stay
until its work is done.
"""
from __future__ import annotations

import ctypes
import struct

from .streams import elsewhere

_I64, _I32, _P, _F = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float

MT_DTYPE_F32 = 3
MT_DTYPE_E4M3 = 4
MT_E4M3_MAX = 448.0
MT_SCALE_MIN = 2.0 ** -126

MT_ACT_NONE, MT_ACT_RELU, MT_ACT_GELU, MT_ACT_GELU_TANH, MT_ACT_SILU = range(5)
ACTIVATIONS = {None: MT_ACT_NONE, "none": MT_ACT_NONE, "relu": MT_ACT_RELU, "gelu": MT_ACT_GELU,
               "gelu_tanh": MT_ACT_GELU_TANH, "silu": MT_ACT_SILU}


class mt_rms_norm_args(ctypes.Structure):
    _fields_ = [("rows", _I64), ("d", _I64), ("x", _P), ("ldx", _I64), ("residual", _P),
                ("ldr", _I64), ("weight", _P), ("h", _P), ("ldh", _I64), ("y", _P),
                ("ldy", _I64), ("scale", _P), ("rstd", _P), ("eps", _F), ("dtype", _I32),
                ("out_dtype", _I32), ("weight_dtype", _I32)]


class mt_rms_norm_backward_args(ctypes.Structure):
    _fields_ = [("rows", _I64), ("d", _I64), ("dy", _P), ("lddy", _I64), ("h", _P),
                ("ldh", _I64), ("weight", _P), ("rstd", _P), ("dh", _P), ("lddh", _I64),
                ("dx", _P), ("lddx", _I64), ("dweight", _P), ("dtype", _I32),
                ("weight_dtype", _I32), ("fault_inject", _I32), ("reserved", _I32)]


class mt_linear_args(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64), ("A", _P), ("lda", _I64), ("B", _P),
                ("ldb", _I64), ("Y", _P), ("ldy", _I64), ("Z", _P), ("ldz", _I64),
                ("residual", _P), ("ldr", _I64), ("bias", _P), ("scale_a", _P),
                ("scale_b", _P), ("trans_b", _I32), ("dtype", _I32), ("out_dtype", _I32),
                ("activation", _I32), ("fault_inject", _I32), ("reserved", _I32)]


class mt_linear_backward_args(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64), ("dY", _P), ("lddy", _I64), ("Z", _P),
                ("ldz", _I64), ("A", _P), ("lda", _I64), ("B", _P), ("ldb", _I64), ("dA", _P),
                ("ldda", _I64), ("dB", _P), ("lddb", _I64), ("dbias", _P), ("trans_b", _I32),
                ("dtype", _I32), ("db_dtype", _I32), ("activation", _I32)]


# name -> (restype, argtypes): every function include/mt_layers.h declares.
# The argument structure is passed as its bytes or by reference.
SIGNATURES = {
    "mt_rms_norm": (ctypes.c_int, [_P, _P]),
    "mt_rms_norm_backward": (ctypes.c_int, [_P, _P]),
    "mt_linear": (ctypes.c_int, [_P, _P]),
    "mt_linear_backward": (ctypes.c_int, [_P, _P]),
    "mt_linear_plan": (ctypes.c_int, [_P, ctypes.c_int, _P]),
}


def _packer(cls):
    """struct.Struct.pack with the layout of a ctypes structure: one call
    fills every field (None is not taken: NULL is 0)."""
    code = {_I64: "q", _I32: "i", _P: "Q", _F: "f", ctypes.c_uint64: "Q", ctypes.c_double: "d"}
    s = struct.Struct("@" + "".join(code[t] for _, t in cls._fields_))
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_rms_norm = _packer(mt_rms_norm_args)
_pack_rms_norm_backward = _packer(mt_rms_norm_backward_args)
_pack_linear = _packer(mt_linear_args)
_pack_linear_backward = _packer(mt_linear_backward_args)


# --- the C entry points, same names -----------------------------------------
def mt_rms_norm(args: mt_rms_norm_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_rms_norm(ctypes.byref(args), stream)


def mt_rms_norm_backward(args: mt_rms_norm_backward_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_rms_norm_backward(ctypes.byref(args), stream)


def mt_linear(args: mt_linear_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_linear(ctypes.byref(args), stream)


def mt_linear_plan(args: mt_linear_args, sms: int):
    from . import lib, mt_plan
    out = mt_plan()
    st = lib().mt_linear_plan(ctypes.byref(args), sms, ctypes.byref(out))
    return st, out


def mt_linear_backward(args: mt_linear_backward_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_linear_backward(ctypes.byref(args), stream)


# --- torch convenience (marshalling only) ------------------------------------
# What a call needs of torch and the library, looked up at the first call:
# for a few tokens the host's time is what a call takes.
_torch = None
_codes = {}
_FLOATS = _HALVES = _PRODUCTS = _F32 = _F8 = None
_empty = _raw_stream = _device_now = None
_functions = {}
_native = None


def _setup():
    global _torch, _FLOATS, _HALVES, _PRODUCTS, _F32, _F8, _empty, _raw_stream, _device_now
    import torch
    from . import lib
    handle = lib()
    for name in SIGNATURES:
        _functions[name] = getattr(handle, name)
    _codes.update({torch.float16: 1, torch.bfloat16: 2, torch.float32: MT_DTYPE_F32,
                   torch.float8_e4m3fn: MT_DTYPE_E4M3})
    _HALVES = (torch.float16, torch.bfloat16)
    _FLOATS = (*_HALVES, torch.float32)
    _F32, _F8 = torch.float32, torch.float8_e4m3fn
    _PRODUCTS = (*_HALVES, _F8)
    _empty, _device_now = torch.empty, torch.cuda.current_device
    _load_native()
    # The current stream's handle without building a Stream object.
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch


def _load_native():
    """The native marshalling, if it was built for this torch (calls are the
    same without it, and take the host longer)."""
    global _native
    import importlib.util
    import os
    from .build import binding_path
    path = binding_path()
    if os.path.exists(path):
        spec = importlib.util.spec_from_file_location("mt_torch_binding", path)
        _native = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_native)
        _point_native()


def _point_native():
    """Points the native marshalling at the library the binding calls."""
    if _native is not None:
        _native.use_library(*(ctypes.cast(_functions[n], _P).value
                              for n in ("mt_rms_norm", "mt_rms_norm_backward", "mt_linear",
                                        "mt_linear_backward")))


def _done(result, name):
    """What a native call returned: the results, or a status to raise."""
    if type(result) is int:
        from . import MtError
        raise MtError(result, name)
    return result


def _first(t, name, dtypes):
    """(rows, columns, dtype, device, pointer, row pitch) of the operand whose
    device and type the others follow."""
    if not isinstance(t, _torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dtype, shape, device = t.dtype, t.shape, t.device
    if dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(map(str, dtypes))}")
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    return rows, cols, dtype, device, *_matrix(t, name, rows, cols, dtype, device)


def _matrix(t, name, rows, cols, dtype, device):
    """(pointer, row pitch) of a rows x cols matrix on `device` with unit
    column stride; any pitch that holds a row serves a single row."""
    try:
        right = t.dtype == dtype and t.device == device
    except AttributeError:
        right = False
    if not right:
        _refuse(t, name, (dtype,), device)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {rows} x {cols}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1:
        return t.data_ptr(), cols or 1
    if ld < 1:
        raise ValueError(f"{name}'s rows overlap")
    return t.data_ptr(), ld


def _vector(t, name, n, dtypes, device):
    """(pointer, dtype code) of a contiguous vector of n values on `device`."""
    try:
        dtype = t.dtype
        right = dtype in dtypes and t.device == device
    except AttributeError:
        right = False
    if not right:
        _refuse(t, name, dtypes, device)
    if t.shape != (n,) or (n > 1 and t.stride() != (1,)):
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr(), _codes[dtype]


def _refuse(t, name, dtypes, device):
    """Says what is wrong with an operand of another type or place."""
    if not isinstance(t, _torch.Tensor) or t.dtype not in dtypes or not t.is_cuda:
        raise TypeError(f"{name} must be a {' or '.join(map(str, dtypes))} CUDA tensor")
    raise ValueError(f"{name} is on {t.device}, the other operands on {device}")


def _result(out, name, rows, cols, dtype, device):
    """(tensor, pointer, row pitch): `out` checked, or a new matrix."""
    if out is None:
        out = _empty((rows, cols), dtype=dtype, device=device)
        return out, out.data_ptr(), cols or 1
    return (out, *_matrix(out, name, rows, cols, dtype, device))


def _call(name, packed, device):
    """Runs one packed C call on the operands' device, on its current stream."""
    index = device.index
    stream = _raw_stream(index)
    if index == _device_now():
        st = _functions[name](packed, stream)
    else:
        with _torch.cuda.device(device):
            st = _functions[name](packed, stream)
    if st:
        from . import MtError
        raise MtError(st, name)


def rms_norm(x, weight, residual=None, eps=1e-6, out_dtype=None, out=None, h_out=None,
             stream=None):
    """Root-mean-square norm of h = x + residual over the last dimension,
    times ``weight``, through mt_rms_norm.

    x, residual: 2-D CUDA tensors of one dtype (float16, bfloat16 or
    float32), rows may be strided; weight: a vector in that dtype or float32
    (None: ones).  Returns ``(y, h, rstd)``; with ``out_dtype=
    torch.float8_e4m3fn`` ``(q, scale, h, rstd)``: 8-bit rows with one
    float32 scale each, y = q * scale.  h is x + residual in x's dtype (x
    itself when there is no residual), rstd the float32 reciprocal norms
    that ``rms_norm_backward`` takes.  ``out`` and ``h_out`` receive y (or q)
    and h when given; h_out may be residual or x."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(rms_norm, stream, x, weight, residual, eps, out_dtype, out, h_out)
    if _native is not None and out is None and h_out is None:
        r = _native.rms_norm(x, weight, residual, float(eps), out_dtype)
        if r is not None:
            return _done(r, "mt_rms_norm")
    rows, d, dt, dev, xp, ldx = _first(x, "x", _FLOATS)
    if out_dtype is None:
        out_dtype = dt
    elif out_dtype != dt and out_dtype != _F8:
        raise TypeError("out_dtype must be x's dtype or torch.float8_e4m3fn")
    rp = ldr = hp = ldh = wp = sp = wcode = 0
    if weight is not None:
        wp, wcode = _vector(weight, "weight", d, (dt, _F32), dev)
    h = x
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", rows, d, dt, dev)
        h, hp, ldh = _result(h_out, "h_out", rows, d, dt, dev)
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    y, yp, ldy = _result(out, "out", rows, d, out_dtype, dev)
    rstd = _empty(rows, dtype=_F32, device=dev)
    scale = None
    if out_dtype == _F8:
        scale = _empty(rows, dtype=_F32, device=dev)
        sp = scale.data_ptr()
    _call("mt_rms_norm",
          _pack_rms_norm(rows, d, xp, ldx, rp, ldr, wp, hp, ldh, yp, ldy, sp, rstd.data_ptr(),
                         eps, _codes[dt], _codes[out_dtype], wcode), dev)
    return (y, h, rstd) if scale is None else (y, scale, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, dh=None, need_weight=True, out=None, stream=None):
    """``(dx, dweight)``: the gradient of ``rms_norm`` through
    mt_rms_norm_backward.

    dy: gradient of y; h and rstd: the forward call's; dh: the gradient that
    reaches h directly (the residual stream), added to dx.  dx, in dy's
    dtype, is the gradient of x and of the residual alike; dweight is
    float32 (None when ``need_weight`` is false).  ``out`` receives dx when
    given and may be dy or dh."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(rms_norm_backward, stream, dy, h, weight, rstd, dh, need_weight, out)
    if _native is not None and out is None:
        r = _native.rms_norm_backward(dy, h, weight, rstd, dh, bool(need_weight))
        if r is not None:
            return _done(r, "mt_rms_norm_backward")
    rows, d, dt, dev, dyp, lddy = _first(dy, "dy", _FLOATS)
    hp, ldh = _matrix(h, "h", rows, d, dt, dev)
    rp, _ = _vector(rstd, "rstd", rows, (_F32,), dev)
    wp = wcode = dhp = lddh = dwp = 0
    if weight is not None:
        wp, wcode = _vector(weight, "weight", d, (dt, _F32), dev)
    if dh is not None:
        dhp, lddh = _matrix(dh, "dh", rows, d, dt, dev)
    dx, dxp, lddx = _result(out, "out", rows, d, dt, dev)
    dweight = None
    if need_weight:
        dweight = _empty(d, dtype=_F32, device=dev)
        dwp = dweight.data_ptr()
    _call("mt_rms_norm_backward",
          _pack_rms_norm_backward(rows, d, dyp, lddy, hp, ldh, wp, rp, dhp, lddh, dxp, lddx, dwp,
                                  _codes[dt], wcode, 0, 0), dev)
    return dx, dweight


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {sorted(k for k in ACTIVATIONS if k)} "
                         "or None") from None


def linear(a, b, bias=None, activation=None, residual=None, trans_b=False, scale_a=None,
           scale_b=None, out_dtype=None, out=None, preact=False, stream=None):
    """act(a @ op(b) + bias) + residual in one pass, through mt_linear.

    a: M x K, b: K x N (or N x K with ``trans_b``), 2-D CUDA tensors of one
    16-bit dtype, rows may be strided; bias: N float32 values; residual:
    M x N in the output's dtype; activation: None, "relu", "gelu",
    "gelu_tanh" or "silu".  With float8_e4m3fn a and b (``trans_b`` only) the
    product is scaled by ``scale_a`` (M float32 values, one per row of a)
    and ``scale_b`` (N, one per column of the output).  ``out_dtype``: a's
    dtype (bfloat16 for 8-bit inputs) unless given; float32 is always
    allowed.  Returns the output (``out`` when given, which may be the
    residual), or ``(output, z)`` with the pre-activation z in the output's
    dtype when ``preact`` is set."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(linear, stream, a, b, bias, activation, residual, trans_b, scale_a,
                         scale_b, out_dtype, out, preact)
    act = _activation(activation)
    if _native is not None and out is None:
        r = _native.linear(a, b, bias, act, residual, bool(trans_b), scale_a, scale_b, out_dtype,
                           bool(preact))
        if r is not None:
            return _done(r, "mt_linear")
    M, K, dt, dev, ap, lda = _first(a, "a", _PRODUCTS)
    if not isinstance(b, _torch.Tensor) or b.dim() != 2:
        raise ValueError("b must be a 2-D CUDA tensor")
    bias_p = rp = ldr = zp = ldz = sap = sbp = 0
    if trans_b:
        N = b.shape[0]
        bp, ldb = _matrix(b, "b", N, K, dt, dev)
    else:
        N = b.shape[1]
        bp, ldb = _matrix(b, "b", K, N, dt, dev)
    if dt == _F8:
        if not trans_b:
            raise ValueError("8-bit inputs need b stored N x K (trans_b)")
        sap, _ = _vector(scale_a, "scale_a", M, (_F32,), dev)
        sbp, _ = _vector(scale_b, "scale_b", N, (_F32,), dev)
        out_dtype = out_dtype or _torch.bfloat16
        if out_dtype not in _FLOATS:
            raise TypeError("out_dtype must be float16, bfloat16 or float32")
    else:
        if scale_a is not None or scale_b is not None:
            raise ValueError("scales go with float8_e4m3fn inputs")
        if out_dtype is None:
            out_dtype = dt
        elif out_dtype != dt and out_dtype != _F32:
            raise TypeError("out_dtype must be a's dtype or float32")
    if bias is not None:
        bias_p, _ = _vector(bias, "bias", N, (_F32,), dev)
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", M, N, out_dtype, dev)
    y, yp, ldy = _result(out, "out", M, N, out_dtype, dev)
    z = None
    if preact:
        z, zp, ldz = _result(None, "z", M, N, out_dtype, dev)
    _call("mt_linear",
          _pack_linear(M, N, K, ap, lda, bp, ldb, yp, ldy, zp, ldz, rp, ldr, bias_p, sap, sbp,
                       1 if trans_b else 0, _codes[dt], _codes[out_dtype], act, 0, 0),
          dev)
    return (y, z) if preact else y


def linear_backward(dy, a, b, z=None, activation=None, trans_b=False, need_a=True, need_b=True,
                    need_bias=True, db_dtype=None, stream=None):
    """``(da, db, dbias)``: the gradient of ``linear`` with 16-bit inputs,
    through mt_linear_backward (None for what is not needed; the residual's
    gradient is dy itself).

    dy: M x N gradient of the output, in a's dtype; z: the forward call's
    pre-activation (needed unless ``activation`` is None); a, b, ``trans_b``
    as there.  da has a's dtype, db is stored as b in ``db_dtype`` (a's, or
    float32), dbias is float32."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(linear_backward, stream, dy, a, b, z, activation, trans_b, need_a, need_b,
                         need_bias, db_dtype)
    act = _activation(activation)
    if _native is not None:
        r = _native.linear_backward(dy, a, b, z, act, bool(trans_b), bool(need_a), bool(need_b),
                                    bool(need_bias), db_dtype)
        if r is not None:
            return _done(r, "mt_linear_backward")
    M, N, dt, dev, dyp, lddy = _first(dy, "dy", _HALVES)
    if not isinstance(a, _torch.Tensor) or a.dim() != 2:
        raise ValueError("a must be a 2-D CUDA tensor")
    K = a.shape[1]
    if db_dtype is None:
        db_dtype = dt
    elif db_dtype != dt and db_dtype != _F32:
        raise TypeError("db_dtype must be a's dtype or float32")
    ap, lda = _matrix(a, "a", M, K, dt, dev)
    rows, cols = (N, K) if trans_b else (K, N)
    bp, ldb = _matrix(b, "b", rows, cols, dt, dev)
    zp = ldz = dap = ldda = dbp = lddb = dbiasp = 0
    if act != MT_ACT_NONE:
        zp, ldz = _matrix(z, "z", M, N, dt, dev)
    da = db = dbias = None
    if need_a:
        da, dap, ldda = _result(None, "da", M, K, dt, dev)
    if need_b:
        db, dbp, lddb = _result(None, "db", rows, cols, db_dtype, dev)
    if need_bias:
        dbias = _empty(N, dtype=_F32, device=dev)
        dbiasp = dbias.data_ptr()
    _call("mt_linear_backward",
          _pack_linear_backward(M, N, K, dyp, lddy, zp, ldz, ap, lda, bp, ldb, dap, ldda, dbp,
                                lddb, dbiasp, 1 if trans_b else 0, _codes[dt],
                                _codes[db_dtype], act), dev)
    return da, db, dbias
