"""Binding of the feed-forward operators (include/mt_layers.h).

``rms_norm``, ``linear`` and their gradients on torch CUDA tensors, and the C entry points under their own
names taking a filled argument structure.  Marshalling only, as in the
package's ``__init__``, which re-exports everything here.
"""
from __future__ import annotations

import ctypes
import struct

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
                ("weight_dtype", _I32)]


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
    code = {_I64: "q", _I32: "i", _P: "Q", _F: "f"}
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
_codes = {}


def _dtype_codes():
    if not _codes:
        import torch
        _codes.update({torch.float16: 1, torch.bfloat16: 2, torch.float32: MT_DTYPE_F32,
                       torch.float8_e4m3fn: MT_DTYPE_E4M3})
    return _codes


def _matrix(t, name, rows, cols, dtype, device):
    """(pointer, row pitch) of a rows x cols CUDA matrix with unit column
    stride; any pitch that holds a row serves a single row."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be {rows} x {cols}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows <= 1 or ld < 1:
        if rows > 1:
            raise ValueError(f"{name}'s rows overlap")
        ld = max(cols, 1)
    return t.data_ptr(), ld


def _vector(t, name, n, dtypes, device):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a {' or '.join(map(str, dtypes))} CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")
    return t.data_ptr()


def _first(t, name, dtypes):
    """Checks of the operand whose device and type the others follow."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(map(str, dtypes))}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")


def _call(fn, packed, device, stream):
    """Runs one packed C call on the operands' device and stream."""
    import torch
    from . import MT_OK, MtError, lib
    s = stream if stream is not None else torch.cuda.current_stream(device).cuda_stream
    f = getattr(lib(), fn)
    if device.index == torch.cuda.current_device():
        st = f(packed, s)
    else:
        with torch.cuda.device(device):
            st = f(packed, s)
    if st != MT_OK:
        raise MtError(st, fn)


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
    import torch
    codes = _dtype_codes()
    _first(x, "x", (torch.float16, torch.bfloat16, torch.float32))
    rows, d = x.shape
    dt, dev = x.dtype, x.device
    e4m3 = out_dtype == torch.float8_e4m3fn
    if out_dtype is None:
        out_dtype = dt
    elif not e4m3 and out_dtype != dt:
        raise TypeError("out_dtype must be x's dtype or torch.float8_e4m3fn")
    xp, ldx = _matrix(x, "x", rows, d, dt, dev)
    rp = ldr = hp = ldh = wp = sp = wcode = 0
    if weight is not None:
        wp = _vector(weight, "weight", d, (dt, torch.float32), dev)
        wcode = codes[weight.dtype]
    h = x
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", rows, d, dt, dev)
        h = torch.empty((rows, d), dtype=dt, device=dev) if h_out is None else h_out
        hp, ldh = _matrix(h, "h_out", rows, d, dt, dev)
    elif h_out is not None:
        raise ValueError("h_out needs a residual")
    y = torch.empty((rows, d), dtype=out_dtype, device=dev) if out is None else out
    yp, ldy = _matrix(y, "out", rows, d, out_dtype, dev)
    # One allocation: the reciprocal norms, then the scales.
    stats = torch.empty((2 if e4m3 else 1, rows), dtype=torch.float32, device=dev)
    rstd = stats[0]
    if e4m3:
        scale = stats[1]
        sp = scale.data_ptr()
    _call("mt_rms_norm",
          _pack_rms_norm(rows, d, xp, ldx, rp, ldr, wp, hp, ldh, yp, ldy, sp, rstd.data_ptr(),
                         eps, codes[dt], codes[out_dtype], wcode), dev, stream)
    return (y, scale, h, rstd) if e4m3 else (y, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, dh=None, need_weight=True, out=None, stream=None):
    """``(dx, dweight)``: the gradient of ``rms_norm`` through
    mt_rms_norm_backward.

    dy: gradient of y; h and rstd: the forward call's; dh: the gradient that
    reaches h directly (the residual stream), added to dx.  dx, in dy's
    dtype, is the gradient of x and of the residual alike; dweight is
    float32 (None when ``need_weight`` is false).  ``out`` receives dx when
    given and may be dy or dh."""
    import torch
    codes = _dtype_codes()
    _first(dy, "dy", (torch.float16, torch.bfloat16, torch.float32))
    rows, d = dy.shape
    dt, dev = dy.dtype, dy.device
    dyp, lddy = _matrix(dy, "dy", rows, d, dt, dev)
    hp, ldh = _matrix(h, "h", rows, d, dt, dev)
    rp = _vector(rstd, "rstd", rows, (torch.float32,), dev)
    wp = wcode = dhp = lddh = dwp = 0
    if weight is not None:
        wp = _vector(weight, "weight", d, (dt, torch.float32), dev)
        wcode = codes[weight.dtype]
    if dh is not None:
        dhp, lddh = _matrix(dh, "dh", rows, d, dt, dev)
    dx = torch.empty((rows, d), dtype=dt, device=dev) if out is None else out
    dxp, lddx = _matrix(dx, "out", rows, d, dt, dev)
    dweight = None
    if need_weight:
        dweight = torch.empty(d, dtype=torch.float32, device=dev)
        dwp = dweight.data_ptr()
    _call("mt_rms_norm_backward",
          _pack_rms_norm_backward(rows, d, dyp, lddy, hp, ldh, wp, rp, dhp, lddh, dxp, lddx, dwp,
                                  codes[dt], wcode), dev, stream)
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
    import torch
    codes = _dtype_codes()
    _first(a, "a", (torch.float16, torch.bfloat16, torch.float8_e4m3fn))
    M, K = a.shape
    dt, dev = a.dtype, a.device
    if not isinstance(b, torch.Tensor) or b.dim() != 2:
        raise ValueError("b must be a 2-D CUDA tensor")
    N = b.shape[0] if trans_b else b.shape[1]
    ap, lda = _matrix(a, "a", M, K, dt, dev)
    bp, ldb = _matrix(b, "b", *((N, K) if trans_b else (K, N)), dt, dev)
    bias_p = rp = ldr = zp = ldz = sap = sbp = 0
    if dt == torch.float8_e4m3fn:
        if not trans_b:
            raise ValueError("8-bit inputs need b stored N x K (trans_b)")
        sap = _vector(scale_a, "scale_a", M, (torch.float32,), dev)
        sbp = _vector(scale_b, "scale_b", N, (torch.float32,), dev)
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in (torch.float16, torch.bfloat16, torch.float32):
            raise TypeError("out_dtype must be float16, bfloat16 or float32")
    else:
        if scale_a is not None or scale_b is not None:
            raise ValueError("scales go with float8_e4m3fn inputs")
        out_dtype = out_dtype or dt
        if out_dtype not in (dt, torch.float32):
            raise TypeError("out_dtype must be a's dtype or float32")
    if bias is not None:
        bias_p = _vector(bias, "bias", N, (torch.float32,), dev)
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", M, N, out_dtype, dev)
    y = torch.empty((M, N), dtype=out_dtype, device=dev) if out is None else out
    yp, ldy = _matrix(y, "out", M, N, out_dtype, dev)
    if preact:
        z = torch.empty((M, N), dtype=out_dtype, device=dev)
        zp, ldz = z.data_ptr(), max(N, 1)
    _call("mt_linear",
          _pack_linear(M, N, K, ap, lda, bp, ldb, yp, ldy, zp, ldz, rp, ldr, bias_p, sap, sbp,
                       int(trans_b), codes[dt], codes[out_dtype], _activation(activation), 0, 0),
          dev, stream)
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
    import torch
    codes = _dtype_codes()
    _first(dy, "dy", (torch.float16, torch.bfloat16))
    M, N = dy.shape
    dt, dev = dy.dtype, dy.device
    act = _activation(activation)
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a must be a 2-D CUDA tensor")
    K = a.shape[1]
    db_dtype = db_dtype or dt
    if db_dtype not in (dt, torch.float32):
        raise TypeError("db_dtype must be a's dtype or float32")
    dyp, lddy = _matrix(dy, "dy", M, N, dt, dev)
    ap, lda = _matrix(a, "a", M, K, dt, dev)
    shape = (N, K) if trans_b else (K, N)
    bp, ldb = _matrix(b, "b", *shape, dt, dev)
    zp = ldz = dap = dbp = dbiasp = 0
    if act != MT_ACT_NONE:
        zp, ldz = _matrix(z, "z", M, N, dt, dev)
    da = db = dbias = None
    if need_a:
        da = torch.empty((M, K), dtype=dt, device=dev)
        dap = da.data_ptr()
    if need_b:
        db = torch.empty(shape, dtype=db_dtype, device=dev)
        dbp = db.data_ptr()
    if need_bias:
        dbias = torch.empty(N, dtype=torch.float32, device=dev)
        dbiasp = dbias.data_ptr()
    _call("mt_linear_backward",
          _pack_linear_backward(M, N, K, dyp, lddy, zp, ldz, ap, lda, bp, ldb, dap, max(K, 1),
                                dbp, max(shape[1], 1), dbiasp, int(trans_b), codes[dt],
                                codes[db_dtype], act), dev, stream)
    return da, db, dbias
