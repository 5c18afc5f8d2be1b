"""Binding of the residual joins and the vocabulary's loss
(include/mt_model.h).

``layer_norm``, ``dropout``, ``linear_cross_entropy`` and their gradients on
torch CUDA tensors, and the C entry points under their own names taking a
filled argument structure.  Marshalling only, as in ``layers`` (natively where
a call allocates its outputs); ``stream`` (a
handle; None: the current stream) runs a call elsewhere, its outputs in that
stream's memory; operands have to stay until its work is done.
"""
from __future__ import annotations

import ctypes

from . import layers
from .streams import elsewhere

_I64, _I32, _P, _F = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
_U64, _D = ctypes.c_uint64, ctypes.c_double


class mt_layer_norm_args(ctypes.Structure):
    _fields_ = [("rows", _I64), ("d", _I64), ("x", _P), ("ldx", _I64), ("residual", _P),
                ("ldr", _I64), ("weight", _P), ("bias", _P), ("h", _P), ("ldh", _I64), ("y", _P),
                ("ldy", _I64), ("mean", _P), ("rstd", _P), ("seed", _P), ("sequence", _U64),
                ("dropout", _D), ("eps", _F), ("dtype", _I32), ("weight_dtype", _I32),
                ("reserved", _I32)]


class mt_layer_norm_backward_args(ctypes.Structure):
    _fields_ = [("rows", _I64), ("d", _I64), ("dy", _P), ("lddy", _I64), ("h", _P),
                ("ldh", _I64), ("weight", _P), ("mean", _P), ("rstd", _P), ("dh", _P),
                ("lddh", _I64), ("dx", _P), ("lddx", _I64), ("dresidual", _P), ("lddres", _I64),
                ("dweight", _P), ("dbias", _P), ("seed", _P), ("sequence", _U64),
                ("dropout", _D), ("dtype", _I32), ("weight_dtype", _I32),
                ("fault_inject", _I32), ("reserved", _I32)]


class mt_dropout_args(ctypes.Structure):
    _fields_ = [("rows", _I64), ("d", _I64), ("x", _P), ("ldx", _I64), ("residual", _P),
                ("ldr", _I64), ("y", _P), ("ldy", _I64), ("seed", _P), ("sequence", _U64),
                ("p", _D), ("dtype", _I32), ("reserved", _I32)]


class mt_linear_cross_entropy_args(ctypes.Structure):
    _fields_ = [("T", _I64), ("K", _I64), ("V", _I64), ("A", _P), ("lda", _I64), ("B", _P),
                ("ldb", _I64), ("target", _P), ("loss", _P), ("lse", _P),
                ("ignore_index", _I64), ("label_smoothing", _F), ("z_loss", _F),
                ("trans_b", _I32), ("dtype", _I32), ("fault_inject", _I32), ("reserved", _I32)]


class mt_linear_cross_entropy_backward_args(ctypes.Structure):
    _fields_ = [("T", _I64), ("K", _I64), ("V", _I64), ("dloss", _P), ("A", _P), ("lda", _I64),
                ("B", _P), ("ldb", _I64), ("target", _P), ("lse", _P), ("dA", _P),
                ("ldda", _I64), ("dB", _P), ("lddb", _I64), ("ignore_index", _I64),
                ("label_smoothing", _F), ("z_loss", _F), ("trans_b", _I32), ("dtype", _I32),
                ("db_dtype", _I32), ("reserved", _I32)]


# name -> (restype, argtypes): every function include/mt_model.h declares.
# The argument structure is passed as its bytes or by reference.
SIGNATURES = {name: (ctypes.c_int, [_P, _P]) for name in (
    "mt_layer_norm", "mt_layer_norm_backward", "mt_dropout", "mt_linear_cross_entropy",
    "mt_linear_cross_entropy_backward")}

_pack_layer_norm = layers._packer(mt_layer_norm_args)
_pack_layer_norm_backward = layers._packer(mt_layer_norm_backward_args)
_pack_dropout = layers._packer(mt_dropout_args)
_pack_loss = layers._packer(mt_linear_cross_entropy_args)
_pack_loss_backward = layers._packer(mt_linear_cross_entropy_backward_args)


# --- the C entry points, same names -----------------------------------------
def mt_layer_norm(args: mt_layer_norm_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_layer_norm(ctypes.byref(args), stream)


def mt_layer_norm_backward(args: mt_layer_norm_backward_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_layer_norm_backward(ctypes.byref(args), stream)


def mt_dropout(args: mt_dropout_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_dropout(ctypes.byref(args), stream)


def mt_linear_cross_entropy(args: mt_linear_cross_entropy_args, stream: int = 0) -> int:
    from . import lib
    return lib().mt_linear_cross_entropy(ctypes.byref(args), stream)


def mt_linear_cross_entropy_backward(args: mt_linear_cross_entropy_backward_args,
                                     stream: int = 0) -> int:
    from . import lib
    return lib().mt_linear_cross_entropy_backward(ctypes.byref(args), stream)


# --- torch convenience (marshalling only) ------------------------------------
_torch = None


def _setup():
    global _torch
    if layers._torch is None:
        layers._setup()
    from . import lib
    handle = lib()
    for name in SIGNATURES:
        layers._functions.setdefault(name, getattr(handle, name))
    _point_native()
    _torch = layers._torch


def _point_native():
    """Points the native marshalling at the library the binding calls."""
    if layers._native is not None:
        layers._native.use_model_library(
            *(ctypes.cast(layers._functions[n], _P).value for n in SIGNATURES))


def _dropped(p, seed, sequence, device):
    """(p, seed's address, sequence), checked."""
    p, sequence = float(p), int(sequence)
    if not 0.0 <= p < 1.0:
        raise ValueError("the probability to drop must be in [0, 1)")
    if not 0 <= sequence < 2 ** 64:
        raise ValueError("sequence must be in [0, 2^64)")
    if p == 0.0 and seed is None:
        return p, 0, sequence
    if not isinstance(seed, _torch.Tensor) or seed.dtype != _torch.int64 or not seed.is_cuda or \
            seed.numel() != 1:
        raise TypeError("seed must be an int64 CUDA tensor of one value")
    if seed.device != device:
        raise ValueError(f"seed is on {seed.device}, the other operands on {device}")
    return p, seed.data_ptr(), sequence


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5, dropout=0.0, seed=None,
               sequence=0, out=None, h_out=None, stream=None):
    """Layer norm of h = drop(x) + residual over the last dimension, times
    ``weight`` plus ``bias``, through mt_layer_norm.

    x, residual: 2-D CUDA tensors of one dtype (float16, bfloat16 or
    float32), rows may be strided; weight, bias: vectors, both in that dtype or
    both float32 (None: ones, zeros).  ``dropout``: the probability to drop an
    element of x; its mask comes from ``seed`` (an int64 CUDA tensor of one
    value, read when the kernel runs) and ``sequence`` (an integer that tells
    the calls of one seed apart) and is never stored.  Returns ``(y, h, mean,
    rstd)``: h in x's dtype (x itself when nothing is dropped or added), mean
    and rstd the float32 statistics that ``layer_norm_backward`` takes.
    ``out`` and ``h_out`` receive y and h when given; h_out may be residual or
    x."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(layer_norm, stream, x, weight, bias, residual, eps, dropout, seed,
                         sequence, out, h_out)
    if layers._native is not None and out is None and h_out is None:
        r = layers._native.layer_norm(x, weight, bias, residual, float(eps), dropout, seed,
                                      sequence)
        if r is not None:
            return layers._done(r, "mt_layer_norm")
    rows, d, dt, dev, xp, ldx = layers._first(x, "x", layers._FLOATS)
    p, sp, sequence = _dropped(dropout, seed, sequence, dev)
    rp = ldr = hp = ldh = wp = bp = wcode = 0
    kinds = (dt, _torch.float32)
    if weight is not None:
        wp, wcode = layers._vector(weight, "weight", d, kinds, dev)
        kinds = (weight.dtype,)
    if bias is not None:
        bp, wcode = layers._vector(bias, "bias", d, kinds, dev)
    h = x
    if residual is not None:
        rp, ldr = layers._matrix(residual, "residual", rows, d, dt, dev)
    if residual is not None or p > 0.0:
        h, hp, ldh = layers._result(h_out, "h_out", rows, d, dt, dev)
    elif h_out is not None:
        raise ValueError("h_out needs a residual or dropout")
    y, yp, ldy = layers._result(out, "out", rows, d, dt, dev)
    mean = layers._empty(rows, dtype=_torch.float32, device=dev)
    rstd = layers._empty(rows, dtype=_torch.float32, device=dev)
    layers._call("mt_layer_norm",
                 _pack_layer_norm(rows, d, xp, ldx, rp, ldr, wp, bp, hp, ldh, yp, ldy,
                                  mean.data_ptr(), rstd.data_ptr(), sp, sequence, p, eps,
                                  layers._codes[dt], wcode, 0), dev)
    return y, h, mean, rstd


def layer_norm_backward(dy, h, weight, mean, rstd, dh=None, dropout=0.0, seed=None, sequence=0,
                        need_weight=True, need_bias=True, out=None, stream=None):
    """``(dx, dresidual, dweight, dbias)``: the gradient of ``layer_norm``
    through mt_layer_norm_backward.

    dy: gradient of y; h, mean and rstd: the forward call's; dh: the gradient
    that reaches h directly (the residual stream), added; ``dropout``, ``seed``
    and ``sequence``: the forward call's.  dx and dresidual have dy's dtype and
    are the same tensor without dropout; dweight and dbias are float32 (None
    when not needed).  ``out`` receives dx when given and may be dy or dh."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(layer_norm_backward, stream, dy, h, weight, mean, rstd, dh, dropout,
                         seed, sequence, need_weight, need_bias, out)
    if layers._native is not None and out is None:
        r = layers._native.layer_norm_backward(dy, h, weight, mean, rstd, dh, dropout, seed,
                                               sequence, bool(need_weight), bool(need_bias))
        if r is not None:
            return layers._done(r, "mt_layer_norm_backward")
    rows, d, dt, dev, dyp, lddy = layers._first(dy, "dy", layers._FLOATS)
    p, sp, sequence = _dropped(dropout, seed, sequence, dev)
    f32 = _torch.float32
    hp, ldh = layers._matrix(h, "h", rows, d, dt, dev)
    mp, _ = layers._vector(mean, "mean", rows, (f32,), dev)
    rp, _ = layers._vector(rstd, "rstd", rows, (f32,), dev)
    wp = wcode = dhp = lddh = dresp = lddres = dwp = dbp = 0
    if weight is not None:
        wp, wcode = layers._vector(weight, "weight", d, (dt, f32), dev)
    if dh is not None:
        dhp, lddh = layers._matrix(dh, "dh", rows, d, dt, dev)
    dx, dxp, lddx = layers._result(out, "out", rows, d, dt, dev)
    dres = dx
    if p > 0.0:
        dres, dresp, lddres = layers._result(None, "dresidual", rows, d, dt, dev)
    dweight = dbias = None
    if need_weight:
        dweight = layers._empty(d, dtype=f32, device=dev)
        dwp = dweight.data_ptr()
    if need_bias:
        dbias = layers._empty(d, dtype=f32, device=dev)
        dbp = dbias.data_ptr()
    layers._call("mt_layer_norm_backward",
                 _pack_layer_norm_backward(rows, d, dyp, lddy, hp, ldh, wp, mp, rp, dhp, lddh,
                                           dxp, lddx, dresp, lddres, dwp, dbp, sp, sequence, p,
                                           layers._codes[dt], wcode, 0, 0), dev)
    return dx, dres, dweight, dbias


def dropout(x, p, seed, sequence=0, residual=None, out=None, stream=None):
    """drop(x) + residual through mt_dropout: each element of x is dropped
    with probability ``p``, the others divided by 1 - p.

    x, residual: 2-D CUDA tensors of one dtype (float16, bfloat16 or
    float32), rows may be strided; ``seed`` and ``sequence`` as in
    ``layer_norm``: the same ones drop the same elements of any x of as many
    rows and columns or more, so the gradient of x is
    ``dropout(dy, p, seed, sequence)``.  ``out`` receives the result when given
    and may be x or residual."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(dropout, stream, x, p, seed, sequence, residual, out)
    if layers._native is not None and out is None:
        r = layers._native.dropout(x, p, seed, sequence, residual)
        if r is not None:
            return layers._done(r, "mt_dropout")
    rows, d, dt, dev, xp, ldx = layers._first(x, "x", layers._FLOATS)
    if seed is None:
        raise TypeError("seed must be an int64 CUDA tensor of one value")
    p, sp, sequence = _dropped(p, seed, sequence, dev)
    rp = ldr = 0
    if residual is not None:
        rp, ldr = layers._matrix(residual, "residual", rows, d, dt, dev)
    y, yp, ldy = layers._result(out, "out", rows, d, dt, dev)
    layers._call("mt_dropout",
                 _pack_dropout(rows, d, xp, ldx, rp, ldr, yp, ldy, sp, sequence, p,
                               layers._codes[dt], 0), dev)
    return y


def _head(a, b, target, trans_b):
    """(T, K, V, dtype, device, a, lda, b, ldb, target) of the loss's operands."""
    T, K, dt, dev, ap, lda = layers._first(a, "a", layers._HALVES)
    if not isinstance(b, _torch.Tensor) or b.dim() != 2:
        raise ValueError("b must be a 2-D CUDA tensor")
    V = b.shape[0 if trans_b else 1]
    bp, ldb = layers._matrix(b, "b", *((V, K) if trans_b else (K, V)), dt, dev)
    if not isinstance(target, _torch.Tensor) or target.dtype != _torch.int64 or \
            not target.is_cuda:
        raise TypeError("target must be an int64 CUDA tensor")
    if target.device != dev:
        raise ValueError(f"target is on {target.device}, the other operands on {dev}")
    if target.shape != (T,) or (T > 1 and target.stride() != (1,)):
        raise ValueError(f"target must be a contiguous vector of {T}")
    if T > 0 and V == 0:
        raise ValueError("a loss needs a vocabulary")
    return T, K, V, dt, dev, ap, lda, bp, ldb, target.data_ptr()


def _loss_options(label_smoothing, z_loss):
    s, c = float(label_smoothing), float(z_loss)
    if not 0.0 <= s <= 1.0:
        raise ValueError("label_smoothing must be in [0, 1]")
    if not 0.0 <= c < float("inf"):
        raise ValueError("z_loss must be finite and not negative")
    return s, c


def linear_cross_entropy(a, b, target, trans_b=False, ignore_index=-100, label_smoothing=0.0,
                         z_loss=0.0, stream=None):
    """Softmax cross entropy of the logits a @ op(b), which are never stored,
    through mt_linear_cross_entropy.

    a: T x K hidden states, b: K x V weight of the vocabulary (or V x K with
    ``trans_b``), 2-D CUDA tensors of one 16-bit dtype, rows may be strided;
    target: T int64 values.  Returns ``(loss, lse)``, T float32 values each:
    per token lse - (1 - s) z[target] - s mean(z) + z_loss lse^2 with s =
    ``label_smoothing`` (0 where the target is ``ignore_index``, NaN where it
    is outside the vocabulary otherwise), and the logits' log-sum-exp, which
    ``linear_cross_entropy_backward`` takes."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(linear_cross_entropy, stream, a, b, target, trans_b, ignore_index,
                         label_smoothing, z_loss)
    if layers._native is not None:
        r = layers._native.linear_cross_entropy(a, b, target, bool(trans_b), ignore_index,
                                                label_smoothing, z_loss)
        if r is not None:
            return layers._done(r, "mt_linear_cross_entropy")
    T, K, V, dt, dev, ap, lda, bp, ldb, tp = _head(a, b, target, trans_b)
    s, c = _loss_options(label_smoothing, z_loss)
    loss = layers._empty(T, dtype=_torch.float32, device=dev)
    lse = layers._empty(T, dtype=_torch.float32, device=dev)
    layers._call("mt_linear_cross_entropy",
                 _pack_loss(T, K, V, ap, lda, bp, ldb, tp, loss.data_ptr(), lse.data_ptr(),
                            int(ignore_index), s, c, 1 if trans_b else 0, layers._codes[dt], 0,
                            0), dev)
    return loss, lse


def linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=False, ignore_index=-100,
                                  label_smoothing=0.0, z_loss=0.0, need_a=True, need_b=True,
                                  db_dtype=None, stream=None):
    """``(da, db)``: the gradient of ``linear_cross_entropy``'s loss through
    mt_linear_cross_entropy_backward (None for what is not needed).

    dloss: T float32 values, the gradient of the loss; lse: the forward
    call's; the other arguments as there.  da has a's dtype, db is stored as b
    in ``db_dtype`` (a's, or float32).  The logits are computed again, a piece
    of the vocabulary at a time."""
    if _torch is None:
        _setup()
    if stream is not None:
        return elsewhere(linear_cross_entropy_backward, stream, dloss, a, b, target, lse, trans_b,
                         ignore_index, label_smoothing, z_loss, need_a, need_b, db_dtype)
    if layers._native is not None:
        r = layers._native.linear_cross_entropy_backward(
            dloss, a, b, target, lse, bool(trans_b), ignore_index, label_smoothing, z_loss,
            bool(need_a), bool(need_b), db_dtype)
        if r is not None:
            return layers._done(r, "mt_linear_cross_entropy_backward")
    T, K, V, dt, dev, ap, lda, bp, ldb, tp = _head(a, b, target, trans_b)
    s, c = _loss_options(label_smoothing, z_loss)
    f32 = _torch.float32
    gp, _ = layers._vector(dloss, "dloss", T, (f32,), dev)
    lp, _ = layers._vector(lse, "lse", T, (f32,), dev)
    if db_dtype is None:
        db_dtype = dt
    elif db_dtype != dt and db_dtype != f32:
        raise TypeError("db_dtype must be a's dtype or float32")
    dap = ldda = dbp = lddb = 0
    da = db = None
    if need_a:
        da, dap, ldda = layers._result(None, "da", T, K, dt, dev)
    if need_b:
        db, dbp, lddb = layers._result(None, "db", *((V, K) if trans_b else (K, V)), db_dtype,
                                       dev)
    layers._call("mt_linear_cross_entropy_backward",
                 _pack_loss_backward(T, K, V, gp, ap, lda, bp, ldb, tp, lp, dap, ldda, dbp, lddb,
                                     int(ignore_index), s, c, 1 if trans_b else 0,
                                     layers._codes[dt], layers._codes[db_dtype], 0), dev)
    return da, db
