"""Measured cases of the feed-forward block's operators.

Five operators, as a transformer's feed-forward block uses them next to the
library's products:

* ``norm``        residual addition and root-mean-square norm, 16-bit output or
                  e4m3 output with one scale per row;
* ``norm_grad``   its gradient;
* ``linear``      product with bias, activation and residual in its epilogue,
                  16-bit inputs;
* ``linear8``     the same product on e4m3 rows with scales;
* ``linear_grad`` the gradient of ``linear``.

With ``own`` true ``run`` calls the library; otherwise it computes the plain
form: elementary torch operations in 32 bits, rounded once at the end.
``exact`` gives the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-5


# --- cases --------------------------------------------------------------------
# norm, norm_grad: rows x d.  linear*: A is m x k, the weight k x n (n x k when
# trans), the output m x n.  pad: elements between the end of one row of the
# activations and the start of the next (rows cut from a wider buffer).
def listed():
    return [
        # One decoded token through a block's norm: nothing but latency.
        dict(name="norm one token", op="norm", rows=1, d=4096, dtype="bf16", out="same",
             residual=True, pad=0),
        # A long prompt whose norm feeds an 8-bit product.
        dict(name="norm e4m3 prompt", op="norm", rows=32768, d=8192, dtype="bf16", out="e4m3",
             residual=True, pad=0),
        # Odd width, no alignment anywhere, fp16 training.
        dict(name="norm grad ragged", op="norm_grad", rows=2053, d=3001, dtype="f16", pad=3,
             carried=True),
        # A training batch's norm gradient, the residual stream's gradient added.
        dict(name="norm grad batch", op="norm_grad", rows=16384, d=8192, dtype="bf16", pad=0,
             carried=True),
        # One decoded token: the weight is read once and little else happens.
        dict(name="linear one token", op="linear", m=1, n=8192, k=4096, dtype="bf16",
             act="silu", bias=True, residual=True, trans=True, save=False, pad=0),
        # A few tokens decoded together; weight stored k x n.
        dict(name="linear few tokens", op="linear", m=24, n=4096, k=8192, dtype="f16",
             act="none", bias=False, residual=True, trans=False, save=False, pad=0),
        # Every edge ragged, rows that no 16-byte access can start on.
        dict(name="linear ragged", op="linear", m=4097, n=3001, k=2053, dtype="f16",
             act="gelu", bias=True, residual=True, trans=False, save=False, pad=0),
        # A training batch's first product: the pre-activation is kept.
        dict(name="linear batch", op="linear", m=8192, n=8192, k=8192, dtype="bf16",
             act="gelu_tanh", bias=True, residual=False, trans=True, save=True, pad=0),
        # 8-bit serving of a few tokens.
        dict(name="linear8 few tokens", op="linear8", m=16, n=8192, k=8192, dtype="bf16",
             act="none", bias=False, residual=True, pad=0),
        # 8-bit serving of a prompt.
        dict(name="linear8 prompt", op="linear8", m=4096, n=8192, k=8192, dtype="bf16",
             act="silu", bias=True, residual=False, pad=0),
        # Small fine-tuning batch.
        dict(name="linear grad small", op="linear_grad", m=512, n=1024, k=1024, dtype="f16",
             act="gelu", trans=False, pad=0),
        # A training batch.
        dict(name="linear grad batch", op="linear_grad", m=8192, n=8192, k=4096, dtype="bf16",
             act="silu", trans=True, pad=0),
    ]


def _log(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]: round, aligned or odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    how = rng.randrange(4)
    if how == 0 and v >= 16:
        v = 1 << (v.bit_length() - 1)
    elif how == 1 and v >= 16:
        v = v // 8 * 8
    elif how == 2:
        v |= 1
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear8", "linear_grad"])
    dtype = rng.choice(["f16", "bf16"])
    pad = rng.choice([0, 0, 3, 8])
    if op in ("norm", "norm_grad"):
        d = _log(rng, 64, 16384)
        most = 32768 * 8192 if op == "norm" else 16384 * 8192
        rows = _log(rng, 1, min(65536, most // d))
        if op == "norm":
            return dict(op=op, rows=rows, d=d, dtype=dtype, out=rng.choice(["same", "e4m3"]),
                        residual=rng.random() < 0.7, pad=pad)
        return dict(op=op, rows=rows, d=d, dtype=dtype, pad=pad, carried=rng.random() < 0.7)
    m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    if op == "linear8":
        m = min(m, 4096)
        return dict(op=op, m=m, n=n, k=k, dtype=dtype, act=act, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, pad=rng.choice([0, 0, 16, 3]))
    trans = rng.random() < 0.5
    if op == "linear":
        return dict(op=op, m=m, n=n, k=k, dtype=dtype, act=act, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, trans=trans, save=rng.random() < 0.3, pad=pad)
    k = min(k, 4096)
    return dict(op=op, m=m, n=n, k=k, dtype=dtype, act=act, trans=trans, pad=pad)


# --- inputs -------------------------------------------------------------------
def _rows(g, rows, cols, pad, dtype, scale=1.0, outliers=False):
    """Normal rows inside a buffer with `pad` more columns; `outliers`: one
    channel in 64 is eight times larger, as hidden states have them."""
    buf = torch.randn(rows, cols + pad, generator=g, device="cuda")
    if outliers:
        buf[:, ::64] *= 8.0
    return (buf * scale).to(dtype)[:, :cols]


def _quantised(g, rows, cols, pad, scale, outliers):
    buf = _rows(g, rows, cols + pad, 0, torch.float32, scale, outliers)
    s = (buf.abs().amax(dim=1) / E4M3_MAX).clamp(min=SCALE_MIN)
    q = (buf / s[:, None]).to(E4M3)
    return q[:, :cols], s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt, pad = case["op"], DTYPES[case["dtype"]], case["pad"]
    s = dict(case)
    if op in ("norm", "norm_grad"):
        rows, d = case["rows"], case["d"]
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        if op == "norm":
            s["x"] = _rows(g, rows, d, pad, dt, 1.0, True)
            s["res"] = _rows(g, rows, d, pad, dt, 2.0, True) if case["residual"] else None
        else:
            s["h"] = _rows(g, rows, d, pad, dt, 2.0, True)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
            s["dy"] = _rows(g, rows, d, pad, dt, 0.5)
            s["dh"] = _rows(g, rows, d, pad, dt, 0.5) if case["carried"] else None
        return s
    m, n, k = case["m"], case["n"], case["k"]
    w = 1.0 / math.sqrt(k)
    if op == "linear8":
        s["a"], s["sa"] = _quantised(g, m, k, pad, 1.0, True)
        s["b"], s["sb"] = _quantised(g, n, k, 0, w, False)
    else:
        s["a"] = _rows(g, m, k, pad, dt, 1.0, op == "linear")
        s["b"] = _rows(g, n, k, 0, dt, w) if case["trans"] else _rows(g, k, n, 0, dt, w)
    if op == "linear_grad":
        s["z"] = _rows(g, m, n, pad, dt) if case["act"] != "none" else None
        s["dy"] = _rows(g, m, n, pad, dt, 0.5)
    else:
        s["bias_v"] = (0.1 * torch.randn(n, generator=g, device="cuda")) if case["bias"] else None
        s["res"] = _rows(g, m, n, pad, dt) if case["residual"] else None
    return s


# --- plain form, 32 bits ------------------------------------------------------
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
        return (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi)
                * (1.0 + 3.0 * 0.044715 * z * z))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain(s):
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op == "norm":
        h = s["x"].float()
        if s["res"] is not None:
            h = h + s["res"].float()
        r = torch.rsqrt(h.square().mean(dim=1) + EPS)
        y = h * r[:, None] * s["weight"].float()
        out = {"rstd": r}
        if s["res"] is not None:
            out["h"] = h.to(dt)
        if s["out"] == "same":
            out["y"] = y.to(dt)
        else:
            sc = torch.clamp(y.abs().amax(dim=1) / E4M3_MAX, min=SCALE_MIN)
            out["scale"] = sc
            out["q"] = (y / sc[:, None]).to(E4M3)
        return out
    if op == "norm_grad":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        xhat = s["h"].float() * r
        gw = dy * s["weight"].float()
        dx = r * (gw - xhat * (gw * xhat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(dim=0)}
    if op == "linear_grad":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), s["act"])
        a, b = s["a"].float(), s["b"].float()
        da = dz @ b if s["trans"] else dz @ b.t()
        db = dz.t() @ a if s["trans"] else a.t() @ dz
        return {"da": da.to(dt), "db": db.to(dt), "dbias": dz.sum(dim=0)}
    if op == "linear8":
        z = (s["a"].float() @ s["b"].float().t()) * s["sa"][:, None] * s["sb"]
    else:
        b = s["b"].float()
        z = s["a"].float() @ (b.t() if s["trans"] else b)
    if s["bias_v"] is not None:
        z = z + s["bias_v"]
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(dt)}
    if s.get("save"):
        out["z"] = z.to(dt)
    return out


# --- the library --------------------------------------------------------------
def _own(s):
    import tiled_fp32_gemm_gb300 as mt
    op = s["op"]
    if op == "norm":
        if s["out"] == "same":
            y, h, rstd = mt.rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS)
            out = {"rstd": rstd, "y": y}
        else:
            q, scale, h, rstd = mt.rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS,
                                            out_dtype=E4M3)
            out = {"rstd": rstd, "q": q, "scale": scale}
        if s["res"] is not None:
            out["h"] = h
        return out
    if op == "norm_grad":
        dx, dweight = mt.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "linear_grad":
        da, db, dbias = mt.linear_backward(s["dy"], s["a"], s["b"], z=s["z"],
                                           activation=s["act"], trans_b=s["trans"])
        return {"da": da, "db": db, "dbias": dbias}
    if op == "linear8":
        return {"y": mt.linear(s["a"], s["b"], bias=s["bias_v"], activation=s["act"],
                               residual=s["res"], trans_b=True, scale_a=s["sa"],
                               scale_b=s["sb"], out_dtype=DTYPES[s["dtype"]])}
    if s["save"]:
        y, z = mt.linear(s["a"], s["b"], bias=s["bias_v"], activation=s["act"],
                         residual=s["res"], trans_b=s["trans"], preact=True)
        return {"y": y, "z": z}
    return {"y": mt.linear(s["a"], s["b"], bias=s["bias_v"], activation=s["act"],
                           residual=s["res"], trans_b=s["trans"])}


def run(state):
    return _own(state) if own else _plain(state)


# --- what a pass cannot do without --------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, d = case["rows"], case["d"]
        e = rows * d
        if op == "norm":
            per = 2 + (4 if case["residual"] else 0) + (2 if case["out"] == "same" else 1)
            extra = 2 * d + 4 * rows + (4 * rows if case["out"] == "e4m3" else 0)
            return {"bytes": e * per + extra, "flops": 6 * e}
        return {"bytes": e * (8 if case["carried"] else 6) + 6 * d + 4 * rows, "flops": 10 * e}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear_grad":
        act = case["act"] != "none"
        return {"bytes": 2 * (m * n * (2 if act else 1) + 2 * m * k + 2 * k * n) + 4 * n,
                "flops": 4 * m * n * k}
    width = 1 if op == "linear8" else 2
    outs = 1 + (1 if case["residual"] else 0) + (1 if case.get("save") else 0)
    small = (4 * n if case["bias"] else 0) + (4 * (m + n) if op == "linear8" else 0)
    return {"bytes": width * (m * k + k * n) + 2 * m * n * outs + small, "flops": 2 * m * n * k}


# --- definition, 64 bits ------------------------------------------------------
def _f64_act(z, act):
    """(activation, derivative)."""
    if act == "relu":
        on = torch.where(z > 0, 1.0, 0.0).double()
        return on * z, on
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2u.
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * c * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "norm":
        h = s["x"].double() + (s["res"].double() if s["res"] is not None else 0.0)
        rms = (torch.einsum("id,id->i", h, h) / h.shape[1] + EPS).sqrt()
        y = h / rms.unsqueeze(1) * s["weight"].double()
        out = {"rstd": 1 / rms}
        if s["res"] is not None:
            out["h"] = h
        if s["out"] == "same":
            out["y"] = y
        else:
            top = y.abs().max(dim=1).values / E4M3_MAX
            out["scale"] = top.clamp(min=SCALE_MIN)
            out["q"] = y / out["scale"].unsqueeze(1)
        return out
    if op == "norm_grad":
        dy, h, w = s["dy"].double(), s["h"].double(), s["weight"].double()
        r = s["rstd"].double().unsqueeze(1)
        dot = torch.einsum("id,id,d->i", dy, h, w).unsqueeze(1)
        dx = r * dy * w - r ** 3 * h * dot / h.shape[1]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("id,id,i->d", dy, h, r[:, 0])}
    if op == "linear_grad":
        dz = s["dy"].double()
        if s["z"] is not None:
            dz = dz * _f64_act(s["z"].double(), s["act"])[1]
        a, b = s["a"].double(), s["b"].double()
        if s["trans"]:
            return {"da": torch.mm(dz, b), "db": torch.mm(dz.t(), a), "dbias": dz.sum(0)}
        return {"da": torch.mm(dz, b.t()), "db": torch.mm(a.t(), dz), "dbias": dz.sum(0)}
    a, b = s["a"].double(), s["b"].double()
    if op == "linear8":
        a, b = a * s["sa"].double().unsqueeze(1), b * s["sb"].double().unsqueeze(1)
    z = torch.mm(a, b.t()) if op == "linear8" or s["trans"] else torch.mm(a, b)
    if s["bias_v"] is not None:
        z = z + s["bias_v"].double()
    y = _f64_act(z, s["act"])[0]
    if s["res"] is not None:
        y = y + s["res"].double()
    out = {"y": y}
    if s.get("save"):
        out["z"] = z
    return out
