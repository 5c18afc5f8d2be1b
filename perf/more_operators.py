"""Measured cases of the operators that join a transformer block's residual
stream in training, and of the loss that ends a model.

Five operators:

* ``norm``       layer norm of residual + dropout(x) (either may be missing);
* ``norm_grad``  its gradient;
* ``dropout``    dropout alone, with or without a residual's addition; its mask
                 comes from a counter-based generator and is never stored;
* ``loss``       softmax cross entropy of a product with the vocabulary's
                 weight, whose logits are never stored;
* ``loss_grad``  its gradient.

With ``own`` true ``run`` calls the library; otherwise it computes the plain
form: elementary torch operations in 32 bits, rounded once at the end.
``exact`` gives the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
IGNORED = -100
LARGEST_NORM = 16384 * 8192
LARGEST_NORM_GRAD = 16384 * 4096
LARGEST_LOSS = 8192 * 4096 * 131072
LARGEST_LOSS_GRAD = 4096 * 4096 * 131072


# --- cases --------------------------------------------------------------------
# norm, norm_grad, dropout: rows x d, p the probability to drop.  pad: elements
# between the end of one row and the start of the next (rows cut from a wider
# buffer).  loss, loss_grad: `tokens` hidden states of d values, the weight
# vocab x d (d x vocab without trans); smooth: label smoothing; z_loss: factor
# of lse^2; ignored: share of tokens without a target.
def listed():
    return [
        # One decoded token through a block's norm: nothing but latency.
        dict(name="norm one token", op="norm", rows=1, d=4096, dtype="bf16", residual=True,
             p=0.0, pad=0),
        # A training batch joining the residual stream, with dropout.
        dict(name="norm batch", op="norm", rows=16384, d=8192, dtype="bf16", residual=True,
             p=0.1, pad=0),
        # Odd width, no alignment anywhere, fp16 training.
        dict(name="norm grad ragged", op="norm_grad", rows=2053, d=3001, dtype="f16", pad=3,
             carried=True, p=0.0),
        # A training batch's norm gradient, the residual stream's gradient added.
        dict(name="norm grad batch", op="norm_grad", rows=16384, d=4096, dtype="bf16", pad=0,
             carried=True, p=0.1),
        # Dropout of a small fine-tuning batch's odd rows.
        dict(name="dropout small", op="dropout", rows=37, d=1001, dtype="f16", residual=False,
             p=0.25, pad=0),
        # Dropout of a training batch on its way into the residual stream.
        dict(name="dropout batch", op="dropout", rows=16384, d=8192, dtype="bf16",
             residual=True, p=0.1, pad=0),
        # One token scored: the vocabulary's weight is read once.
        dict(name="loss one token", op="loss", tokens=1, d=4096, vocab=131072, dtype="bf16",
             trans=True, smooth=0.0, z_loss=0.0, ignored=0.0, pad=0),
        # Every edge ragged, weight stored d x vocab, smoothed targets.
        dict(name="loss ragged", op="loss", tokens=2047, d=1001, vocab=32003, dtype="f16",
             trans=False, smooth=0.1, z_loss=1e-4, ignored=0.2, pad=0),
        # A training batch.
        dict(name="loss batch", op="loss", tokens=8192, d=4096, vocab=131072, dtype="bf16",
             trans=True, smooth=0.0, z_loss=0.0, ignored=0.05, pad=0),
        # Small fine-tuning batch.
        dict(name="loss grad small", op="loss_grad", tokens=256, d=1024, vocab=8192,
             dtype="bf16", trans=True, smooth=0.0, z_loss=0.0, ignored=0.1, pad=0),
        # Every edge ragged, weight stored d x vocab, fp16 with a scaled loss.
        dict(name="loss grad ragged", op="loss_grad", tokens=1021, d=2049, vocab=32003,
             dtype="f16", trans=False, smooth=0.1, z_loss=1e-4, ignored=0.2, pad=0),
        # A training batch.
        dict(name="loss grad batch", op="loss_grad", tokens=4096, d=4096, vocab=131072,
             dtype="bf16", trans=True, smooth=0.0, z_loss=0.0, ignored=0.05, pad=0),
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
    op = rng.choice(["norm", "norm_grad", "dropout", "loss", "loss_grad"])
    if op in ("norm", "norm_grad", "dropout"):
        d = _log(rng, 64, 16384)
        most = LARGEST_NORM_GRAD if op == "norm_grad" else LARGEST_NORM
        dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
        if dtype == "f32":
            most //= 2
        rows = _log(rng, 1, min(65536, most // d))
        case = dict(op=op, rows=rows, d=d, dtype=dtype, pad=rng.choice([0, 0, 3, 8]),
                    p=rng.choice([0.0, 0.1, 0.1, 0.25, 0.5]))
        if op == "dropout":
            case["p"] = case["p"] or 0.2
        case["carried" if op == "norm_grad" else "residual"] = rng.random() < 0.7
        return case
    d, vocab = _log(rng, 64, 8192), _log(rng, 256, 131072)
    most = LARGEST_LOSS if op == "loss" else LARGEST_LOSS_GRAD
    tokens = _log(rng, 1, min(8192, most // (d * vocab)))
    return dict(op=op, tokens=tokens, d=d, vocab=vocab, dtype=rng.choice(["f16", "bf16"]),
                trans=rng.random() < 0.6, smooth=rng.choice([0.0, 0.0, 0.1]),
                z_loss=rng.choice([0.0, 0.0, 1e-4]), ignored=rng.choice([0.0, 0.1, 0.5]),
                pad=rng.choice([0, 0, 3, 8]))


# --- inputs -------------------------------------------------------------------
def _rows(g, rows, cols, pad, dtype, scale=1.0, outliers=False):
    """Normal rows inside a buffer with `pad` more columns; `outliers`: one
    channel in 64 is eight times larger, as hidden states have them."""
    buf = torch.randn(rows, cols + pad, generator=g, device="cuda")
    if outliers:
        buf[:, ::64] *= 8.0
    return (buf * scale).to(dtype)[:, :cols]


def _lse(a, b, trans):
    """Log-sum-exp of the rows of a @ op(b), a block of tokens at a time."""
    w = b.float().t() if trans else b.float()
    return torch.cat([torch.logsumexp(x.float() @ w, dim=1) for x in a.split(1024)])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt, pad = case["op"], DTYPES[case["dtype"]], case["pad"]
    s = dict(case)
    if op in ("norm", "norm_grad", "dropout"):
        rows, d = case["rows"], case["d"]
        s["seed"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (1,), generator=g, device="cuda",
                                  dtype=torch.int64)
        s["sequence"] = seed % 1000 + 2 ** 32 * (seed % 7)
        if op == "dropout":
            s["x"] = _rows(g, rows, d, pad, dt, 1.0, True)
            s["res"] = _rows(g, rows, d, pad, dt, 2.0, True) if case["residual"] else None
            return s
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
        if op == "norm":
            s["bias"] = (0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)
            s["x"] = _rows(g, rows, d, pad, dt, 1.0, True)
            s["res"] = _rows(g, rows, d, pad, dt, 2.0, True) if case["residual"] else None
        else:
            s["h"] = _rows(g, rows, d, pad, dt, 2.0, True)
            h = s["h"].float()
            s["mean"] = h.mean(dim=1)
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(dim=1) + EPS)
            s["dy"] = _rows(g, rows, d, pad, dt, 0.5)
            s["dh"] = _rows(g, rows, d, pad, dt, 0.5) if case["carried"] else None
        return s
    n, d, vocab = case["tokens"], case["d"], case["vocab"]
    w = 1.5 / math.sqrt(d)
    s["a"] = _rows(g, n, d, pad, dt)
    s["b"] = _rows(g, vocab, d, 0, dt, w) if case["trans"] else _rows(g, d, vocab, 0, dt, w)
    # Frequent tokens first, as vocabularies are sorted.
    u = torch.rand(n, generator=g, device="cuda")
    s["target"] = (u * u * vocab).long().clamp(max=vocab - 1)
    if case["ignored"]:
        drop = torch.rand(n, generator=g, device="cuda") < case["ignored"]
        s["target"] = torch.where(drop, torch.full_like(s["target"], IGNORED), s["target"])
    if op == "loss_grad":
        s["lse"] = _lse(s["a"], s["b"], case["trans"])
        # The mean over the tokens, some weighted more; fp16 training scales
        # its loss.
        share = (16384.0 if case["dtype"] == "f16" else 1.0) / n
        s["dloss"] = share * (0.5 + torch.rand(n, generator=g, device="cuda"))
    return s


# --- plain form, 32 bits ------------------------------------------------------
_M32 = 0xFFFFFFFF


def _mul_hi_lo(a, m):
    """Upper and lower 32 bits of a * m for 32-bit values in 64-bit integers
    (a product past 2^63 wraps, and its bits are right)."""
    t = a * m
    return (t >> 32) & _M32, t & _M32


def _random_words(rows, d, seed, sequence):
    """rows x d 32-bit words of Philox4x32-10: key = seed, counter =
    (column / 4, row, sequence), word column % 4."""
    at = torch.arange((d + 3) // 4, device="cuda")
    row = torch.arange(rows, device="cuda")
    c0 = at[None, :].expand(rows, -1)
    c1 = row[:, None].expand(-1, at.numel())
    c2 = torch.full_like(c0, sequence & _M32)
    c3 = torch.full_like(c0, (sequence >> 32) & _M32)
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    return torch.stack([c0, c1, c2, c3], dim=2).reshape(rows, -1)[:, :d]


def _drop(x, s):
    """Dropout of fp32 values."""
    if s["p"] == 0.0:
        return x
    kept = _random_words(s["rows"], s["d"], s["seed"], s["sequence"]) >= int(s["p"] * 2.0 ** 32)
    return torch.where(kept, x * (1.0 / (1.0 - s["p"])), torch.zeros_like(x))


def _logits(s):
    b = s["b"].float()
    return s["a"].float() @ (b.t() if s["trans"] else b)


def _plain(s):
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op in ("norm", "dropout"):
        h = _drop(s["x"].float(), s)
        if s["res"] is not None:
            h = h + s["res"].float()
        if op == "dropout":
            return {"y": h.to(dt)}
        mean = h.mean(dim=1)
        c = h - mean[:, None]
        r = torch.rsqrt(c.square().mean(dim=1) + EPS)
        out = {"y": (c * r[:, None] * s["weight"].float() + s["bias"].float()).to(dt),
               "mean": mean, "rstd": r}
        if s["res"] is not None or s["p"] > 0.0:
            out["h"] = h.to(dt)
        return out
    if op == "norm_grad":
        dy, r = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["h"].float() - s["mean"][:, None]) * r
        g = dy * s["weight"].float()
        dres = r * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dres = dres + s["dh"].float()
        out = {"dx": _drop(dres, s).to(dt), "dweight": (dy * xhat).sum(dim=0),
               "dbias": dy.sum(dim=0)}
        if s["p"] > 0.0:
            out["dresidual"] = dres.to(dt)
        return out
    live = s["target"] != IGNORED
    target = torch.where(live, s["target"], 0)
    z = _logits(s)
    if op == "loss":
        top = z.amax(dim=1)
        lse = top + (z - top[:, None]).exp().sum(dim=1).log()
        loss = lse - (1.0 - s["smooth"]) * z.gather(1, target[:, None])[:, 0]
        if s["smooth"]:
            loss = loss - s["smooth"] * z.mean(dim=1)
        if s["z_loss"]:
            loss = loss + s["z_loss"] * lse.square()
        return {"loss": torch.where(live, loss, 0.0), "lse": lse}
    lse = s["lse"]
    grad = (z - lse[:, None]).exp_()
    if s["z_loss"]:
        grad *= (1.0 + 2.0 * s["z_loss"] * lse)[:, None]
    if s["smooth"]:
        grad -= s["smooth"] / s["vocab"]
    grad.scatter_add_(1, target[:, None], torch.full_like(lse, s["smooth"] - 1.0)[:, None])
    grad *= torch.where(live, s["dloss"], 0.0)[:, None]
    a, b = s["a"].float(), s["b"].float()
    da = grad @ b if s["trans"] else grad @ b.t()
    db = grad.t() @ a if s["trans"] else a.t() @ grad
    return {"da": da.to(dt), "db": db.to(dt)}


# --- the library --------------------------------------------------------------
def _own(s):
    import tiled_fp32_gemm_gb300 as mt
    op = s["op"]
    if op == "dropout":
        return {"y": mt.dropout(s["x"], s["p"], s["seed"], sequence=s["sequence"],
                                residual=s["res"])}
    if op == "norm":
        y, h, mean, rstd = mt.layer_norm(s["x"], s["weight"], s["bias"], residual=s["res"],
                                         eps=EPS, dropout=s["p"], seed=s["seed"],
                                         sequence=s["sequence"])
        out = {"y": y, "mean": mean, "rstd": rstd}
        if s["res"] is not None or s["p"] > 0.0:
            out["h"] = h
        return out
    if op == "norm_grad":
        dx, dres, dweight, dbias = mt.layer_norm_backward(
            s["dy"], s["h"], s["weight"], s["mean"], s["rstd"], dh=s["dh"], dropout=s["p"],
            seed=s["seed"], sequence=s["sequence"])
        out = {"dx": dx, "dweight": dweight, "dbias": dbias}
        if s["p"] > 0.0:
            out["dresidual"] = dres
        return out
    if op == "loss":
        loss, lse = mt.linear_cross_entropy(s["a"], s["b"], s["target"], trans_b=s["trans"],
                                            ignore_index=IGNORED, label_smoothing=s["smooth"],
                                            z_loss=s["z_loss"])
        return {"loss": loss, "lse": lse}
    da, db = mt.linear_cross_entropy_backward(s["dloss"], s["a"], s["b"], s["target"], s["lse"],
                                              trans_b=s["trans"], ignore_index=IGNORED,
                                              label_smoothing=s["smooth"], z_loss=s["z_loss"])
    return {"da": da, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


# --- what a pass cannot do without --------------------------------------------
def work(case):
    op = case["op"]
    width = 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_grad", "dropout"):
        rows, d = case["rows"], case["d"]
        e = rows * d
        if op == "dropout":
            return {"bytes": width * e * (3 if case["residual"] else 2), "flops": 2 * e}
        if op == "norm":
            moved = 2 + (1 if case["residual"] else 0) + (
                1 if case["residual"] or case["p"] > 0.0 else 0)
            return {"bytes": width * (e * moved + 2 * d) + 8 * rows, "flops": 8 * e}
        moved = 3 + (1 if case["carried"] else 0) + (1 if case["p"] > 0.0 else 0)
        return {"bytes": width * (e * moved + d) + 8 * d + 8 * rows, "flops": 14 * e}
    n, d, vocab = case["tokens"], case["d"], case["vocab"]
    if op == "loss":
        return {"bytes": 2 * (n * d + vocab * d) + 16 * n, "flops": 2 * n * d * vocab}
    return {"bytes": 4 * (n * d + vocab * d) + 16 * n, "flops": 6 * n * d * vocab}


# --- definition, 64 bits ------------------------------------------------------
def _mul32(a, b):
    """(upper, lower) words of a product of 32-bit words, in 16-bit digits."""
    a0, a1, b0, b1 = a % 65536, a // 65536, b % 65536, b // 65536
    low, mid1, mid2, high = a0 * b0, a1 * b0, a0 * b1, a1 * b1
    mid = low // 65536 + mid1 % 65536 + mid2 % 65536
    return high + mid1 // 65536 + mid2 // 65536 + mid // 65536, low % 65536 + mid % 65536 * 65536


def _kept(case, seed, sequence):
    """The mask, a column of every group of four at a time."""
    rows, d = case["rows"], case["d"]
    groups = (d + 3) // 4
    key = int(seed.item()) % 2 ** 64
    key = [key % 2 ** 32, key // 2 ** 32]
    n = torch.arange(rows * groups, device="cuda")
    ctr = [n % groups, n // groups, torch.zeros_like(n) + sequence % 2 ** 32,
           torch.zeros_like(n) + sequence // 2 ** 32]
    for turn in range(10):
        up0, down0 = _mul32(ctr[0], 0xD2511F53)
        up2, down2 = _mul32(ctr[2], 0xCD9E8D57)
        ctr = [up2.bitwise_xor(ctr[1]).bitwise_xor((key[0] + turn * 0x9E3779B9) % 2 ** 32), down2,
               up0.bitwise_xor(ctr[3]).bitwise_xor((key[1] + turn * 0xBB67AE85) % 2 ** 32), down0]
    border = math.floor(case["p"] * 2 ** 32)
    mask = torch.empty(rows, 4 * groups, dtype=torch.bool, device="cuda")
    for k in range(4):
        mask[:, k::4] = (ctr[k] >= border).view(rows, groups)
    return mask[:, :d]


def _f64_dropped(v, case, s):
    if not case["p"]:
        return v
    return v * _kept(case, s["seed"], s["sequence"]) / (1.0 - case["p"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "dropout"):
        h = _f64_dropped(s["x"].double(), case, s)
        if s["res"] is not None:
            h = h + s["res"].double()
        if op == "dropout":
            return {"y": h}
        var, mean = torch.var_mean(h, dim=1, correction=0)
        std = (var + EPS).sqrt()
        y = torch.addcmul(s["bias"].double(), (h - mean.unsqueeze(1)) / std.unsqueeze(1),
                          s["weight"].double())
        out = {"y": y, "mean": mean, "rstd": 1 / std}
        if s["res"] is not None or case["p"]:
            out["h"] = h
        return out
    if op == "norm_grad":
        dy, w, r = s["dy"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
        c = s["h"].double() - s["mean"].double().unsqueeze(1)
        d = case["d"]
        along = torch.einsum("id,id,d->i", dy, c, w).unsqueeze(1)
        dres = r * dy * w - (r / d) * (dy @ w).unsqueeze(1) - (r ** 3 / d) * along * c
        if s["dh"] is not None:
            dres = dres + s["dh"].double()
        out = {"dx": _f64_dropped(dres, case, s), "dweight": torch.einsum("id,id->d", dy, c * r),
               "dbias": dy.sum(0)}
        if case["p"]:
            out["dresidual"] = dres
        return out
    # Blocks of tokens: a training batch's logits in 64 bits fill memory.
    w = s["b"].double()
    w = w.t() if case["trans"] else w  # d x vocab
    vocab, smooth, zl = case["vocab"], case["smooth"], case["z_loss"]
    parts, db = [], torch.zeros_like(w) if op == "loss_grad" else None
    for at in range(0, case["tokens"], 1024):
        a, t = s["a"][at:at + 1024].double(), s["target"][at:at + 1024]
        live, z = t.ne(IGNORED), torch.mm(a, w)
        hot = torch.arange(len(t), device="cuda"), t.clamp(min=0)
        if op == "loss":
            lse = torch.logsumexp(z, 1)
            nll = -((1 - smooth) * z[hot] + smooth * z.mean(1)) + lse + zl * lse ** 2
            parts.append((nll * live, lse))
            continue
        lse = s["lse"][at:at + 1024].double().unsqueeze(1)
        z.sub_(lse).exp_().mul_(1 + 2 * zl * lse).sub_(smooth / vocab)
        z[hot] -= 1 - smooth
        z.mul_((s["dloss"][at:at + 1024].double() * live).unsqueeze(1))
        parts.append((torch.mm(z, w.t()),))
        db.addmm_(a.t(), z)
    if op == "loss":
        return {"loss": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}
    return {"da": torch.cat([p[0] for p in parts]), "db": db.t() if case["trans"] else db}
