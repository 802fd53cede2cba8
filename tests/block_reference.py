"""Plain 64-bit definitions of an expert block's operators (matrix products with
their epilogue, the expert layer, the norms around a block) and the error bounds
that fp32 arithmetic allows against them, on the device of their inputs.

U is half a step of fp32 relative to the value; a sum of n terms in any order is
off by at most n U sum|terms|."""
import math

import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_close(got, want, err, what=""):
    """|got - want| <= err plus half a step of got's type, element by element."""
    g, w = got.detach().double(), want.double()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    tol = err + half_step(got.dtype) * (w.abs() + err)
    bad = ~((g - w).abs() <= tol)
    if bool(bad.any()):
        at = bad.reshape(-1).nonzero()[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {g.reshape(-1)[at]}, "
                             f"want {w.reshape(-1)[at]}, allowed {tol.reshape(-1)[at]}")


# -------------------------------------------------------------- activations --
def act(z, kind):
    """(value, slope) in 64 bits, from the formulas."""
    if kind == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if kind == "gelu":
        phi = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    return z, torch.ones_like(z)


def act_error(z, ez, kind):
    """Bounds of value and slope for an argument off by ez, the functions evaluated in fp32.

    The exponential of a rounded product z log2 e is off by a relative 2 |z| U, and 4 U for itself; the argument of Phi is off
    by 2 U |z|, which changes Phi by a relative (z^2 + 1) 2 U in its tail.  |slope| <= 1.13; the slope's own derivative is at
    most 0.8 (gelu), 0.5 (silu)."""
    v, s = act(z, kind)
    a = z.abs().clamp(max=100.0)
    if kind == "relu":
        return ez, torch.zeros_like(z)
    if kind == "gelu":
        phi = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
        bell = z.abs() * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        rel = (4 * a * a + 20) * U
        return 1.13 * ez + rel * v.abs() + 1e-37, 0.8 * ez + rel * (phi + bell) + 1e-37
    if kind == "silu":
        sg = 1 / (1 + torch.exp(-z))
        rel = (2 * a + 12) * U
        return 1.1 * ez + rel * v.abs() + 1e-37, 0.5 * ez + 2 * rel * sg * (1 + z.abs() * (1 - sg)) + 1e-37
    return ez, torch.zeros_like(z)


# ---------------------------------------------------------- matrix products --
def linear(x, w, bias, residual, kind, gated):
    """One run's rows: (y, z) and their error bounds."""
    x, w = x.double(), w.double()
    z, ez = x @ w.t(), (x.shape[1] + 8) * U * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * (z.abs() + bias.double().abs())
    n = w.shape[0] // 2 if gated else w.shape[0]
    v, _ = act(z[:, :n], kind)
    ev, _ = act_error(z[:, :n], ez[:, :n], kind)
    if gated:
        u, eu = z[:, n:], ez[:, n:]
        ev = ev * (u.abs() + eu) + v.abs() * eu
        v = v * u
        ev = ev + 2 * U * v.abs()
    if residual is not None:
        v = v + residual.double()
        ev = ev + U * (v.abs() + residual.double().abs())
    return (v, z), (ev, ez)


def linear_backward(dy, x, w, z, kind, gated):
    """One run's rows: (dx, dweight, dbias) for the given z (None: dz is dy), and their error bounds.  For bf16 tensors dz is
    rounded before its products, unless it is dy itself."""
    dtype = x.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    n = dy.shape[1]
    if kind == "none" and not gated:
        dz, ed = dy, torch.zeros_like(dy)
        rounded = ed
    else:
        z = z.double()
        v, s = act(z[:, :n], kind)
        ev, es = act_error(z[:, :n], torch.zeros_like(z[:, :n]), kind)
        if gated:
            u = z[:, n:]
            dz = torch.cat([dy * u * s, dy * v], 1)
            ed = torch.cat([(dy * u).abs() * (es + 3 * U * s.abs()), dy.abs() * (ev + 2 * U * v.abs())], 1) + 1e-40
        else:
            dz, ed = dy * s, dy.abs() * (es + 2 * U * s.abs()) + 1e-40
        rounded = ed + half_step(dtype) * (dz.abs() + ed)
    rows = x.shape[0]
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    edx = rounded @ w.abs() + (w.shape[0] + 8) * U * (dz.abs() @ w.abs())
    edw = rounded.t() @ x.abs() + (rows + 8) * U * (dz.abs().t() @ x.abs())
    edb = ed.sum(0) + (rows + 16) * U * dz.abs().sum(0)
    return (dx, dw, db), (edx, edw, edb)


# -------------------------------------------------------- the experts' layer --
def layer(x, experts, weights, w_in, w_out, b_in, b_out, residual, kind, gated):
    """All tokens [T, cols] with experts, weights [T, topk] and all experts' weights [E, ...]: (out, error bound).

    Between the products a value is kept in fp32, or for bf16 in two parts: off by half a step of half a step."""
    dtype = x.dtype
    t, k = experts.shape
    out = residual.double().clone() if residual is not None else torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    err, size = torch.zeros_like(out), out.abs()
    kept = half_step(dtype) ** 2 if dtype == torch.bfloat16 else U
    for e in range(w_in.shape[0]):
        hit = experts == e
        tok = hit.any(1).nonzero()[:, 0]
        if tok.numel() == 0:
            continue
        w = torch.where(hit, weights.double(), 0.0).sum(1)[tok][:, None]
        aw = torch.where(hit, weights.double().abs(), 0.0).sum(1)[tok][:, None] * (1 + k * U)
        (h, _), (eh, _) = linear(x[tok], w_in[e], b_in[e] if b_in is not None else None, None, kind, gated)
        eh = aw * eh + (k + 2) * U * aw * h.abs()
        h = h * w
        eh = eh + kept * (h.abs() + eh)
        w2 = w_out[e].double()
        y = h @ w2.t()
        out[tok] += y
        err[tok] += eh @ w2.abs().t()
        mag = h.abs() @ w2.abs().t()
        if b_out is not None:
            out[tok] += w * b_out[e].double()
            mag = mag + aw * b_out[e].double().abs()
        size[tok] += mag
    n = k * (w_out.shape[2] + 2) + 8 + 16
    return out, err + n * U * size


# ------------------------------------------------------ norms around a block --
def _chain(n: int) -> float:
    # a thread adds at most n / 64 terms of a row, the trees over lanes and waves some more
    return n / 64.0 + 24.0


def _norm(v, ev, w, b, eps, rms):
    """(output, mean, rstd) of rows v that are off by ev, and their bounds."""
    c = v.shape[1]
    mean = torch.zeros_like(v[:, :1]) if rms else v.mean(1, keepdim=True)
    em = torch.zeros_like(mean) if rms else (_chain(c) + 2) * U * v.abs().mean(1, keepdim=True) + ev.mean(1, keepdim=True)
    d = v - mean
    ed = em + ev + (0 if rms else U) * d.abs()
    var = d.square().mean(1, keepdim=True)
    evar = (_chain(c) + 4) * U * var + 2 * (ed * d.abs()).mean(1, keepdim=True) + ed.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    er = rstd * (0.5 * evar / (var + eps) * 1.01 + 4 * U) + 1e-30
    n = d * rstd
    en = rstd * ed + d.abs() * er + 2 * U * n.abs()
    out, size = n * w, (n * w).abs()
    if b is not None:
        out, size = out + b, size + b.abs()
    return (out, mean, rstd), (w.abs() * en + 3 * U * size, em, er)


def _d(t):
    return None if t is None else t.double()


def block(z, x, gate, w1, b1, w2, b2, scale, rms, eps):
    """All ranks' rows: dict of h, y, stats -> (value, bound)."""
    z, x, gate, w1, b1, w2, b2 = (_d(t) for t in (z, x, gate, w1, b1, w2, b2))
    none = torch.zeros_like(z[:, :1])
    p, ep, first, efirst = z, torch.zeros_like(z), (none, none), (none, none)
    if w1 is not None:
        (p, *first), (ep, *efirst) = _norm(z, ep, w1, b1, eps, rms)
    f = torch.full_like(z[:1], scale) if gate is None else scale * gate
    h = x + f * p
    eh = f.abs() * ep + 3 * U * (f * p).abs() + U * (x.abs() + (f * p).abs())
    out, second, esecond = dict(h=(h, eh)), (none, none), (none, none)
    if w2 is not None:
        (y, *second), (ey, *esecond) = _norm(h, eh, w2, b2, eps, rms)
        out["y"] = (y, ey)
    out["stats"] = (torch.cat([*first, *second], 1), torch.cat([*efirst, *esecond], 1))
    return out


def _norm_back(g, eg, n, rstd, rms):
    """rstd (g - mean(g) - n mean(g n)) for a gradient that is off by eg, and its bound."""
    c = g.shape[1]
    m1 = torch.zeros_like(g[:, :1]) if rms else g.mean(1, keepdim=True)
    e1 = torch.zeros_like(m1) if rms else eg.mean(1, keepdim=True) + (_chain(c) + 3) * U * g.abs().mean(1, keepdim=True)
    m2 = (g * n).mean(1, keepdim=True)
    e2 = (eg * n.abs()).mean(1, keepdim=True) + (_chain(c) + 8) * U * (g * n).abs().mean(1, keepdim=True)
    out = rstd * (g - m1 - n * m2)
    return out, rstd.abs() * (eg + 4 * U * g.abs() + e1 + 3 * U * m1.abs() + n.abs() * e2 + 8 * U * (n * m2).abs())


def block_backward(dy, dh, z, h, gate, w1, b1, w2, stats, scale, rms):
    """All ranks' rows: dict of dx, dz, dgate (of every row), dpost_weight ... -> (value, bound); shared sums are over all rows."""
    dy, dh, z, h, gate, w1, b1, w2, stats = (_d(t) for t in (dy, dh, z, h, gate, w1, b1, w2, stats))
    m1, r1, m2, r2 = stats.split(1, 1)
    rows, out = stats.shape[0], {}

    def total(name, v, ev):
        out[name] = (v.sum(0), ev.sum(0) + (rows + 24) * U * v.abs().sum(0))

    like = dy if dy is not None else dh
    dx = dh if dh is not None else torch.zeros_like(like)
    ex = torch.zeros_like(dx)
    if w2 is not None:
        n = (h - m2) * r2
        g = dy * w2
        part, epart = _norm_back(g, U * g.abs(), n, r2, rms)
        total("dpre_weight", dy * n, 5 * U * (dy * n).abs())
        total("dpre_bias", dy, torch.zeros_like(dy))
        ex = epart + 2 * U * (dx.abs() + part.abs())
        dx = dx + part
    out["dx"] = (dx, ex)
    f = scale if gate is None else scale * gate
    du = dx * f
    eu = ex * (abs(f) if gate is None else f.abs()) + 3 * U * du.abs()
    if z is None:
        z = torch.zeros_like(dx)
    if w1 is not None:
        n = (z - m1) * r1
        p = n * w1 if b1 is None else n * w1 + b1
        ep = 6 * U * ((n * w1).abs() + (0 if b1 is None else b1.abs()))
        g = du * w1
        out["dz"] = _norm_back(g, eu * w1.abs() + U * g.abs(), n, r1, rms)
        total("dpost_weight", du * n, eu * n.abs() + 5 * U * (du * n).abs())
        total("dpost_bias", du, eu)
    else:
        p, ep = z, torch.zeros_like(z)
        out["dz"] = (du, eu)
    dg = dx * p * scale
    eg = (ex * p.abs() + dx.abs() * ep) * abs(scale) + 5 * U * dg.abs()
    out["dgate"] = (dg, eg)
    total("dgate_sum", dg, eg)
    return out
