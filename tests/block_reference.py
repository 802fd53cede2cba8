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
