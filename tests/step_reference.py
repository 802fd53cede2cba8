"""Plain 64-bit definitions of the model-step operators, and the error bounds
that fp32 arithmetic allows against them.

U is half a step of fp32 relative to the value.  A sum of n fp32 terms whose
longest chain of additions is L is off by at most L * U * sum|terms|; `chain`
below is such an L for the library's kernels (a thread's own run of terms,
then trees over lanes and waves)."""
import math

import torch

U = 2.0 ** -24


def chain(n: int) -> float:
    # the shortest run per thread any kernel uses is n / 64, the trees add at most 6 + 4 steps
    return n / 64.0 + 16.0


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_close(got, want, err, what=""):
    """|got - want| <= err plus half a step of got's type, element by element."""
    g, w = got.detach().double().cpu(), want.double().cpu()
    e = err.double().cpu() if isinstance(err, torch.Tensor) else torch.full_like(w, float(err))
    assert g.shape == w.shape, (what, g.shape, w.shape)
    tol = e + half_step(got.dtype) * (w.abs() + e)
    bad = ~((g - w).abs() <= tol)
    if bool(bad.any()):
        at = bad.reshape(-1).nonzero()[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: got {g.reshape(-1)[at]}, "
                             f"want {w.reshape(-1)[at]}, allowed {tol.reshape(-1)[at]}")


# -------------------------------------------------------------- layer norm --
def norm(x, w, b, eps):
    """x [N, C] -> (y, mean, rstd) and their error bounds."""
    x, w = x.double(), w.double()
    c = x.shape[1]
    mean = x.sum(1, keepdim=True) / c
    d = x - mean
    var = d.square().sum(1, keepdim=True) / c
    rstd = 1.0 / torch.sqrt(var + eps)
    n = d * rstd
    y = n * w + (b.double() if b is not None else 0.0)
    em = (chain(c) + 2) * U * x.abs().mean(1, keepdim=True)
    ed = em + U * d.abs()
    ev = (chain(c) + 4) * U * var + 2 * (ed * d.abs()).mean(1, keepdim=True) + ed.square().mean(1, keepdim=True)
    er = rstd * (0.5 * ev / (var + eps) * 1.01 + 4 * U) + 1e-30
    en = rstd * ed + d.abs() * er + 2 * U * n.abs()
    ey = w.abs() * en + 3 * U * ((n * w).abs() + (b.double().abs() if b is not None else 0.0))
    return (y, mean.reshape(-1), rstd.reshape(-1)), (ey, em.reshape(-1), er.reshape(-1))


def norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) for given statistics, and their error bounds."""
    dy, x, w, mean, rstd = dy.double(), x.double(), w.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, c = x.shape
    n = (x - mean) * rstd
    en = 3 * U * n.abs()
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * n).mean(1, keepdim=True)
    e1 = (chain(c) + 3) * U * g.abs().mean(1, keepdim=True)
    e2 = (chain(c) + 8) * U * (g * n).abs().mean(1, keepdim=True)
    dx = rstd * (g - m1 - n * m2)
    edx = rstd * (4 * U * g.abs() + e1 + 3 * U * m1.abs() + n.abs() * e2 + (en + 4 * U * n.abs()) * m2.abs())
    lw = rows + 16  # any order of the rows' additions
    dw, db = (dy * n).sum(0), dy.sum(0)
    edw = (lw + 6) * U * (dy * n).abs().sum(0)
    edb = lw * U * dy.abs().sum(0)
    return (dx, dw, db), (edx, edw, edb)


# ----------------------------------------------------------------- routing --
def route(x, k, bias=None, groups=1, topk_groups=1, score="softmax", renormalize=True, scale=1.0):
    """One token at a time, in Python: (experts [N, k], weights [N, k], error bound)."""
    x = x.double().cpu()
    bias = None if bias is None else bias.double().cpu()
    n, e = x.shape
    experts, weights = torch.full((n, k), -1, dtype=torch.int64), torch.zeros((n, k), dtype=torch.float64)
    bound = torch.zeros((n, k), dtype=torch.float64)
    biggest = torch.finfo(torch.float32).max
    for t in range(n):
        row = [min(v, biggest) for v in x[t].tolist()]
        finite = [i for i in range(e) if row[i] > -math.inf]  # False for NaN
        live = [i for i in finite if bias is None or bias[i].item() > -math.inf]
        if score == "softmax":
            top = max((row[i] for i in finite), default=0.0)
            z = sum(math.exp(row[i] - top) for i in finite)
            s = {i: math.exp(row[i] - top) / z for i in finite}
        else:
            s = {i: 1.0 / (1.0 + math.exp(-row[i])) if row[i] > -700 else 0.0 for i in finite}
        c = {i: s[i] + (0.0 if bias is None else bias[i].item()) for i in live}
        if groups > 1:
            per = e // groups
            scored = []
            for g in range(groups):
                best = sorted((c[i] for i in live if i // per == g), reverse=True)[:2]
                if best:
                    scored.append((-sum(best), g))
            stay = {g for _, g in sorted(scored)[:topk_groups]}
            live = [i for i in live if i // per in stay]
        key = (lambda i: (-row[i], i)) if bias is None else (lambda i: (-c[i], i))
        chosen = sorted(live, key=key)[:k]
        if not chosen:
            continue
        if renormalize:
            top = max(row[i] for i in chosen)
            w = [s[i] for i in chosen] if score == "sigmoid" and top > -60 else [math.exp(row[i] - top) for i in chosen]
            w = [v / sum(w) for v in w]
        else:
            w = [s[i] for i in chosen]
        spread = max(abs(row[i]) for i in chosen) + max((abs(v) for v in row if abs(v) < 1e30), default=0.0)
        for j, i in enumerate(chosen):
            experts[t, j], weights[t, j] = i, w[j] * scale
            # two exponentials of rounded arguments (4 U each plus the argument's U), a sum of e terms, divisions
            bound[t, j] = (2 * min(spread, 1e4) + chain(e) + 24) * U * abs(w[j] * scale) + 1e-37
    return experts, weights, bound


def route_backward(x, experts, dw, score="softmax", renormalize=True, scale=1.0):
    """By the closed formula in 64 bits: (dx, error bound)."""
    x, g = x.double().cpu(), dw.double().cpu() * scale
    experts = experts.long().cpu()
    n, e = x.shape
    x = torch.where(x > -math.inf, x.clamp(max=torch.finfo(torch.float32).max), torch.tensor(-math.inf, dtype=torch.float64))
    ok = (experts >= 0) & (experts < e)
    at = experts.clamp(0, e - 1)
    xj = torch.where(ok, x.gather(1, at), torch.tensor(-math.inf, dtype=torch.float64))
    ok = xj > -math.inf
    xz = torch.where(ok, xj, 0.0)
    s = torch.softmax(x, 1).nan_to_num(0.0) if score == "softmax" else torch.sigmoid(x)
    sj = torch.where(ok, s.gather(1, at), 0.0)
    if renormalize:
        ln = torch.where(ok, xj if score == "softmax" else -torch.log1p(torch.exp(-xz.clamp(min=-600))), -math.inf)
        w = torch.softmax(ln, 1).nan_to_num(0.0)
        t = w * (g - (g * w).sum(1, keepdim=True))
        size = w * (g.abs() + (g * w).abs().sum(1, keepdim=True))
        f = 1.0 / (1.0 + torch.exp(xz)) if score == "sigmoid" else torch.ones_like(xz)
        t, size = t * f, size * f
        dx = torch.zeros_like(x).scatter_add(1, at, torch.where(ok, t, 0.0))
        mag = torch.zeros_like(x).scatter_add(1, at, torch.where(ok, size, 0.0))
    elif score == "sigmoid":
        t = torch.where(ok, g * sj / (1.0 + torch.exp(xz)), 0.0)
        dx = torch.zeros_like(x).scatter_add(1, at, t)
        mag = torch.zeros_like(x).scatter_add(1, at, t.abs())
    else:
        ds = torch.zeros_like(x).scatter_add(1, at, torch.where(ok, g, 0.0))
        da = torch.zeros_like(x).scatter_add(1, at, torch.where(ok, g.abs(), 0.0))
        dx = s * (ds - (ds * s).sum(1, keepdim=True))
        mag = s * (da + (da * s).sum(1, keepdim=True))
    spread = torch.where(x.abs() < 1e30, x.abs(), 0.0).amax(1, keepdim=True)
    return dx, (4 * spread + 2 * chain(e) + 40) * U * mag + 1e-37


# ---------------------------------------------------------------- exchange --
def plan(experts, nexperts, capacity):
    """positions per rank, offsets per rank, and the (rank, token) of every row of every rank's buffer."""
    p = len(experts)
    per = nexperts // p
    positions = [torch.full(e.shape, -1, dtype=torch.int32) for e in experts]
    offsets, rows = [], []
    for q in range(p):
        off, mine = [0], []
        for ex in range(q * per, (q + 1) * per):
            for r in range(p):
                for t, j in (experts[r].cpu() == ex).nonzero().tolist():
                    if len(mine) < capacity[q]:
                        positions[r][t, j] = len(mine)
                        mine.append((r, t, j))
            off.append(len(mine))
        offsets.append(torch.tensor(off, dtype=torch.int32))
        rows.append(mine)
    return positions, offsets, rows


# -------------------------------------------------------------------- loss --
def loss(hidden, shards, targets, dloss=None, ignore_index=-100):
    """64-bit loss, lse and gradients with the bounds that fp32 sums (and, for
    bf16 inputs, the logits' gradient rounded to bf16) allow."""
    x, w = hidden.double().cpu(), torch.cat([s.double().cpu() for s in shards])
    t = targets.cpu()
    n, v, h = x.shape[0], w.shape[0], x.shape[1]
    use = (t != ignore_index) & (t >= 0) & (t < v)
    at = torch.where(use, t, 0)
    z = x @ w.t()
    ez = (h + 8) * U * (x.abs() @ w.abs().t())  # any order of the h additions
    lse = torch.logsumexp(z, 1)
    spread = (z.amax(1) - z.amin(1)).clamp(max=100.0)
    el = ez.amax(1) + (v / 16.0 + 64 + 2 * spread) * U + 8 * U * lse.abs()
    rows = torch.arange(n)
    out = dict(lse=(lse, el), loss=(torch.where(use, lse - z[rows, at], 0.0),
                                    torch.where(use, el + ez[rows, at] + 4 * U * z[rows, at].abs(), 0.0)))
    if dloss is None:
        return out
    g = torch.where(use, dloss.double().cpu(), 0.0)[:, None]
    p = torch.softmax(z, 1)
    ep = p * (ez + el[:, None] + (8 + 2 * spread[:, None]) * U) * 1.01
    one = torch.zeros_like(p)
    one[rows, at] = 1.0
    d = (p - one) * g
    ed = ep * g.abs() + 4 * U * ((p + one) * g).abs() + 1e-40
    if hidden.dtype == torch.bfloat16:
        ed = ed + half_step(torch.bfloat16) * (d.abs() + ed)
    dx = d @ w
    edx = ed @ w.abs() + (v + 8) * U * (d.abs() @ w.abs())
    dw = d.t() @ x
    edw = ed.t() @ x.abs() + (n + 8) * U * (d.abs().t() @ x.abs())
    sizes = [s.shape[0] for s in shards]
    out.update(dhidden=(dx, edx), dweight=(list(dw.split(sizes)), list(edw.split(sizes))))
    return out
