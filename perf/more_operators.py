"""Cases for timing the operators of an expert block over the ranks of one GPU: matrix products with bias, activation and
residual over runs of rows (the experts' products between dispatch and combine, or a dense layer), the whole expert layer for
a few tokens, and the norms after and before a block with its gate and residual, each in a plain form of elementary torch
operations and as the library's calls.

``own`` chooses which of the two ``run`` computes.  Every rank's tensors are elements of lists, as everywhere in the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}
_EPS = 1e-5


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # A training batch's rows after dispatch: eight ranks of eight experts, the gated first product of their layer.
        dict(name="linear-experts-forward", op="linear", way="forward", dtype="bf16", ranks=8, rows=8192, uneven=False, runs=8, fill=0.8, cols=4096,
             outs=2048, gated=True, act="silu", bias=False, residual=False, keep=True),
        # Its backward pass: both gradients of every expert.
        dict(name="linear-experts-backward", op="linear", way="backward", dtype="bf16", ranks=8, rows=8192, uneven=False, runs=8, fill=0.8, cols=4096,
             outs=2048, gated=True, act="silu", bias=False, residual=False, keep=True),
        # A dense layer's product with bias and gelu over a prompt whose tokens are split over four ranks.
        dict(name="linear-dense-forward", op="linear", way="forward", dtype="bf16", ranks=4, rows=2048, uneven=False, runs=1, fill=1.0, cols=4096,
             outs=11008, gated=False, act="gelu", bias=True, residual=False, keep=False),
        # The product that leaves the block while decoding: four rows per rank, bias and residual, latency and the weight's bytes.
        dict(name="linear-decode", op="linear", way="forward", dtype="bf16", ranks=4, rows=4, uneven=False, runs=1, fill=1.0, cols=4096, outs=4096,
             gated=False, act="none", bias=True, residual=True, keep=False),
        # A small fp32 model with odd widths, ragged ranks and runs: its gradients.
        dict(name="linear-ragged-backward", op="linear", way="backward", dtype="fp32", ranks=3, rows=1403, uneven=True, runs=4, fill=0.9, cols=1001,
             outs=509, gated=False, act="gelu", bias=True, residual=True, keep=True),
        # One token meets two of its layer's 64 experts: latency alone counts.
        dict(name="layer-one-token", op="layer", way="forward", dtype="bf16", ranks=1, rows=1, uneven=False, cols=2048, inner=1024, experts=64, topk=2,
             gated=True, act="silu", bias=False, residual=False),
        # Decoding a batch of 16 tokens per rank: the weights' bytes count.
        dict(name="layer-decode", op="layer", way="forward", dtype="bf16", ranks=8, rows=16, uneven=False, cols=4096, inner=2048, experts=64, topk=4,
             gated=True, act="silu", bias=False, residual=True),
        # A small fp32 layer with biases, odd widths and ragged tokens.
        dict(name="layer-ragged", op="layer", way="forward", dtype="fp32", ranks=3, rows=11, uneven=True, cols=1001, inner=509, experts=12, topk=3,
             gated=False, act="gelu", bias=True, residual=False),
        # Between two blocks over a long batch: both RMS norms with a gate per channel, as in serving a prompt.
        dict(name="block-forward-large", op="block", way="forward", dtype="bf16", ranks=8, rows=4096, uneven=False, cols=8192, rms=True, post=True,
             pre=True, bias=False, gate="channel", scale=1.0),
        # The backward pass in a training step, layer norms with biases, all parameter gradients summed over the ranks.
        dict(name="block-backward", op="block", way="backward", dtype="bf16", ranks=8, rows=4096, uneven=False, cols=4096, rms=False, post=True,
             pre=True, bias=True, gate="channel", scale=0.5),
        # A small fp32 model of odd width, with a gate of its own for every token.
        dict(name="block-ragged-backward", op="block", way="backward", dtype="fp32", ranks=5, rows=403, uneven=True, cols=1001, rms=False, post=True,
             pre=True, bias=True, gate="token", scale=1.0),
        # One token per rank while decoding, no norm after the block: latency alone counts.
        dict(name="block-decode", op="block", way="forward", dtype="bf16", ranks=8, rows=1, uneven=False, cols=4096, rms=True, post=False, pre=True,
             bias=False, gate="none", scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else -(-n // 64) * 64


def draw(rng):
    op = rng.choice(("linear", "linear", "layer", "block"))
    c = dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp32")), ranks=rng.choice((1, 2, 3, 4, 6, 8)), uneven=rng.random() < 0.5)
    if op == "linear":
        c.update(way=rng.choice(("forward", "backward")), cols=_width(rng, 16, 8192), outs=_width(rng, 16, 8192), gated=rng.random() < 0.4,
                 act=rng.choice(("none", "relu", "gelu", "silu")), bias=rng.random() < 0.5)
        if c["act"] == "none":
            c["gated"] = False
        c["runs"] = rng.choice((1, _log(rng, 1, 32), _log(rng, 1, 32)))
        c["runs"] = max(1, min(c["runs"], (1 << 28) // (c["cols"] * c["outs"] * c["ranks"])))
        c["fill"] = 1.0 if c["runs"] == 1 else rng.choice((0.5, 0.8, 1.0))
        most = (1 << (37 if c["dtype"] == "fp32" else 39)) // (c["cols"] * c["outs"] * c["ranks"])
        c["rows"] = _log(rng, 1, max(1, min(8192, most)))
        c.update(residual=rng.random() < 0.5, keep=c["way"] == "backward" or rng.random() < 0.5)
    elif op == "layer":
        c.update(way="forward", cols=_width(rng, 64, 8192), inner=_width(rng, 32, 4096), gated=rng.random() < 0.6, act=rng.choice(("relu", "gelu", "silu")),
                 bias=rng.random() < 0.4, residual=rng.random() < 0.5)
        per = max(1, min(64, (1 << 28) // (c["cols"] * c["inner"] * c["ranks"])))
        c["experts"] = c["ranks"] * _log(rng, 1, per)
        c["topk"] = rng.randint(1, min(8, c["experts"]))
        c["rows"] = _log(rng, 1, max(1, 160 // c["ranks"]))
    else:
        c.update(way=rng.choice(("forward", "backward")), cols=_width(rng, 16, 16384), rms=rng.random() < 0.5, pre=rng.random() < 0.85,
                 gate=rng.choice(("none", "channel", "token")), scale=rng.choice((1.0, 0.5)))
        c["post"] = not c["pre"] or rng.random() < 0.6
        c["bias"] = not c["rms"] and rng.random() < 0.7
        c["rows"] = _log(rng, 1, max(1, min(16384, (1 << 27) // (c["cols"] * c["ranks"]))))
    return c


# ----------------------------------------------------------------- inputs --
def _parts(mean, n, uneven):
    """n counts around a mean: equal, or spread from about half of it to half as much again, from the sizes alone."""
    if not uneven:
        return [mean] * n
    parts = [int(mean * (0.5 + (0.37 * (i + 1) * 2.6180339887) % 1.0)) for i in range(n)]
    return [max(1, parts[0])] + parts[1:]


def _filled(c):
    """Rows of each rank that its runs cover."""
    return [math.ceil(n * c["fill"]) if c["runs"] > 1 else n for n in _parts(c["rows"], c["ranks"], c["uneven"])]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt, p = _DT[c["dtype"]], c["ranks"]
    rows = _parts(c["rows"], p, c["uneven"])

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    def zeros(shapes, dtype=dt):
        return [torch.zeros(s, device="cuda", dtype=dtype) for s in shapes]

    st = dict(case=c)
    if c["op"] == "linear":
        k, n, m = c["cols"], c["outs"], c["outs"] * (2 if c["gated"] else 1)
        st["x"] = [normal(r, k) for r in rows]
        st["weight"] = [torch.stack([normal(m, k, std=k ** -0.5) for _ in range(c["runs"])]) for _ in range(p)]
        st["bias"] = [normal(c["runs"], m, std=0.1) for _ in range(p)] if c["bias"] else None
        st["offsets"] = None
        if c["runs"] > 1:  # some experts are liked more than others
            st["offsets"] = []
            for f in _filled(c):
                share = (torch.randn((c["runs"],), generator=g, device="cuda") * 0.4).exp().double().cumsum(0)
                ends = (share / share[-1:] * f).round().to(torch.int32)
                st["offsets"].append(torch.cat([torch.zeros(1, device="cuda", dtype=torch.int32), ends]))
        if c["way"] == "forward":
            st["residual"] = [normal(r, n) for r in rows] if c["residual"] else None
            st["y"] = zeros([(r, n) for r in rows])
            st["pre"] = zeros([(r, m) for r in rows]) if c["keep"] else None
        else:
            st["pre"] = [normal(r, m) for r in rows] if c["act"] != "none" else None  # what the forward pass kept
            st["dy"] = [normal(r, n, std=1e-2) for r in rows]
            st["dx"], st["dweight"] = zeros([(r, k) for r in rows]), zeros([w.shape for w in st["weight"]])
            st["dbias"] = zeros([(c["runs"], m)] * p) if c["bias"] else None
        return st
    if c["op"] == "layer":
        k, n, m, e = c["cols"], c["inner"], c["inner"] * (2 if c["gated"] else 1), c["experts"]
        st["x"] = [normal(r, k) for r in rows]
        lean = torch.randn((1, e), generator=g, device="cuda") * 0.3
        scores = [torch.randn((r, e), generator=g, device="cuda") + lean for r in rows]
        top = [s.topk(c["topk"], dim=1) for s in scores]
        st["experts"] = [t.indices.to(torch.int32) for t in top]
        st["weights"] = [t.values.softmax(1) for t in top]
        if sum(rows) > 32:  # padded tokens go nowhere
            for x in st["experts"]:
                x[torch.rand((x.shape[0],), generator=g, device="cuda") < 0.02] = -1
        st["w_in"] = [torch.stack([normal(m, k, std=k ** -0.5) for _ in range(e // p)]) for _ in range(p)]
        st["w_out"] = [torch.stack([normal(k, n, std=n ** -0.5) for _ in range(e // p)]) for _ in range(p)]
        st["b_in"] = [normal(e // p, m, std=0.1) for _ in range(p)] if c["bias"] else None
        st["b_out"] = [normal(e // p, k, std=0.1) for _ in range(p)] if c["bias"] else None
        st["residual"] = [normal(r, k) for r in rows] if c["residual"] else None
        st["out"] = zeros([(r, k) for r in rows])
        return st
    h = c["cols"]
    st["z"] = [normal(r, h, std=2.0, mean=0.3) for r in rows]
    for name, there in (("post", c["post"]), ("pre", c["pre"])):
        st[name + "_weight"] = [normal(h, std=0.1, mean=1.0)] * p if there else None
        st[name + "_bias"] = [normal(h, std=0.1)] * p if there and c["bias"] else None
    channel = normal(h, std=0.2, mean=0.5)
    st["gate"] = None if c["gate"] == "none" else [channel] * p if c["gate"] == "channel" else [normal(r, h, std=0.5) for r in rows]
    if c["way"] == "forward":
        st["x"] = [normal(r, h, std=3.0) for r in rows]
        st["h"], st["y"] = zeros([(r, h) for r in rows]), zeros([(r, h) for r in rows]) if c["pre"] else None
        st["stats"] = zeros([(r, 4) for r in rows], torch.float32)
        return st
    st["h"] = [normal(r, h, std=3.0) for r in rows]
    st["stats"] = [torch.cat([*_moments(z.double(), c["rms"]), *_moments(v.double(), c["rms"])], 1).float() for z, v in zip(st["z"], st["h"])]
    st["dy"] = [normal(r, h, std=1e-2) for r in rows] if c["pre"] else None
    st["dh"] = [normal(r, h, std=1e-2) for r in rows]
    st["dz"], st["dx"] = zeros([(r, h) for r in rows]), zeros([(r, h) for r in rows])
    st["dgate"] = None if c["gate"] == "none" else zeros([(h,)] * p) if c["gate"] == "channel" else zeros([(r, h) for r in rows])
    for name in ("post", "pre"):
        st[f"d{name}_weight"] = zeros([(h,)] * p) if c[name] else None
        st[f"d{name}_bias"] = zeros([(h,)] * p) if c[name] and c["bias"] else None
    return st


# ------------------------------------------------------------- plain forms --
def _phi(z):
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, 0.0)
    if kind == "gelu":
        return z * _phi(z)
    if kind == "silu":
        return z / (1.0 + (-z).exp())
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return _phi(z) + z * (-0.5 * z * z).exp() * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "silu":
        s = 1.0 / (1.0 + (-z).exp())
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _runs(st):
    """Every rank's runs as (first row, end)."""
    if st["offsets"] is None:
        return [[(0, x.shape[0])] for x in st["x"]]
    ends = torch.stack(st["offsets"]).tolist()  # the plain products need their sizes on the host
    return [list(zip(e[:-1], e[1:])) for e in ends]


def _plain_linear(st):
    c, n = st["case"], st["case"]["outs"]
    out = {k: [] for k in (("y", "pre") if c["way"] == "forward" else ("dx", "dweight", "dbias"))}
    for q, runs in enumerate(_runs(st)):
        x, ws = st["x"][q].float(), st["weight"][q]
        if c["way"] == "forward":
            y, pre = torch.zeros_like(st["y"][q]), torch.zeros_like(st["pre"][q]) if c["keep"] else None
        else:
            dx, dw = torch.zeros_like(st["dx"][q]), torch.zeros_like(ws)
            db = torch.zeros_like(st["dbias"][q]) if c["bias"] else None
        for e, (lo, hi) in enumerate(runs):
            if lo == hi:
                continue
            w = ws[e].float()
            if c["way"] == "forward":
                z = x[lo:hi] @ w.t()
                if c["bias"]:
                    z = z + st["bias"][q][e].float()
                if c["keep"]:
                    pre[lo:hi] = z.to(pre.dtype)
                a = _act(z[:, :n], c["act"])
                a = a * z[:, n:] if c["gated"] else a
                y[lo:hi] = (a + st["residual"][q][lo:hi].float() if c["residual"] else a).to(y.dtype)
                continue
            dz = st["dy"][q][lo:hi].float()
            if c["act"] != "none":
                z = st["pre"][q][lo:hi].float()
                s = _slope(z[:, :n], c["act"])
                dz = torch.cat([dz * z[:, n:] * s, dz * _act(z[:, :n], c["act"])], 1) if c["gated"] else dz * s
            dx[lo:hi] = (dz @ w).to(dx.dtype)
            dw[e] = (dz.t() @ x[lo:hi]).to(dw.dtype)
            if c["bias"]:
                db[e] = dz.sum(0).to(db.dtype)
        got = dict(y=y, pre=pre) if c["way"] == "forward" else dict(dx=dx, dweight=dw, dbias=db)
        for k, v in got.items():
            out[k].append(v)
    return {k: v for k, v in out.items() if v[0] is not None}


def _plain_layer(st):
    c = st["case"]
    p, n, per, dt = c["ranks"], c["inner"], c["experts"] // c["ranks"], _DT[c["dtype"]]
    rows = [x.shape[0] for x in st["x"]]
    x, ex, wt = torch.cat(st["x"]).float(), torch.cat(st["experts"]).reshape(-1).long(), torch.cat(st["weights"]).reshape(-1)
    key = torch.where(ex >= 0, ex, c["experts"])
    order = key.sort(stable=True).indices
    counts = torch.zeros(c["experts"] + 1, device="cuda", dtype=torch.int64).scatter_add_(0, key, torch.ones_like(key)).tolist()
    out = torch.cat(st["residual"]).float() if c["residual"] else torch.zeros_like(x)
    at = 0
    for e, count in enumerate(counts[:-1]):
        if count == 0:
            continue
        slots = order[at:at + count]
        at += count
        q, i, tok = e // per, e % per, slots // c["topk"]
        z = x[tok] @ st["w_in"][q][i].float().t()
        if c["bias"]:
            z = z + st["b_in"][q][i].float()
        a = _act(z[:, :n], c["act"])
        a = a * z[:, n:] if c["gated"] else a
        y = a @ st["w_out"][q][i].float().t()
        if c["bias"]:
            y = y + st["b_out"][q][i].float()
        out.index_add_(0, tok, y * wt[slots].unsqueeze(1))
    return dict(out=list(out.to(dt).split(rows)))


def _moments(x, rms):
    """(mean, 1 / deviation) of each row; RMS norms take no mean off."""
    mean = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    return mean, ((x - mean).square().mean(1, keepdim=True) + _EPS).rsqrt()


def _plain_block(st):
    c, p, dt = st["case"], st["case"]["ranks"], _DT[st["case"]["dtype"]]
    rows = [z.shape[0] for z in st["z"]]
    z = torch.cat(st["z"]).float()
    vec = {k: st[k][0].float() if st[k] is not None else None for k in ("post_weight", "post_bias", "pre_weight", "pre_bias")}
    gate = None if c["gate"] == "none" else st["gate"][0].float() if c["gate"] == "channel" else torch.cat(st["gate"]).float()
    factor = c["scale"] if gate is None else gate * c["scale"]
    if c["way"] == "forward":
        none = torch.zeros_like(z[:, :1])
        mean, rstd, u = none, none, z
        if c["post"]:
            mean, rstd = _moments(z, c["rms"])
            u = (z - mean) * rstd * vec["post_weight"]
            u = u + vec["post_bias"] if c["bias"] else u
        h = torch.cat(st["x"]).float() + factor * u
        stats = [mean, rstd, none, none]
        out = dict(h=list(h.to(dt).split(rows)))
        if c["pre"]:
            stats[2:] = _moments(h, c["rms"])
            y = (h - stats[2]) * stats[3] * vec["pre_weight"]
            out["y"] = list((y + vec["pre_bias"] if c["bias"] else y).to(dt).split(rows))
        out["stats"] = list(torch.cat(stats, 1).split(rows))
        return out
    m1, r1, m2, r2 = torch.cat(st["stats"]).split(1, dim=1)
    mean = (lambda t: 0.0) if c["rms"] else (lambda t: t.mean(1, keepdim=True))
    dx, out = torch.cat(st["dh"]).float(), {}

    def every_rank(name, total):
        total = total.to(dt)
        out[name] = [total.clone() for _ in range(p)]

    if c["pre"]:
        dy, n = torch.cat(st["dy"]).float(), (torch.cat(st["h"]).float() - m2) * r2
        a = dy * vec["pre_weight"]
        dx = dx + r2 * (a - mean(a) - n * (a * n).mean(1, keepdim=True))
        every_rank("dpre_weight", (dy * n).sum(0))
        if c["bias"]:
            every_rank("dpre_bias", dy.sum(0))
    out["dx"] = list(dx.to(dt).split(rows))
    du, n = dx * factor, z
    u = z
    if c["post"]:
        n = (z - m1) * r1
        u = n * vec["post_weight"] + vec["post_bias"] if c["bias"] else n * vec["post_weight"]
        a = du * vec["post_weight"]
        dz = r1 * (a - mean(a) - n * (a * n).mean(1, keepdim=True))
        every_rank("dpost_weight", (du * n).sum(0))
        if c["bias"]:
            every_rank("dpost_bias", du.sum(0))
    else:
        dz = du
    out["dz"] = list(dz.to(dt).split(rows))
    if gate is not None:
        dgate = dx * u * c["scale"]
        if c["gate"] == "channel":
            every_rank("dgate", dgate.sum(0))
        else:
            out["dgate"] = list(dgate.to(dt).split(rows))
    return out


# ------------------------------------------------------ the library's calls --
def _own_linear(st, dt):
    c = st["case"]
    if c["way"] == "forward":
        dt.dt_linear(st["x"], st["weight"], st["y"], bias=st["bias"], residual=st["residual"], pre=st["pre"], offsets=st["offsets"], act=c["act"],
                     gated=c["gated"])
        return dict(y=st["y"], pre=st["pre"]) if c["keep"] else dict(y=st["y"])
    dt.dt_linear_backward(st["dy"], st["x"], st["weight"], st["dx"], st["dweight"], pre=st["pre"], dbias=st["dbias"], offsets=st["offsets"],
                          act=c["act"], gated=c["gated"])
    out = dict(dx=st["dx"], dweight=st["dweight"])
    if c["bias"]:
        out["dbias"] = st["dbias"]
    return out


def _own_layer(st, dt):
    c = st["case"]
    dt.dt_moe_layer(st["x"], st["experts"], st["weights"], st["w_in"], st["w_out"], st["out"], b_in=st["b_in"], b_out=st["b_out"],
                    residual=st["residual"], act=c["act"], gated=c["gated"])
    return dict(out=st["out"])


def _own_block(st, dt):
    c = st["case"]
    if c["way"] == "forward":
        dt.dt_block_norm(st["z"], st["x"], st["h"], st["y"], gate=st["gate"], scale=c["scale"], post_weight=st["post_weight"], post_bias=st["post_bias"],
                         pre_weight=st["pre_weight"], pre_bias=st["pre_bias"], stats=st["stats"], rms=c["rms"], eps=_EPS)
        return dict(h=st["h"], y=st["y"], stats=st["stats"]) if c["pre"] else dict(h=st["h"], stats=st["stats"])
    dt.dt_block_norm_backward(st["dy"], st["dh"], st["z"], st["h"], st["stats"], st["dz"], st["dx"], gate=st["gate"], scale=c["scale"],
                              post_weight=st["post_weight"], post_bias=st["post_bias"], pre_weight=st["pre_weight"], dgate=st["dgate"],
                              dpost_weight=st["dpost_weight"], dpost_bias=st["dpost_bias"], dpre_weight=st["dpre_weight"],
                              dpre_bias=st["dpre_bias"], rms=c["rms"])
    names = ("dx", "dz", "dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")
    return {k: st[k] for k in names if st[k] is not None}


_PLAIN = dict(linear=_plain_linear, layer=_plain_layer, block=_plain_block)
_OWN = dict(linear=_own_linear, layer=_own_layer, block=_own_block)


def run(state):
    op = state["case"]["op"]
    if own:
        import collective_communication_primitives_amd as dt

        return _OWN[op](state, dt)
    return _PLAIN[op](state)


# -------------------------------------------------------------------- work --
def work(case):
    c, s, p = case, _SIZE[case["dtype"]], case["ranks"]
    if c["op"] == "linear":
        n = sum(_filled(c))
        k, m = c["cols"], c["outs"] * (2 if c["gated"] else 1)
        weights = min(c["runs"] * p, n) * m * k * s  # a run without rows needs no weights
        vec = min(c["runs"] * p, n) * m * s if c["bias"] else 0
        if c["way"] == "forward":
            wide = c["outs"] * (2 if c["residual"] else 1) + (m if c["keep"] else 0)
            return dict(bytes=n * (k + wide) * s + weights + vec, flops=2 * n * m * k)
        wide = 2 * k + c["outs"] + (m if c["act"] != "none" else 0)
        return dict(bytes=n * wide * s + weights + c["runs"] * p * m * (k + (1 if c["bias"] else 0)) * s, flops=4 * n * m * k)
    rows = sum(_parts(c["rows"], p, c["uneven"]))
    if c["op"] == "layer":
        k, n, m, e = c["cols"], c["inner"], c["inner"] * (2 if c["gated"] else 1), c["experts"]
        touched = e * (1.0 - (1.0 - c["topk"] / e) ** rows)  # experts that some token chose, on average
        return dict(bytes=int(touched * (m * k + k * n) * s) + rows * ((3 if c["residual"] else 2) * k * s + 8 * c["topk"]),
                    flops=2 * rows * c["topk"] * (m * k + k * n))
    h = c["cols"]
    vecs = (int(c["post"]) + int(c["pre"])) * (2 if c["bias"] else 1) + (1 if c["gate"] == "channel" else 0)
    token = 1 if c["gate"] == "token" else 0
    if c["way"] == "forward":
        return dict(bytes=(rows * (3 + int(c["pre"]) + token) + vecs) * h * s + 16 * rows, flops=rows * h * (4 + 8 * (int(c["post"]) + int(c["pre"]))))
    wide = 3 + 2 * int(c["pre"]) + 2 * token + (1 if c["post"] or c["gate"] != "none" else 0)  # dh, dz, dx; dy, h; the gate and its gradient; z
    return dict(bytes=(rows * wide + vecs * (1 + p)) * h * s + 16 * rows, flops=rows * h * (4 + 14 * (int(c["post"]) + int(c["pre"]))))


# --------------------------------------------------------------- 64 bits --
_F = torch.nn.functional


def _smooth(z, kind):
    """The activations as the library of functions has them, for 64-bit tensors."""
    return dict(none=lambda t: t, relu=torch.relu, gelu=_F.gelu, silu=_F.silu)[kind](z)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(linear=_exact_linear, layer=_exact_layer, block=_exact_block)[case["op"]](st, st["case"])


def _exact_linear(st, c):
    n, got = c["outs"], {}
    for q in range(c["ranks"]):
        x = st["x"][q].double()
        bounds = [0, x.shape[0]] if st["offsets"] is None else st["offsets"][q].tolist()
        if c["way"] == "forward":
            y, pre = torch.zeros(st["y"][q].shape, device="cuda", dtype=torch.float64), None
            if c["keep"]:
                pre = torch.zeros(st["pre"][q].shape, device="cuda", dtype=torch.float64)
            for e in range(c["runs"]):
                part = slice(bounds[e], bounds[e + 1])
                z = torch.addmm(st["bias"][q][e].double() if c["bias"] else x.new_zeros(()), x[part], st["weight"][q][e].double().t())
                if c["keep"]:
                    pre[part] = z
                y[part] = _smooth(z[:, :n], c["act"]) * (z[:, n:] if c["gated"] else 1.0)
                if c["residual"]:
                    y[part] += st["residual"][q][part].double()
            got.setdefault("y", []).append(y)
            if c["keep"]:
                got.setdefault("pre", []).append(pre)
            continue
        dx, m = torch.zeros_like(x), st["weight"][q].shape[1]
        dw = torch.zeros(st["weight"][q].shape, device="cuda", dtype=torch.float64)
        db = torch.zeros((c["runs"], m), device="cuda", dtype=torch.float64)
        for e in range(c["runs"]):
            part = slice(bounds[e], bounds[e + 1])
            dz = st["dy"][q][part].double()
            if c["act"] != "none":  # by differentiation of the activation
                z = st["pre"][q][part].double().requires_grad_(True)
                a = _smooth(z[:, :n], c["act"]) * (z[:, n:] if c["gated"] else 1.0)
                dz = torch.autograd.grad(a, z, dz)[0]
            dx[part] = torch.mm(dz, st["weight"][q][e].double())
            dw[e] = torch.mm(dz.t().contiguous(), x[part])
            db[e] = torch.ones((1, dz.shape[0]), device="cuda", dtype=torch.float64).mm(dz)[0]
        got.setdefault("dx", []).append(dx)
        got.setdefault("dweight", []).append(dw)
        if c["bias"]:
            got.setdefault("dbias", []).append(db)
    return got


def _exact_layer(st, c):
    per, n, outs = c["experts"] // c["ranks"], c["inner"], []
    for r in range(c["ranks"]):
        x, total = st["x"][r].double(), torch.zeros(st["x"][r].shape, device="cuda", dtype=torch.float64)
        ids = st["experts"][r]
        for e in sorted(set(ids.reshape(-1).tolist()) - {-1}):
            q, i = divmod(e, per)
            hit = ids == e
            t = hit.any(1).nonzero()[:, 0]
            w = torch.where(hit, st["weights"][r].double(), 0.0).sum(1)[t]
            z = torch.mm(x[t], st["w_in"][q][i].double().t().contiguous())
            z = z + st["b_in"][q][i].double() if c["bias"] else z
            a = _smooth(z[:, :n], c["act"]) * (z[:, n:] if c["gated"] else 1.0)
            y = torch.mm(a, st["w_out"][q][i].double().t().contiguous())
            y = y + st["b_out"][q][i].double() if c["bias"] else y
            total[t] += w[:, None] * y
        outs.append(total + st["residual"][r].double() if c["residual"] else total)
    return dict(out=outs)


def _exact_block(st, c):
    p, got = c["ranks"], {}
    d = lambda t: None if t is None else t.double()
    first = lambda name: d(st[name][0]) if st[name] is not None else None
    w1, b1, w2, b2 = first("post_weight"), first("post_bias"), first("pre_weight"), first("pre_bias")
    if c["way"] == "forward":
        got = dict(h=[], stats=[])
        for r in range(p):
            z, stats = d(st["z"][r]), torch.zeros(st["stats"][r].shape, device="cuda", dtype=torch.float64)

            def norm(v, w, b, at):
                if c["rms"]:
                    mean, var = torch.zeros_like(v[:, 0]), torch.linalg.vector_norm(v, dim=1).square() / v.shape[1]
                else:
                    var, mean = torch.var_mean(v, dim=1, unbiased=False)
                stats[:, at], stats[:, at + 1] = mean, 1.0 / torch.sqrt(var + _EPS)
                out = (v - mean[:, None]) / torch.sqrt(var + _EPS)[:, None] * w
                return out if b is None else out + b

            u = norm(z, w1, b1, 0) if c["post"] else z
            if c["gate"] != "none":
                u = u * d(st["gate"][r])
            h = torch.add(d(st["x"][r]), u, alpha=c["scale"])
            got["h"].append(h)
            if c["pre"]:
                got.setdefault("y", []).append(norm(h, w2, b2, 2))
            got["stats"].append(stats)
        return got
    sums = {}

    def add(name, value):
        sums[name] = sums[name] + value if name in sums else value

    ones = lambda t: torch.ones((1, t.shape[0]), device="cuda", dtype=torch.float64)
    for r in range(p):
        z, dx = d(st["z"][r]), d(st["dh"][r]).clone()
        m1, r1, m2, r2 = (d(st["stats"][r][:, i:i + 1]) for i in range(4))

        def back(n, a, rstd):
            off = 0.0 if c["rms"] else torch.einsum("ij->i", a)[:, None] / n.shape[1]
            return rstd * (a - off - n * (torch.einsum("ij,ij->i", a, n)[:, None] / n.shape[1]))

        if c["pre"]:
            dy, n = d(st["dy"][r]), (d(st["h"][r]) - m2) * r2
            dx += back(n, dy * w2, r2)
            add("dpre_weight", torch.einsum("ij,ij->j", dy, n))
            add("dpre_bias", ones(dy).mm(dy)[0])
        got.setdefault("dx", []).append(dx)
        f = d(st["gate"][r]) if c["gate"] != "none" else 1.0
        du = dx * (c["scale"] * f)
        n = (z - m1) * r1 if c["post"] else z
        u = n if not c["post"] else n * w1 + (b1 if c["bias"] else 0.0)
        if c["gate"] == "channel":
            add("dgate", torch.einsum("ij,ij->j", dx, u) * c["scale"])
        elif c["gate"] == "token":
            got.setdefault("dgate", []).append(dx * u * c["scale"])
        if c["post"]:
            add("dpost_weight", torch.einsum("ij,ij->j", du, n))
            add("dpost_bias", ones(du).mm(du)[0])
            du = back(n, du * w1, r1)
        got.setdefault("dz", []).append(du)
    for k, v in sums.items():
        if c["bias"] or not k.endswith("bias"):
            got[k] = [v] * p
    return got
