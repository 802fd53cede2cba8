"""GPU: matrix products of every rank's rows with bias, activation and residual,
one weight per run of rows, and their gradients, against the 64-bit definition,
with canaries around every written buffer and rows outside the runs left alone."""
import pytest
import torch

import block_reference as ref
from gpu_util import Guarded, note

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def normal(g, dtype, *shape, std=1.0, offset=0):
    """A tensor that starts `offset` elements behind an aligned address."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.empty(offset + n, dtype=dtype, device="cuda")
    buf[offset:] = (torch.randn(n, generator=g, device="cuda") * std).to(dtype)
    return buf[offset:].view(*shape)


class Case:
    """Ranks' rows cut into runs: ends[r] are the runs' ends of rank r, None: one run of all rows, no offsets."""

    def __init__(self, rows, ends, cols, outs, gated, dtype, offset=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.rows, self.cols, self.outs, self.gated, self.dtype, self.at = g, rows, cols, outs, gated, dtype, offset
        self.p, self.wide = len(rows), outs * (2 if gated else 1)
        self.ends = ends
        self.runs = 1 if ends is None else len(ends[0]) - 1
        self.offsets = None if ends is None else [torch.tensor(e, dtype=torch.int32, device="cuda") for e in ends]
        self.x = [self.new(n, cols) for n in rows]
        self.weight = [self.new(self.runs, self.wide, cols, std=cols ** -0.5) for _ in rows]

    def new(self, *shape, std=1.0):
        return normal(self.g, self.dtype, *shape, std=std, offset=self.at)

    def guards(self, sizes):
        return [Guarded(n, self.dtype, offset_elems=self.at).poison() for n in sizes]

    def parts(self, r):
        e = [0, self.rows[r]] if self.ends is None else [min(max(v, 0), self.rows[r]) for v in self.ends[r]]
        return list(zip(e[:-1], e[1:]))

    def untouched(self, r, t):
        """The rows outside the runs hold what they held."""
        inside = torch.zeros(self.rows[r], dtype=torch.bool, device="cuda")
        for lo, hi in self.parts(r):
            inside[lo:hi] = True
        outside = t.reshape(self.rows[r], t.numel() // max(1, self.rows[r]))[~inside].contiguous()
        assert bool((outside.view(torch.uint8) == 0xFF).all()), "a row outside the runs was written"


def check_forward(dt, c, kind, bias, residual, keep):
    bs = [c.new(c.runs, c.wide, std=0.5) for _ in c.rows] if bias else None
    rs = [c.new(n, c.outs) for n in c.rows] if residual else None
    y = c.guards([n * c.outs for n in c.rows])
    pre = c.guards([n * c.wide for n in c.rows]) if keep else None
    weight = c.weight if c.offsets is not None else [w[0] for w in c.weight]
    dt.dt_linear(c.x, weight, [t.t for t in y], bias=bs, residual=rs, pre=[t.t for t in pre] if keep else None, offsets=c.offsets, act=kind,
                 gated=c.gated)
    torch.cuda.synchronize()
    for r in range(c.p):
        y[r].check()
        got = y[r].t.view(c.rows[r], c.outs)
        c.untouched(r, got)
        if keep:
            pre[r].check()
            c.untouched(r, pre[r].t)
        for e, (lo, hi) in enumerate(c.parts(r)):
            want, err = ref.linear(c.x[r][lo:hi], c.weight[r][e], bs[r][e] if bias else None, rs[r][lo:hi] if residual else None, kind, c.gated)
            ref.assert_close(got[lo:hi], want[0], err[0], f"y[{r}] run {e}")
            if keep:
                ref.assert_close(pre[r].t.view(c.rows[r], c.wide)[lo:hi], want[1], err[1], f"pre[{r}] run {e}")


def check_backward(dt, c, kind, dbias):
    need = kind != "none" or c.gated
    pre = [c.new(n, c.wide, std=1.5) for n in c.rows] if need else None
    dy = [c.new(n, c.outs, std=0.1) for n in c.rows]
    dx, dw = c.guards([n * c.cols for n in c.rows]), c.guards([w.numel() for w in c.weight])
    db = c.guards([c.runs * c.wide] * c.p) if dbias else None
    dt.dt_linear_backward(dy, c.x, c.weight, [t.t for t in dx], [t.t for t in dw], pre=pre, dbias=[t.t for t in db] if dbias else None,
                          offsets=c.offsets, act=kind, gated=c.gated)
    torch.cuda.synchronize()
    for r in range(c.p):
        for t in [dx[r], dw[r]] + ([db[r]] if dbias else []):
            t.check()
        got = dx[r].t.view(c.rows[r], c.cols)
        c.untouched(r, got)
        for e, (lo, hi) in enumerate(c.parts(r)):
            want, err = ref.linear_backward(dy[r][lo:hi], c.x[r][lo:hi], c.weight[r][e], pre[r][lo:hi] if need else None, kind, c.gated)
            ref.assert_close(got[lo:hi], want[0], err[0], f"dx[{r}] run {e}")
            ref.assert_close(dw[r].t.view(c.weight[r].shape)[e], want[1], err[1], f"dweight[{r}] run {e}")
            if dbias:
                ref.assert_close(db[r].t.view(c.runs, c.wide)[e], want[2], err[2], f"dbias[{r}] run {e}")


SHAPES = [
    # rows, runs' ends, cols, outs, elements past an aligned start
    ([1], None, 1, 1, 0),
    ([1, 3], None, 8, 5, 0),
    ([5, 0, 2], None, 64, 64, 0),
    ([17, 1], None, 100, 36, 0),
    ([3], None, 1000, 130, 0),
    ([33, 64], None, 129, 65, 0),
    ([70, 20], None, 96, 200, 1),
    ([70], None, 98, 66, 0),
    ([130], None, 258, 300, 2),
    ([12, 9], [[0, 5, 5, 12], [0, 0, 0, 4]], 72, 40, 0),
    ([9, 0], [[2, 3, 7], [0, 0, 0]], 33, 31, 0),
    ([40], [[-3, 16, 40, 99]], 64, 48, 0),
    ([300, 200], [[0, 1, 130, 290], [10, 140, 140, 200]], 136, 264, 0),
    ([300], [[0, 1, 130, 290]], 135, 263, 1),
    ([700], [[0, 450, 700]], 320, 512, 0),
]


@DTYPES
@pytest.mark.parametrize("rows,ends,cols,outs,offset", SHAPES, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_products(dt, rows, ends, cols, outs, offset, gated, dtype):
    note(f"linear rows={rows} ends={ends} cols={cols} outs={outs} offset={offset} gated={gated} {dtype}")
    c = Case(rows, ends, cols, outs, gated, dtype, offset)
    check_forward(dt, c, "silu", True, True, True)
    check_forward(dt, c, "none", False, False, False)
    check_backward(dt, c, "silu", True)
    check_backward(dt, c, "none", True)


@DTYPES
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_activations(dt, kind, gated, dtype):
    note(f"linear act={kind} gated={gated} {dtype}")
    c = Case([40, 25], [[0, 30, 40], [0, 3, 20]], 80, 48, gated, dtype, seed=3)
    for t in c.x:
        t *= 3.0
    check_forward(dt, c, kind, True, False, True)
    check_backward(dt, c, kind, False)


@DTYPES
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_many_tiles(dt, gated, dtype):
    """More tiles than workgroups run at a time, several steps of the summed index round the stages, runs of many sizes."""
    note(f"linear many tiles gated={gated} {dtype}")
    rows = [2600, 1900]
    ends = [[0, 700, 701, 1500, 1500, 2000, 2050, 2300, 2590], [100, 300, 500, 700, 900, 1100, 1300, 1500, 1899]]
    c = Case(rows, ends, 520, 1032 if dtype == torch.bfloat16 else 520, gated, dtype, seed=5)
    check_forward(dt, c, "gelu", True, True, True)
    check_backward(dt, c, "gelu", True)


def test_wide_tiles(dt):
    """The largest tiles of bf16, on whole rows and on rows that end inside 16 bytes."""
    note("linear wide tiles")
    for cols, gated in ((2560, False), (2562, True)):
        c = Case([3000, 2500], [[0, 1400, 2900], [0, 1300, 2500]], cols, 2560, gated, torch.bfloat16, seed=7)
        check_forward(dt, c, "silu", True, False, False)
        check_backward(dt, c, "silu", False)


def test_what_lies_outside_a_run_does_not_matter(dt):
    """Rows outside the runs, and other runs' rows and weights, hold NaN: no sum meets them."""
    note("linear NaN outside")
    for dtype in (torch.bfloat16, torch.float32):
        for cols in (64, 66, 67):
            c = Case([150], [[10, 60, 60, 130]], cols, 72, True, dtype, seed=8)
            nan = float("nan")
            c.x[0][:10] = nan
            c.x[0][130:] = nan
            c.weight[0][1] = nan   # the run without rows
            check_forward(dt, c, "silu", False, False, True)
            pre, dy = c.new(150, c.wide), c.new(150, c.outs)
            for t in (pre, dy):
                t[:10] = nan
                t[130:] = nan
            dx, dw = torch.zeros_like(c.x[0]), torch.zeros_like(c.weight[0])
            dt.dt_linear_backward([dy], c.x, c.weight, [dx], [dw], pre=[pre], offsets=c.offsets, act="silu", gated=True)
            torch.cuda.synchronize()
            assert bool(dx[10:130].isfinite().all()) and bool(dw.isfinite().all()) and bool((dw[1] == 0).all())


def test_infinite_values_stay_in_their_rows(dt):
    note("linear inf")
    for dtype, cols in ((torch.bfloat16, 70), (torch.float32, 65), (torch.bfloat16, 64)):
        c = Case([20], None, cols, 24, False, dtype, seed=9)
        c.x[0][3, 5] = float("inf")
        c.x[0][7] = float("nan")
        y = torch.zeros(20, 24, dtype=dtype, device="cuda")
        dt.dt_linear(c.x, [c.weight[0][0]], [y])
        torch.cuda.synchronize()
        finite = y.isfinite().all(1)
        assert bool(y[7].isnan().all()) and not bool(finite[3]) and int((~finite).sum()) == 2


def test_gradients_against_differences(dt):
    """dL for L = sum(y * dy), by central differences of the 64-bit definition."""
    note("linear gradients by differences")
    for kind, gated in (("gelu", False), ("silu", True), ("relu", False)):
        c = Case([6], [[0, 2, 6]], 9, 5, gated, torch.float32, seed=11)
        b = [c.new(2, c.wide)]
        y, pre = [torch.zeros(6, 5, device="cuda")], [torch.zeros(6, c.wide, device="cuda")]
        dt.dt_linear(c.x, c.weight, y, bias=b, pre=pre, offsets=c.offsets, act=kind, gated=gated)
        dy, dx, dw, db = [c.new(6, 5)], [torch.zeros_like(c.x[0])], [torch.zeros_like(c.weight[0])], [torch.zeros_like(b[0])]
        dt.dt_linear_backward(dy, c.x, c.weight, dx, dw, pre=pre, dbias=db, offsets=c.offsets, act=kind, gated=gated)
        torch.cuda.synchronize()

        def value(x, w, bias):
            total = 0.0
            for e, (lo, hi) in enumerate(c.parts(0)):
                total += float((ref.linear(x[lo:hi], w[e], bias[e], None, kind, gated)[0][0] * dy[0][lo:hi].double()).sum())
            return total

        at, h = [c.x[0].double(), c.weight[0].double(), b[0].double()], 1e-6
        for which, got in enumerate((dx[0], dw[0], db[0])):
            for i in range(0, at[which].numel(), 7):
                up, dn = [t.clone() for t in at], [t.clone() for t in at]
                up[which].view(-1)[i] += h
                dn[which].view(-1)[i] -= h
                # the second differences are O(1) and the kernel's own error is some U of sums of about 10
                assert abs((value(*up) - value(*dn)) / (2 * h) - float(got.view(-1)[i])) < 1e-4


def test_no_rows(dt):
    note("linear without rows")
    e, w = [torch.empty(0, 16, device="cuda")], [torch.ones(3, 8, 16, device="cuda")]
    off = [torch.zeros(4, dtype=torch.int32, device="cuda")]
    assert dt.dt_linear(e, w, [torch.empty(0, 8, device="cuda")], offsets=off)[0].numel() == 0
    dw, db = [torch.full((3, 8, 16), 7.0, device="cuda")], [torch.full((3, 8), 7.0, device="cuda")]
    dt.dt_linear_backward([torch.empty(0, 8, device="cuda")], e, w, e, dw, dbias=db, offsets=off)
    torch.cuda.synchronize()
    assert bool((dw[0] == 0).all()) and bool((db[0] == 0).all())


def test_offsets_of_a_dispatch(dt):
    """The runs as dt_moe_dispatch leaves them: what the experts make of their rows, brought back, is the layer's definition."""
    note("linear between dispatch and combine")
    p, t, e, k, cols, outs = 2, 37, 6, 2, 48, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [normal(g, torch.float32, t, cols) for _ in range(p)]
    experts = [torch.rand(t, e, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32) for _ in range(p)]
    weights = [torch.rand(t, k, generator=g, device="cuda") for _ in range(p)]
    recv, off = [torch.zeros(p * t * k, cols, device="cuda") for _ in range(p)], [torch.zeros(e // p + 1, dtype=torch.int32, device="cuda") for _ in range(p)]
    pos = [torch.zeros(t, k, dtype=torch.int32, device="cuda") for _ in range(p)]
    w = [normal(g, torch.float32, e // p, outs, cols, std=cols ** -0.5) for _ in range(p)]
    y, out = [torch.zeros(p * t * k, outs, device="cuda") for _ in range(p)], [torch.zeros(t, outs, device="cuda") for _ in range(p)]
    dt.dt_moe_dispatch(x, experts, recv, pos, off, e)
    dt.dt_linear(recv, w, y, offsets=off, act="relu")
    dt.dt_moe_combine(y, experts, pos, weights, out, e)
    torch.cuda.synchronize()
    every = torch.cat(w).double()
    for r in range(p):
        want, err = torch.zeros(t, outs, dtype=torch.float64, device="cuda"), torch.zeros(t, outs, dtype=torch.float64, device="cuda")
        for i in range(t):
            for j in range(k):
                v, ev = ref.linear(x[r][i:i + 1], every[experts[r][i, j]], None, None, "relu", False)
                want[i] += float(weights[r][i, j]) * v[0][0]
                err[i] += abs(float(weights[r][i, j])) * (ev[0][0] + 4 * ref.U * v[0][0].abs())
        ref.assert_close(out[r], want, err, f"out[{r}]")


def test_captured_and_replayed_and_on_another_stream(dt):
    note("linear in a graph")
    c = Case([90, 60], [[0, 20, 80], [0, 30, 60]], 64, 40, True, torch.bfloat16, seed=13)
    dy = [c.new(n, 40) for n in c.rows]
    y, pre = [torch.zeros(n, 40, dtype=c.dtype, device="cuda") for n in c.rows], [torch.zeros(n, 80, dtype=c.dtype, device="cuda") for n in c.rows]
    dx, dw = [torch.zeros_like(t) for t in c.x], [torch.zeros_like(t) for t in c.weight]
    db = [torch.zeros(2, 80, dtype=c.dtype, device="cuda") for _ in c.rows]
    ws = torch.empty(dt.dt_linear_backward_workspace(c.rows, 2, 40, "silu", True, True, c.dtype), dtype=torch.uint8, device="cuda")

    def step(**kw):
        dt.dt_linear(c.x, c.weight, y, pre=pre, offsets=c.offsets, act="silu", gated=True, **kw)
        dt.dt_linear_backward(dy, c.x, c.weight, dx, dw, pre=pre, dbias=db, offsets=c.offsets, act="silu", gated=True, workspace=ws, **kw)

    outs = y + pre + dx + dw + db
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    ready = dt.prepare(dt.dt_linear, c.x, c.weight, y, pre=pre, offsets=c.offsets, act="silu", gated=True)
    y[0].zero_()
    ready()
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0])
