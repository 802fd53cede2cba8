"""GPU: an expert block's operators where its calls are unusual (few rows of many
runs, buffers far larger than their runs, rows whose elements pass 32 bits, two
calls at once) and together, as a training step and a decoding step use them,
against 64-bit arithmetic."""
import pytest
import torch

import block_reference as ref
from gpu_util import Guarded, note
from test_gpu_block import Block
from test_gpu_layer import Layer
from test_gpu_linear import DTYPES, Case, check_backward, check_forward, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def ends_of(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------ few rows of a run --
FEW = {
    # runs' rows of each rank, cols, outs
    "one row of each": ([[1] * 8], 520, 200),
    "some without": ([[0, 3, 0, 16], [17, 0, 1, 2]], 264, 48),
    "all rows in one run of many": ([[0] * 20 + [150] + [0] * 11], 136, 72),
    "32 and 33 rows": ([[32, 33, 31]], 1032, 96),
    "about 48 rows": ([[48, 50, 47, 47]], 300, 130),
    "more features than one wave of workgroups": ([[5, 2, 9, 7]], 72, 2200),
    "a long summed index": ([[2, 1]], 9000, 20),
    "odd rows": ([[3, 12]], 77, 33),
}


@DTYPES
@pytest.mark.parametrize("which", FEW, ids=lambda k: k.replace(" ", "_"))
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_few_rows(dt, which, gated, dtype):
    note(f"few rows: {which} gated={gated} {dtype}")
    counts, cols, outs = FEW[which]
    c = Case([sum(n) for n in counts], [ends_of(n) for n in counts], cols, outs, gated, dtype, seed=21)
    check_forward(dt, c, "gelu", True, True, True)
    check_backward(dt, c, "gelu", True)


@DTYPES
def test_as_many_runs_as_there_may_be(dt, dtype):
    """1024 runs over all ranks, many of them empty, the last ones among those with rows."""
    note(f"1024 runs {dtype}")
    for per in (1, 60):
        counts = [[per * ((r * 37 + e * 11) % 3) for e in range(256)] for r in range(4)]
        c = Case([sum(n) + 5 for n in counts], [ends_of(n) for n in counts], 40, 24, True, dtype, seed=22)
        check_forward(dt, c, "silu", True, False, True)
        check_backward(dt, c, "silu", True)


@DTYPES
def test_buffers_larger_than_their_runs(dt, dtype):
    """As behind a dispatch: room for every slot of every rank, few rows in use; and runs that fill the buffers' end alone."""
    note(f"capacity {dtype}")
    for ends in ([0, 3, 3, 40, 41], [39000, 39003, 39500, 39999, 40000]):
        c = Case([40000], [ends], 72, 40, True, dtype, seed=23)
        check_forward(dt, c, "silu", True, True, True)
        check_backward(dt, c, "silu", True)


@DTYPES
def test_decreasing_offsets_stay_inside_the_buffers(dt, dtype):
    """They are not allowed, and their rows' values are anyone's: but nothing outside the buffers and the workspace is written."""
    note(f"decreasing offsets {dtype}")
    rows, runs, cols, outs = 200, 8, 64, 48
    g = torch.Generator(device="cuda").manual_seed(39)
    x, dy, w = (normal(g, dtype, *s) for s in ((rows, cols), (rows, outs), (runs, outs, cols)))
    off = [torch.tensor([0, 200, 0, 200, -5, 900, 0, 150, 20], dtype=torch.int32, device="cuda")]
    y, pre, dx, dw, db = (Guarded(n, dtype).poison() for n in (rows * outs, rows * outs, rows * cols, runs * outs * cols, runs * outs))
    need = dt.dt_linear_backward_workspace([rows], runs, outs, "gelu", False, True, dtype)
    space = Guarded((need + 3) // 4, torch.float32).poison()
    dt.dt_linear([x], [w], [y.t], pre=[pre.t], offsets=off, act="gelu")
    dt.dt_linear_backward([dy], [x], [w], [dx.t], [dw.t], pre=[pre.t], dbias=[db.t], offsets=off, act="gelu", workspace=space.t)
    torch.cuda.synchronize()
    for t in (y, pre, dx, dw, db, space):
        t.check()


# -------------------------------------------- few tiles and a long summed index --
LONG = {
    # runs' rows of each rank (None: one run without offsets), cols, outs
    "a router": (None, [2000, 1500], 200, 48),
    "a router of whole lines": (None, [4100], 512, 64),
    "few columns": ([[40, 0, 33]], None, 24, 1500),
    "few rows": ([[1, 3], [0, 2]], None, 136, 2200),
    "odd rows": ([[777]], None, 99, 1033),
    "rows that end inside 16 bytes": ([[300, 411]], None, 66, 1034),
    "few rows that end inside 16 bytes": ([[30, 41]], None, 66, 2070),
    "one long run": ([[2500, 0, 3, 5]], None, 64, 40),
    "a row of many features": (None, [1], 40, 9001),
}


@DTYPES
@pytest.mark.parametrize("which", LONG, ids=lambda k: k.replace(" ", "_"))
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_gradients_with_long_sums(dt, which, gated, dtype):
    """Sums that are formed in parts: over the features for dx, over the rows for dweight."""
    note(f"long sums: {which} gated={gated} {dtype}")
    counts, rows, cols, outs = LONG[which]
    c = Case(rows or [sum(n) + 3 for n in counts], counts and [ends_of(n) for n in counts], cols, outs, gated, dtype, seed=40)
    check_backward(dt, c, "silu", True)
    check_backward(dt, c, "none", False)


@DTYPES
def test_long_sums_meet_only_their_rows(dt, dtype):
    """Rows outside the runs and the weights of a run without rows hold NaN, and an infinity stays in its row of dx."""
    note(f"long sums and NaN {dtype}")
    for cols, outs in ((64, 1200), (66, 1202), (40, 2100)):
        c = Case([3000], [[20, 1500, 1500, 2900]], cols, outs, False, dtype, seed=41)
        dy, nan = c.new(3000, outs), float("nan")
        for t in (c.x[0], dy):
            t[:20], t[2900:] = nan, nan
        c.weight[0][1] = nan
        dy[100, outs - 1] = float("inf")
        dx, dw = torch.zeros_like(c.x[0]), torch.zeros_like(c.weight[0])
        dt.dt_linear_backward([dy], c.x, c.weight, [dx], [dw], offsets=c.offsets)
        torch.cuda.synchronize()
        finite = dx[20:2900].isfinite().all(1)
        assert not bool(finite[80]) and int((~finite).sum()) == 1 and bool((dw[1] == 0).all())
        assert bool(dw[0, :-1].isfinite().all()) and not bool(dw[0, -1].isfinite().any()) and bool(dw[2].isfinite().all())
        assert bool((dx[:20] == 0).all()) and bool((dx[2900:] == 0).all())


# ------------------------------------------------------- elements past 32 bits --
def test_products_of_rows_past_32_bits(dt):
    """Runs at the end of 2^25 rows of 72 and 136 elements: their elements' numbers and bytes pass 2^32."""
    note("linear past 2^31 elements")
    rows, n, cols, outs = 2 ** 25 + 200, 150, 72, 136
    g = torch.Generator(device="cuda").manual_seed(24)
    lo = rows - n
    off = [torch.tensor([lo, lo + 20, rows], dtype=torch.int32, device="cuda")]
    x, y, dx, dy = (torch.empty(rows, k, dtype=torch.bfloat16, device="cuda") for k in (cols, outs, cols, outs))
    pre = torch.empty(rows, outs, dtype=torch.bfloat16, device="cuda")
    w, dw = normal(g, torch.bfloat16, 2, outs, cols, std=cols ** -0.5), torch.empty(2, outs, cols, dtype=torch.bfloat16, device="cuda")
    x[lo:], dy[lo:] = normal(g, torch.bfloat16, n, cols), normal(g, torch.bfloat16, n, outs)
    y[lo - 50:lo] = 7.0
    dx[lo - 50:lo] = 7.0
    dt.dt_linear([x], [w], [y], pre=[pre], offsets=off, act="silu")
    dt.dt_linear_backward([dy], [x], [w], [dx], [dw], pre=[pre], offsets=off, act="silu")
    torch.cuda.synchronize()
    assert bool((y[lo - 50:lo] == 7).all()) and bool((dx[lo - 50:lo] == 7).all())
    for e, (a, b) in enumerate(((lo, lo + 20), (lo + 20, rows))):
        want, err = ref.linear(x[a:b], w[e], None, None, "silu", False)
        ref.assert_close(y[a:b], want[0], err[0], "y")
        ref.assert_close(pre[a:b], want[1], err[1], "pre")
        want, err = ref.linear_backward(dy[a:b], x[a:b], w[e], pre[a:b], "silu", False)
        ref.assert_close(dx[a:b], want[0], err[0], "dx")
        ref.assert_close(dw[e], want[1], err[1], "dweight")


def test_norms_of_rows_past_32_bits(dt):
    note("block past 2^31 elements")
    rows, cols, n = 2 ** 21 + 37, 1032, 70
    b = Block([n], cols, torch.bfloat16, seed=25)
    z, x, h, y, dz, dx = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(6))
    stats = torch.empty(rows, 4, device="cuda")
    for t, last in ((z, b.z[0]), (x, b.x[0])):
        t[:-n] = last[:1]
        t[-n:] = last
    dt.dt_block_norm([z], [x], [h], [y], gate=b.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, pre_bias=b.b2, stats=[stats])
    torch.cuda.synchronize()
    want = ref.block(b.z[0], b.x[0], b.gate[0], b.w1[0], b.b1[0], b.w2[0], b.b2[0], 1.0, False, 1e-5)
    for name, t in dict(h=h, y=y, stats=stats).items():
        ref.assert_close(t[-n:], *want[name], name)
        assert torch.equal(t[:-n].view(torch.int16), t[:1].expand(rows - n, -1).contiguous().view(torch.int16)), name
    # dy and dh take the place of the forward pass's inputs
    y[:-n], y[-n:] = b.dy[0][:1], b.dy[0]
    x[:-n], x[-n:] = b.dh[0][:1], b.dh[0]
    dt.dt_block_norm_backward([y], [x], [z], [h], [stats], [dz], [dx], gate=b.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2)
    torch.cuda.synchronize()
    want = ref.block_backward(b.dy[0], b.dh[0], z[-n:], h[-n:], b.gate[0], b.w1[0], b.b1[0], b.w2[0], stats[-n:], 1.0, False)
    for name, t in dict(dx=dx, dz=dz).items():
        ref.assert_close(t[-n:], *want[name], name)
        assert torch.equal(t[:-n].view(torch.int16), t[:1].expand(rows - n, -1).contiguous().view(torch.int16)), name


@DTYPES
@pytest.mark.parametrize("cols", [1, 3, 9, 61, 301, 1001, 1999, 4001])
def test_rows_that_follow_do_not_matter(dt, cols, dtype):
    """Rows that end inside 16 bytes: every other row is NaN, and nothing of it reaches the rows between."""
    note(f"block between rows of NaN, cols={cols} {dtype}")
    b = Block([41, 2, 1], cols, dtype, gate="row", seed=cols)
    other = Block([41, 2, 1], cols, dtype, gate="row", seed=cols)
    for kind in ("z", "x", "gate", "dy", "dh", "h"):
        for t in getattr(other, kind):
            t[1::2] = float("nan")
    stats = [torch.rand(n, 4, device="cuda") + 0.5 for n in b.rows]
    got = []
    for c in (b, other):
        h, y, dz, dx, dg = ([torch.zeros_like(t) for t in c.z] for _ in range(5))
        dt.dt_block_norm(c.z, c.x, h, y, gate=c.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, pre_bias=b.b2)
        dt.dt_block_norm_backward(c.dy, c.dh, c.z, c.h, stats, dz, dx, gate=c.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, dgate=dg)
        torch.cuda.synchronize()
        got.append(h + y + dz + dx + dg)
    for one, two in zip(*got):
        assert torch.equal(one[::2], two[::2]) and bool(one.isfinite().all()) and bool(two[1::2].isnan().all())


# -------------------------------------------------------------------- together --
def test_a_training_step(dt):
    """Block norm, router, routing, dispatch, the experts' two products, combine, block norm; and the way back: every gradient
    against that of the same step in 64 bits, differentiated by autograd for the routing that the step chose.

    fp32 throughout: a sum has at most 96 terms, so an operator adds a relative error of about (96 + 30) 2^-24 = 8e-6 of the
    largest magnitudes; ten of them one behind the other, each amplifying what came by no more than about 4, stay under 1e-3."""
    note("training step of an expert block")
    p, cols, inner, e, k = 2, 48, 40, 6, 2
    rows, per, cap = [29, 18], 3, 47 * 2
    g = torch.Generator(device="cuda").manual_seed(26)
    f32 = torch.float32
    new = lambda *s, std=1.0: normal(g, f32, *s, std=std)
    like = lambda ts: [torch.zeros_like(t) for t in ts]
    a, x = [new(n, cols) for n in rows], [new(n, cols) for n in rows]
    gate, n1, b1, n2, b2, n3, b3 = ([new(cols, std=0.3) + s] * p for s in (1.0, 1.0, 0.0, 1.0, 0.0, 1.0, 0.0))
    router = [new(e, cols, std=0.4)] * p
    w_in, v_in = [new(per, 2 * inner, cols, std=cols ** -0.5) for _ in rows], [new(per, 2 * inner, std=0.2) for _ in rows]
    w_out, v_out = [new(per, cols, inner, std=inner ** -0.5) for _ in rows], [new(per, cols, std=0.2) for _ in rows]
    dy, dh = [new(n, cols) for n in rows], [new(n, cols) for n in rows]

    room = lambda width: [torch.zeros(cap, width, device="cuda") for _ in rows]
    token = lambda width, dtype=f32: [torch.zeros(n, width, dtype=dtype, device="cuda") for n in rows]
    h1, y1, s1, logits, h2, y2, s2, m = (token(w) for w in (cols, cols, 4, e, cols, cols, 4, cols))
    experts, pos, weights = token(k, torch.int32), token(k, torch.int32), token(k)
    off = [torch.zeros(per + 1, dtype=torch.int32, device="cuda") for _ in rows]
    recv, mid, pre, back = room(cols), room(inner), room(2 * inner), room(cols)
    d_m, d_h1, d_back, d_weights, d_mid, d_recv, d_logits, d_y1, d_y1r, d_a, d_x = (
        token(cols), token(cols), room(cols), token(k), room(inner), room(cols), token(e), token(cols), token(cols), token(cols), token(cols))
    d_w_in, d_v_in, d_w_out, d_v_out, d_router = like(w_in), like(v_in), like(w_out), like(v_out), [torch.zeros_like(router[0]) for _ in rows]
    d_gate, d_n1, d_b1, d_n2, d_b2, d_n3, d_b3 = ([torch.zeros(cols, device="cuda") for _ in rows] for _ in range(7))

    def step():
        dt.dt_block_norm(a, x, h1, y1, gate=gate, post_weight=n1, post_bias=b1, pre_weight=n2, pre_bias=b2, stats=s1)
        dt.dt_linear(y1, router, logits)
        dt.dt_moe_route(logits, experts, weights)
        dt.dt_moe_dispatch(y1, experts, recv, pos, off, e)
        dt.dt_linear(recv, w_in, mid, bias=v_in, pre=pre, offsets=off, act="silu", gated=True)
        dt.dt_linear(mid, w_out, back, bias=v_out, offsets=off)
        dt.dt_moe_combine(back, experts, pos, weights, m, e)
        dt.dt_block_norm(m, h1, h2, y2, scale=0.5, pre_weight=n3, pre_bias=b3, stats=s2, rms=True)
        # and back
        dt.dt_block_norm_backward(dy, dh, m, h2, s2, d_m, d_h1, scale=0.5, pre_weight=n3, dpre_weight=d_n3, dpre_bias=d_b3, rms=True)
        dt.dt_moe_combine_backward(d_m, back, experts, pos, weights, d_back, d_weights, e)
        dt.dt_linear_backward(d_back, mid, w_out, d_mid, d_w_out, dbias=d_v_out, offsets=off)
        dt.dt_linear_backward(d_mid, recv, w_in, d_recv, d_w_in, pre=pre, dbias=d_v_in, offsets=off, act="silu", gated=True)
        dt.dt_moe_combine(d_recv, experts, pos, None, d_y1, e)
        dt.dt_moe_route_backward(logits, experts, d_weights, d_logits)
        dt.dt_linear_backward(d_logits, y1, router, d_y1r, d_router)
        for q in range(p):
            d_y1[q] += d_y1r[q]
        dt.dt_block_norm_backward(d_y1, d_h1, a, h1, s1, d_a, d_x, gate=gate, post_weight=n1, post_bias=b1, pre_weight=n2, dgate=d_gate,
                                  dpost_weight=d_n1, dpost_bias=d_b1, dpre_weight=d_n2, dpre_bias=d_b2)

    step()
    torch.cuda.synchronize()
    leaf = lambda ts: torch.cat(ts).double().requires_grad_()
    one = lambda ts: ts[0].double().requires_grad_()
    A, X, WI, VI, WO, VO = (leaf(t) for t in (a, x, w_in, v_in, w_out, v_out))
    G, N1, B1, N2, B2, N3, B3, R = (one(t) for t in (gate, n1, b1, n2, b2, n3, b3, router))
    chosen = torch.cat(experts).long()

    def norm(v, w, b, rms=False):
        v = v if rms else v - v.mean(1, keepdim=True)
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-5) * w + b

    H1 = X + G * norm(A, N1, B1)
    Y1 = norm(H1, N2, B2)
    L = (Y1[:, None, :] * R).sum(2)
    top = L.detach().topk(k, 1).indices
    assert torch.equal(top.sort(1).values, chosen.sort(1).values)
    W = torch.softmax(L.gather(1, chosen), 1)     # softmax over all, renormalised over the chosen
    M = 0
    for j in range(k):
        z = (WI[chosen[:, j]] * Y1[:, None, :]).sum(2) + VI[chosen[:, j]]
        v = torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]
        M = M + W[:, j:j + 1] * ((WO[chosen[:, j]] * v[:, None, :]).sum(2) + VO[chosen[:, j]])
    H2 = H1 + 0.5 * M
    Y2 = norm(H2, N3, B3, True)
    ((Y2 * torch.cat(dy).double()).sum() + (H2 * torch.cat(dh).double()).sum()).backward()

    def close(name, got, want):
        assert float((got.double() - want).abs().max()) <= 1e-3 * float(want.abs().max()), name

    close("h", torch.cat(h2), H2.detach())
    close("y", torch.cat(y2), Y2.detach())
    for name, got, leaf_ in (("z", d_a, A), ("x", d_x, X), ("w_in", d_w_in, WI), ("b_in", d_v_in, VI), ("w_out", d_w_out, WO),
                             ("b_out", d_v_out, VO)):
        close(name, torch.cat(got), leaf_.grad)
    for name, got, leaf_ in (("gate", d_gate, G), ("post_weight", d_n1, N1), ("post_bias", d_b1, B1), ("pre_weight", d_n2, N2),
                             ("pre_bias", d_b2, B2), ("last weight", d_n3, N3), ("last bias", d_b3, B3)):
        for t in got:
            close(name, t, leaf_.grad)
    close("router", sum(d_router), R.grad)

    # the same step captured, and replayed on other inputs in place
    outs = h2 + y2 + d_a + d_x + d_w_in + d_w_out + d_v_in + d_v_out + d_router + d_gate + d_n1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        for t in a + x:
            t.mul_(-0.9).add_(0.05 * turn)
        for t in recv + mid + pre + back + d_back + d_mid + d_recv:
            t.zero_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(outs, want)), turn


@DTYPES
def test_a_decoding_step(dt, dtype):
    """Few tokens: block norm, router, routing, the experts' layer, block norm with the layer's result, prepared and run again
    with other tokens in place; each operator against its definition on what it was given."""
    note(f"decoding step of an expert block {dtype}")
    c = Layer([5, 3], 256, 96, 8, 2, True, dtype, True, False, seed=27)
    b = Block([5, 3], 256, dtype, gate="none", rms=True, bias=False, seed=28)
    router = [normal(torch.Generator(device="cuda").manual_seed(29), dtype, 8, 256, std=0.1)] * 2
    h, y, m, h2 = ([torch.zeros_like(t) for t in b.z] for _ in range(4))
    y2, logits = [torch.zeros_like(t) for t in b.z], [torch.zeros(n, 8, dtype=dtype, device="cuda") for n in b.rows]
    c.x = y
    calls = [
        dt.prepare(dt.dt_block_norm, b.z, b.x, h, y, post_weight=b.w1, pre_weight=b.w2, rms=True),
        dt.prepare(dt.dt_linear, y, router, logits),
        dt.prepare(dt.dt_moe_route, logits, c.experts, c.weights),
        dt.prepare(dt.dt_moe_layer, y, c.experts, c.weights, c.w_in, c.w_out, m, b_in=c.b_in, b_out=c.b_out, act="silu", gated=True),
        dt.prepare(dt.dt_block_norm, m, h, h2, y2, pre_weight=b.w2, rms=True),
    ]
    cat = torch.cat
    for turn in range(3):
        for t in b.z + b.x:
            t.mul_(-1.25)
        for call in calls:
            call()
        torch.cuda.synchronize()
        first = ref.block(cat(b.z), cat(b.x), None, b.w1[0], None, b.w2[0], None, 1.0, True, 1e-5)
        ref.assert_close(cat(h), *first["h"], "h")
        ref.assert_close(cat(y), *first["y"], "y")
        want, err = ref.linear(cat(y), router[0], None, None, "none", False)
        ref.assert_close(cat(logits), want[0], err[0], "logits")
        want, err = c.reference("silu")
        ref.assert_close(cat(m), want, err, "layer")
        second = ref.block(cat(m), cat(h), None, None, None, b.w2[0], None, 1.0, True, 1e-5)
        ref.assert_close(cat(h2), *second["h"], "second h")
        ref.assert_close(cat(y2), *second["y"], "second y")


def test_two_calls_at_once(dt):
    """The same operators on two streams at a time, each with the workspace that its call takes for itself."""
    note("two streams")
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for i in range(2):
        c = Case([300, 200], [[0, 100, 300], [0, 150, 199]], 256, 200, True, torch.bfloat16, seed=30 + i)
        lay = Layer([20, 30], 256, 128, 8, 2, True, torch.bfloat16, seed=32 + i)
        b = Block([400, 300], 1024, torch.bfloat16, seed=34 + i)
        pre, dy = [c.new(n, c.wide) for n in c.rows], [c.new(n, c.outs) for n in c.rows]
        stats = [torch.rand(n, 4, device="cuda") + 0.5 for n in b.rows]
        dx, dw, out = [torch.zeros_like(t) for t in c.x], [torch.zeros_like(t) for t in c.weight], [torch.zeros_like(t) for t in lay.x]
        bz, bx, bw = [torch.zeros_like(t) for t in b.z], [torch.zeros_like(t) for t in b.z], [torch.zeros_like(t) for t in b.w2]

        def run(c=c, lay=lay, b=b, pre=pre, dy=dy, stats=stats, dx=dx, dw=dw, out=out, bz=bz, bx=bx, bw=bw, **kw):
            dt.dt_linear_backward(dy, c.x, c.weight, dx, dw, pre=pre, offsets=c.offsets, act="silu", gated=True, **kw)
            lay.run(dt, out, "silu", **kw)
            dt.dt_block_norm_backward(b.dy, b.dh, b.z, b.h, stats, bz, bx, gate=b.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2,
                                      dpre_weight=bw, **kw)
            return dx + dw + out + bz + bx + bw

        outs = run()
        torch.cuda.synchronize()
        work.append((run, outs, [t.clone() for t in outs]))
    for _ in range(5):
        for _, outs, want in work:
            for t in outs:
                t[..., ::3] = 5.0
            outs[1][199:] = want[1][199:]   # dx of a row outside the runs, which no call writes
        torch.cuda.synchronize()
        for _ in range(3):
            for s, (run, _, _) in zip(streams, work):
                run(stream=s)
        torch.cuda.synchronize()
        for _, outs, want in work:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
