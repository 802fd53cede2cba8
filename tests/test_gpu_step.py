"""GPU: the model-step operators together, as a sharded training step uses
them (norm -> route -> dispatch -> experts -> combine -> norm -> loss, and
back), against a 64-bit model by automatic differentiation; the same step on
a side stream, prepared, and captured into a graph and replayed."""
import pytest
import torch

import step_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


class Step:
    """P ranks' buffers of one step, and the step itself."""

    def __init__(self, dt, rows, cols, e, k, shards, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dt, self.rows, self.cols, self.e, self.k, self.dtype = dt, rows, cols, e, k, dtype
        p, n = len(rows), sum(rows)
        self.p, self.n = p, n

        def new(*s, std=1.0, mean=0.0):
            return (torch.randn(s, generator=g, device="cuda") * std + mean).to(dtype)

        def empty(*s, kind=dtype):
            return torch.empty(s, dtype=kind, device="cuda")

        self.x = [new(r, cols) for r in rows]
        self.w1, self.b1 = new(cols, std=0.1, mean=1.0), new(cols, std=0.1)
        self.w2 = new(cols, std=0.1, mean=1.0)
        self.router = new(cols, e, std=cols ** -0.5)
        self.gain = [(torch.rand(e // p, 1, generator=g, device="cuda") + 0.5).to(dtype) for _ in range(p)]  # an expert scales its rows
        self.head = [new(v, cols, std=2 * cols ** -0.5) for v in shards]
        self.targets = torch.randint(0, sum(shards), (n,), generator=g, device="cuda")
        self.targets[::7] = -100
        self.dloss = torch.full((n,), 1.0 / n, device="cuda")
        f32, i32 = torch.float32, torch.int32
        cap = n * k
        self.h1, self.m1, self.r1 = [empty(r, cols) for r in rows], [empty(r, kind=f32) for r in rows], [empty(r, kind=f32) for r in rows]
        self.experts, self.weights = [empty(r, k, kind=i32) for r in rows], [empty(r, k, kind=f32) for r in rows]
        self.recv, self.off = [empty(cap, cols) for _ in range(p)], [empty(e // p + 1, kind=i32) for _ in range(p)]
        self.pos = [empty(r, k, kind=i32) for r in rows]
        self.moe = [empty(r, cols) for r in rows]
        # all ranks' hidden rows are gathered before the loss: one tensor, rank r's rows a slice of it
        self.h2 = empty(n, cols)
        self.h2r = list(self.h2.split(rows))
        self.m2, self.r2 = [empty(r, kind=f32) for r in rows], [empty(r, kind=f32) for r in rows]
        self.loss, self.lse = [empty(n, kind=f32) for _ in range(p)], [empty(n, kind=f32) for _ in range(p)]
        self.dh2, self.dhead = [empty(n, cols) for _ in range(p)], [empty(v, cols) for v in shards]
        self.dmoe, self.dw2 = [empty(r, cols) for r in rows], [empty(cols) for _ in range(p)]
        self.dy, self.dwt = [torch.zeros(cap, cols, dtype=dtype, device="cuda") for _ in range(p)], [empty(r, k, kind=f32) for r in rows]
        self.dlog = [empty(r, e) for r in rows]
        self.dh1, self.dx = [empty(r, cols) for r in rows], [empty(r, cols) for r in rows]
        self.dw1, self.db1 = [empty(cols) for _ in range(p)], [empty(cols) for _ in range(p)]

    def outputs(self):
        return [*self.loss, *self.dhead, *self.dx, *self.dw1, *self.db1, *self.dw2, *self.dlog, *self.dwt]

    def __call__(self):
        dt, p = self.dt, self.p
        dt.dt_layer_norm(self.x, [self.w1] * p, [self.b1] * p, self.h1, self.m1, self.r1)
        logits = [h @ self.router for h in self.h1]
        dt.dt_moe_route(logits, self.experts, self.weights, score="softmax", renormalize=True)
        dt.dt_moe_dispatch(self.h1, self.experts, self.recv, self.pos, self.off, self.e)
        rows = torch.arange(self.recv[0].shape[0], device="cuda")
        gain = []
        y = []
        for q in range(p):  # every row's expert from the offsets
            at = (rows[:, None] >= self.off[q][None, 1:]).sum(1).clamp(max=self.e // p - 1)
            gain.append(self.gain[q][at])
            live = rows[:, None] < self.off[q][-1:]
            y.append(torch.where(live, self.recv[q] * gain[q], 0.0))
        dt.dt_moe_combine(y, self.experts, self.pos, self.weights, self.moe, self.e)
        dt.dt_layer_norm(self.moe, [self.w2] * p, None, self.h2r, self.m2, self.r2)
        dt.dt_vocab_loss([self.h2] * p, self.head, [self.targets] * p, self.loss, self.lse)
        dt.dt_vocab_loss_backward([self.h2] * p, self.head, [self.targets] * p, self.lse, [self.dloss] * p, self.dh2, self.dhead)
        mine = [self.dh2[r].split(self.rows)[r] for r in range(p)]
        dt.dt_layer_norm_backward(mine, self.moe, [self.w2] * p, self.m2, self.r2, self.dmoe, self.dw2)
        dt.dt_moe_combine_backward(self.dmoe, y, self.experts, self.pos, self.weights, self.dy, self.dwt, self.e)
        dt.dt_moe_route_backward(logits, self.experts, self.dwt, self.dlog, score="softmax", renormalize=True)
        drecv = [d * g for d, g in zip(self.dy, gain)]
        dt.dt_moe_combine(drecv, self.experts, self.pos, None, self.dh1, self.e)
        total = [a + b @ self.router.t().contiguous() for a, b in zip(self.dh1, self.dlog)]
        dt.dt_layer_norm_backward(total, self.x, [self.w1] * p, self.m1, self.r1, self.dx, self.dw1, self.db1)

    def reference(self):
        """The same step in 64 bits for the same choice of experts."""
        d = lambda t: t.detach().double().cpu()
        x, w1, b1, w2, router = (d(t).requires_grad_(True) for t in (torch.cat(self.x), self.w1, self.b1, self.w2, self.router))
        head = d(torch.cat(self.head)).requires_grad_(True)
        gain = d(torch.cat(self.gain))

        def norm(v, w, b):
            m = v.mean(1, keepdim=True)
            return (v - m) / torch.sqrt((v - m).square().mean(1, keepdim=True) + 1e-5) * w + b

        h1 = norm(x, w1, b1)
        logits = h1 @ router
        ex = torch.cat(self.experts).long().cpu()
        s = logits.softmax(1).gather(1, ex)
        w = s / s.sum(1, keepdim=True)
        moe = (w[:, :, None] * h1[:, None, :] * gain[ex]).sum(1)
        h2 = norm(moe, w2, 0.0)
        z = h2 @ head.t()
        t = self.targets.cpu()
        use = t >= 0
        loss = torch.where(use, torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
        (loss * d(self.dloss)).sum().backward()
        return dict(loss=loss, dx=x.grad, dw1=w1.grad, db1=b1.grad, dw2=w2.grad, dhead=head.grad, logits=logits)


def _norm_error(got, want):
    got, want = got.detach().double().cpu(), want.detach()
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("rows,cols,e,k,shards", [([33, 20, 0, 47], 96, 8, 2, [100, 60, 1, 80]), ([64, 65], 260, 6, 3, [300, 211])])
def test_a_training_step(dt, rows, cols, e, k, shards):
    note(f"step rows={rows} cols={cols}")
    s = Step(dt, rows, cols, e, k, shards, torch.float32)
    s()
    torch.cuda.synchronize()
    want = s.reference()
    n, _, _ = ref.route(want["logits"].detach(), k)
    assert torch.equal(n, torch.cat(s.experts).long().cpu())
    # Sums of at most 512 terms in ten stages one after the other: 10 * (512 + 16) * U = 3.1e-4 of the result's size, if no
    # stage amplifies what it is given; the norms divide by a spread near 1 and the gains and weights are near 1.
    bar = 10 * (512 + 16) * ref.U
    for q in range(s.p):
        assert _norm_error(s.loss[q], want["loss"]) < bar
        assert _norm_error(s.dw1[q], want["dw1"]) < bar and _norm_error(s.db1[q], want["db1"]) < bar
        assert _norm_error(s.dw2[q], want["dw2"]) < bar
    assert _norm_error(torch.cat(s.dx), want["dx"]) < bar
    assert _norm_error(torch.cat(s.dhead), want["dhead"]) < bar


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_a_captured_step_replays(dt, dtype):
    """Every replay gives the eager bits, with eager work and new inputs in between."""
    note(f"captured step {dtype}")
    s, eager = Step(dt, [31, 50], 128, 8, 2, [90, 70], dtype, 3), Step(dt, [31, 50], 128, 8, 2, [90, 70], dtype, 3)
    s()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s()
    for i in range(4):
        new = [torch.randn_like(x.float()).to(dtype) for x in s.x]
        for a, b, v in zip(s.x, eager.x, new):
            a.copy_(v)
            b.copy_(v)
        for t in s.outputs():
            t.fill_(float("nan"))
        eager()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s.outputs(), eager.outputs()):
            assert torch.equal(a, b), f"replay {i}"


def test_side_stream_prepared_and_given_workspace(dt):
    """The async form, the prepared form and a caller's workspace leave the plain call's bits, the first also behind a
    producer that is late."""
    note("step operators async, prepared, with workspace")
    s, t = Step(dt, [40, 9], 200, 4, 2, [130, 61], torch.bfloat16, 5), Step(dt, [40, 9], 200, 4, 2, [130, 61], torch.bfloat16, 5)
    s()
    p = 2
    x = [v.clone() for v in t.x]
    for v in t.x:
        v.zero_()
    torch.cuda._sleep(20_000_000)
    for v, o in zip(t.x, x):
        v.copy_(o)
    work = dt.dt_layer_norm(t.x, [t.w1] * p, [t.b1] * p, t.h1, t.m1, t.r1, async_op=True)
    work.wait()
    logits = [h @ t.router for h in t.h1]
    dt.dt_moe_route(logits, t.experts, t.weights, async_op=True).wait()
    dt.dt_moe_dispatch(t.h1, t.experts, t.recv, t.pos, t.off, t.e, async_op=True).wait()
    torch.cuda.synchronize()
    for a, b in zip(s.h1 + s.experts + s.weights + s.pos + s.off, t.h1 + t.experts + t.weights + t.pos + t.off):
        assert torch.equal(a, b)
    t.h2.copy_(s.h2)
    ws = torch.empty(dt.dt_vocab_loss_workspace([130, 61], 49, 200), dtype=torch.uint8, device="cuda")
    fwd = dt.prepare(dt.dt_vocab_loss, [t.h2] * p, t.head, [t.targets] * p, t.loss, t.lse, workspace=ws)
    wb = torch.empty(dt.dt_vocab_loss_backward_workspace([130, 61], 49, 200), dtype=torch.uint8, device="cuda")
    bwd = dt.prepare(dt.dt_vocab_loss_backward, [t.h2] * p, t.head, [t.targets] * p, t.lse, [t.dloss] * p, t.dh2, t.dhead, workspace=wb)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        fwd(other)
        bwd(other)
    torch.cuda.synchronize()
    for a, b in zip(s.loss + s.lse + s.dh2 + s.dhead, t.loss + t.lse + t.dh2 + t.dhead):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        dt.dt_vocab_loss([t.h2] * p, t.head, [t.targets] * p, t.loss, t.lse, workspace=ws[:8])


def test_the_binding_refuses(dt):
    note("step operators: refusals of the binding")
    x, w = [torch.randn(4, 8, device="cuda")] * 2, [torch.ones(8, device="cuda")] * 2
    y = [torch.empty(4, 8, device="cuda") for _ in range(2)]
    with pytest.raises(ValueError):
        dt.dt_layer_norm(x, w, None, y[:1])
    with pytest.raises(TypeError):
        dt.dt_layer_norm([v.half() for v in x], w, None, y)
    with pytest.raises(TypeError):
        dt.dt_layer_norm(x, [v.bfloat16() for v in w], None, y)
    with pytest.raises(ValueError):
        dt.dt_layer_norm([v.t() for v in x], w, None, y)
    with pytest.raises(ValueError):
        dt.dt_layer_norm([v.cpu() for v in x], w, None, y)
    with pytest.raises(dt.DtError):
        dt.dt_layer_norm([y[0], x[1]], w, None, y)  # in place
    ex, we = [torch.empty(4, 2, dtype=torch.int32, device="cuda")] * 2, [torch.empty(4, 2, device="cuda") for _ in range(2)]
    with pytest.raises(dt.DtError):
        dt.dt_moe_route(x, ex, we)  # one buffer for two ranks' experts
    with pytest.raises(ValueError):
        dt.dt_moe_combine(x, ex, ex, we, y, 3)  # 3 experts on 2 ranks


def test_a_workspace_of_the_library_on_other_streams(dt):
    """The library's own workspace, taken while the current stream still writes a block that was just given back:
    the call on another stream, plain or prepared, neither sees nor disturbs that."""
    note("step operators: workspace of the library on another stream")
    p, rows, cols = 2, 600, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = ([torch.randn(rows, cols, generator=g, device="cuda") for _ in range(p)] for _ in range(2))
    w = [torch.ones(cols, device="cuda")] * p
    y, dx = ([torch.empty_like(v) for v in x] for _ in range(2))
    m, r = ([torch.empty(rows, device="cuda") for _ in range(p)] for _ in range(2))
    want, dw = ([torch.empty(cols, device="cuda") for _ in range(p)] for _ in range(2))
    dt.dt_layer_norm(x, w, None, y, m, r)
    dt.dt_layer_norm_backward(dy, x, w, m, r, dx, want)
    nbytes = dt.dt_layer_norm_workspace([rows] * p, cols)
    other, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for v in dw:
            v.zero_()
        torch.cuda.synchronize()
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(5_000_000)
        block.fill_(255)
        del block
        dt.dt_layer_norm_backward(dy, x, w, m, r, dx, dw, stream=other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(dw, want))
        for v in dw:
            v.zero_()
        torch.cuda.synchronize()
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(5_000_000)
        block.fill_(255)
        del block
        step = dt.prepare(dt.dt_layer_norm_backward, dy, x, w, m, r, dx, dw)
        step(third)
        del step
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(dw, want))
        del block
