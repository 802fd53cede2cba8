"""GPU: the experts' layer for few tokens against its 64-bit definition and the
calls that it stands for, with canaries around the output."""
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


class Layer:
    def __init__(self, rows, cols, inner, experts, topk, gated, dtype, bias=False, residual=False, offset=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        p, per, wide = len(rows), experts // len(rows), inner * (2 if gated else 1)
        self.rows, self.cols, self.inner, self.e, self.k, self.gated, self.dtype, self.at = rows, cols, inner, experts, topk, gated, dtype, offset
        self.p = p

        def new(*shape, std=1.0):
            n = 1
            for s in shape:
                n *= s
            buf = torch.empty(offset + n, dtype=dtype, device="cuda")
            buf[offset:] = (torch.randn(n, generator=g, device="cuda") * std).to(dtype)
            return buf[offset:].view(*shape)

        self.x = [new(n, cols) for n in rows]
        self.experts = [torch.rand(n, experts, generator=g, device="cuda").topk(topk, 1).indices.to(torch.int32) for n in rows]
        self.weights = [torch.rand(n, topk, generator=g, device="cuda") for n in rows]
        self.w_in = [new(per, wide, cols, std=cols ** -0.5) for _ in rows]
        self.w_out = [new(per, cols, inner, std=inner ** -0.5) for _ in rows]
        self.b_in = [new(per, wide, std=0.5) for _ in rows] if bias else None
        self.b_out = [new(per, cols, std=0.5) for _ in rows] if bias else None
        self.residual = [new(n, cols) for n in rows] if residual else None

    def run(self, dt, out, kind, **kw):
        dt.dt_moe_layer(self.x, self.experts, self.weights, self.w_in, self.w_out, out, b_in=self.b_in, b_out=self.b_out,
                        residual=self.residual, act=kind, gated=self.gated, **kw)

    def reference(self, kind):
        cat = lambda v: None if v is None else torch.cat(v)
        return ref.layer(torch.cat(self.x), torch.cat(self.experts), torch.cat(self.weights), torch.cat(self.w_in), torch.cat(self.w_out),
                         cat(self.b_in), cat(self.b_out), cat(self.residual), kind, self.gated)

    def check(self, dt, kind="silu"):
        out = [Guarded(n * self.cols, self.dtype, offset_elems=self.at).poison() for n in self.rows]
        self.run(dt, [t.t for t in out], kind)
        torch.cuda.synchronize()
        for t in out:
            t.check()
        want, err = self.reference(kind)
        ref.assert_close(torch.cat([t.t for t in out]).view(-1, self.cols), want, err, "out")


CASES = [
    # rows, cols, inner, experts, topk, gated, bias, residual, elements past an aligned start
    ([1], 64, 32, 4, 1, True, False, False, 0),
    ([1], 1, 1, 1, 1, False, True, True, 0),
    ([0, 3], 40, 24, 6, 2, True, True, False, 0),
    ([2, 1, 5], 100, 36, 9, 3, False, True, True, 0),
    ([5], 129, 65, 5, 5, True, False, True, 0),
    ([16, 1], 256, 64, 8, 2, True, False, False, 0),
    ([20, 20], 130, 50, 4, 2, True, True, True, 1),
    ([33], 72, 520, 3, 2, False, False, False, 0),
    ([100, 28], 320, 192, 64, 4, True, False, True, 0),
    ([250, 6], 96, 80, 2, 1, True, False, False, 0),
    ([60] * 4, 136, 72, 256, 8, True, True, False, 0),
    ([1] * 16, 512, 264, 1024, 64, True, False, False, 0),
    ([90], 1032, 1000, 2, 2, False, True, False, 0),
]


@DTYPES
@pytest.mark.parametrize("rows,cols,inner,experts,topk,gated,bias,residual,offset", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_layer(dt, rows, cols, inner, experts, topk, gated, bias, residual, offset, dtype):
    note(f"layer rows={rows} cols={cols} inner={inner} experts={experts} topk={topk} gated={gated} {dtype}")
    Layer(rows, cols, inner, experts, topk, gated, dtype, bias, residual, offset).check(dt)


@DTYPES
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_activations(dt, kind, gated, dtype):
    note(f"layer act={kind} gated={gated} {dtype}")
    Layer([9, 2], 48, 40, 4, 2, gated, dtype, True, True, seed=2).check(dt, kind)


@DTYPES
def test_padded_tokens_and_missing_experts(dt, dtype):
    """Slots without an expert add nothing, whatever their weight; a token with none gets its residual, or zeros."""
    note(f"layer with padded tokens {dtype}")
    for residual in (False, True):
        c = Layer([12, 7], 64, 48, 6, 3, True, dtype, True, residual, seed=4)
        c.experts[0][3] = -1
        c.experts[0][5, 1] = -1
        c.experts[1][2] = torch.tensor([6, -7, 2 ** 31 - 1], dtype=torch.int32)
        c.weights[0][3] = float("nan")
        c.x[1][2] = float("nan")
        out = [torch.empty_like(t) for t in c.x]
        c.run(dt, out, "silu")
        torch.cuda.synchronize()
        c.weights[0][3] = 0.0
        c.x[1][2] = 0.0
        want, err = c.reference("silu")
        ref.assert_close(torch.cat(out), want, err, "out")
        assert torch.equal(out[0][3], c.residual[0][3] if residual else torch.zeros_like(out[0][3]))
        for e in c.experts:
            e.fill_(-1)
        c.run(dt, out, "silu")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b if residual else torch.zeros_like(a)) for a, b in zip(out, c.residual if residual else out))


def test_the_same_expert_twice_counts_twice(dt):
    note("layer with repeated experts")
    c = Layer([6], 32, 24, 3, 3, False, torch.float32, True, False, seed=5)
    c.experts[0][0] = torch.tensor([1, 1, 1], dtype=torch.int32)
    c.experts[0][1] = torch.tensor([2, 0, 2], dtype=torch.int32)
    c.check(dt, "gelu")


def test_every_token_to_one_expert(dt):
    note("layer with one expert in use")
    for n in (16, 17, 48, 65, 256):
        c = Layer([n], 64, 64, 8, 1, True, torch.bfloat16, seed=n)
        c.experts[0].fill_(5)
        c.check(dt)


def test_infinite_values_stay_with_their_token(dt):
    note("layer inf")
    for dtype in (torch.bfloat16, torch.float32):
        c = Layer([20], 70, 40, 4, 2, False, dtype, seed=6)
        c.x[0][7] = float("nan")
        out = [torch.empty_like(t) for t in c.x]
        c.run(dt, out, "relu")
        torch.cuda.synchronize()
        finite = out[0].isfinite().all(1)
        assert bool(out[0][7].isnan().any()) and int((~finite).sum()) == 1
        # unused experts' weights are not met: token 7 has lost its experts, and nothing of them is left
        used = torch.zeros(4, dtype=torch.bool)
        used[c.experts[0].long().cpu().reshape(-1)] = True
        c.x[0][7] = 1.0
        c.experts[0][:] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        c.w_in[0][2:] = float("nan")
        c.w_out[0][2:] = float("nan")
        c.run(dt, out, "relu")
        torch.cuda.synchronize()
        assert bool(out[0].isfinite().all())


def test_an_expert_s_infinite_weights_stay_with_its_tokens(dt):
    note("layer with infinite weights")
    for dtype in (torch.bfloat16, torch.float32):
        c = Layer([20, 14], 64, 40, 4, 2, True, dtype, seed=10)
        for e in c.experts:
            e[:, 0], e[:, 1] = 0, 2
            e[::3, 1] = 3
        c.w_out[1][1] = float("inf")
        c.w_out[1][1, ::2] = float("nan")
        out = [torch.empty_like(t) for t in c.x]
        c.run(dt, out, "silu")
        torch.cuda.synchronize()
        for e, o in zip(c.experts, out):
            assert bool(o[(e != 3).all(1)].isfinite().all()) and not bool(o[(e == 3).any(1)].isfinite().any())


def test_as_the_calls_that_it_stands_for(dt):
    """Routing decides; dispatch, two products and combine give what the layer gives."""
    note("layer against dispatch, products and combine")
    c = Layer([30, 21], 96, 64, 8, 2, True, torch.float32, True, False, seed=7)
    logits = [torch.randn(n, 8, device="cuda") for n in c.rows]
    dt.dt_moe_route(logits, c.experts, c.weights)
    cap = sum(c.rows) * 2
    recv, off = [torch.zeros(cap, 96, device="cuda") for _ in range(2)], [torch.zeros(5, dtype=torch.int32, device="cuda") for _ in range(2)]
    pos = [torch.zeros(n, 2, dtype=torch.int32, device="cuda") for n in c.rows]
    mid, back = [torch.zeros(cap, 64, device="cuda") for _ in range(2)], [torch.zeros(cap, 96, device="cuda") for _ in range(2)]
    far, near = [torch.empty_like(t) for t in c.x], [torch.empty_like(t) for t in c.x]
    dt.dt_moe_dispatch(c.x, c.experts, recv, pos, off, 8)
    dt.dt_linear(recv, c.w_in, mid, bias=c.b_in, offsets=off, act="silu", gated=True)
    dt.dt_linear(mid, c.w_out, back, bias=c.b_out, offsets=off)
    dt.dt_moe_combine(back, c.experts, pos, c.weights, far, 8)
    c.run(dt, near, "silu")
    torch.cuda.synchronize()
    want, err = c.reference("silu")
    ref.assert_close(torch.cat(near), want, err, "near")
    ref.assert_close(torch.cat(far), want, 2 * err, "far")


def test_captured_and_replayed_and_on_another_stream(dt):
    """Two captured layers with a workspace each, replayed in turn with new choices in place."""
    note("layer in a graph")
    a, b = (Layer([10, 6], 64, 48, 8, 2, True, torch.bfloat16, seed=s) for s in (8, 9))
    graphs, outs, spaces = [], [], []
    for c in (a, b):
        out = [torch.zeros_like(t) for t in c.x]
        ws = torch.empty(dt.dt_moe_layer_workspace(c.rows, 64, 48, 8, 2, c.dtype), dtype=torch.uint8, device="cuda").fill_(0xFF)
        c.run(dt, out, "silu", workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(dt, out, "silu", workspace=ws)
        graphs.append(graph)
        outs.append(out)
        spaces.append(ws)
    for turn in range(3):
        for c, graph, out in zip((a, b), graphs, outs):
            for e in c.experts:
                e.copy_((e + 1 + turn) % 8)
            graph.replay()
            torch.cuda.synchronize()
            want, err = c.reference("silu")
            ref.assert_close(torch.cat(out), want, err, "replayed")
            other = [torch.zeros_like(t) for t in c.x]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            c.run(dt, other, "silu", stream=side)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, other))
