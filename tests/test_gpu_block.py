"""GPU: the norms after and before a block with its gate and residual, forward
and backward, against the 64-bit definition, with canaries around every written
buffer."""
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


class Block:
    """post, pre: is the norm there; gate: "none", "channel" or "row"."""

    def __init__(self, rows, cols, dtype, post=True, pre=True, bias=True, gate="channel", rms=False, scale=1.0, offset=0, seed=0, mean=0.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.cols, self.dtype, self.post, self.pre, self.bias, self.gate_kind, self.rms, self.scale, self.at = (
            rows, cols, dtype, post, pre, bias, gate, rms, scale, offset)
        self.p = len(rows)

        def new(n, std=1.0, at=0.0):
            buf = torch.empty(offset + n, dtype=dtype, device="cuda")
            buf[offset:] = (torch.randn(n, generator=g, device="cuda") * std + at).to(dtype)
            return buf[offset:]

        self.row = lambda std=1.0, at=0.0: [new(n * cols, std, at).view(n, cols) for n in rows]
        self.z, self.x = self.row(2.0, mean), self.row(1.5, -mean)
        same = lambda there, std, at: [new(cols, std, at)] * self.p if there else None
        self.w1, self.b1 = same(post, 0.2, 1.0), same(post and bias, 0.3, 0.0)
        self.w2, self.b2 = same(pre, 0.2, 1.0), same(pre and bias, 0.3, 0.0)
        self.gate = None if gate == "none" else same(True, 0.5, 0.5) if gate == "channel" else self.row(0.7, 0.2)
        self.dy, self.dh, self.h = self.row(0.3) if pre else None, self.row(0.3), self.row(2.0, mean)

    def guards(self, sizes, dtype=None):
        dtype = dtype or self.dtype
        return [Guarded(n, dtype, offset_elems=self.at if dtype == self.dtype else 0).poison() for n in sizes]

    def every_gate(self):
        return None if self.gate is None else self.gate[0] if self.gate_kind == "channel" else torch.cat(self.gate)

    def forward(self, dt, eps=1e-5):
        sizes = [n * self.cols for n in self.rows]
        h, y, stats = self.guards(sizes), self.guards(sizes) if self.pre else None, self.guards([4 * n for n in self.rows], torch.float32)
        t = lambda gs: None if gs is None else [g.t for g in gs]
        dt.dt_block_norm(self.z, self.x, t(h), t(y), gate=self.gate, scale=self.scale, post_weight=self.w1, post_bias=self.b1,
                         pre_weight=self.w2, pre_bias=self.b2, stats=t(stats), rms=self.rms, eps=eps)
        torch.cuda.synchronize()
        got = dict(h=h, stats=stats, **(dict(y=y) if self.pre else {}))
        first = lambda v: None if v is None else v[0]
        want = ref.block(torch.cat(self.z), torch.cat(self.x), self.every_gate(), first(self.w1), first(self.b1), first(self.w2), first(self.b2),
                         self.scale, self.rms, eps)
        for name, gs in got.items():
            for g in gs:
                g.check()
            ref.assert_close(torch.cat([g.t for g in gs]).view(want[name][0].shape), *want[name], name)

    def stats_of(self, eps=1e-5):
        def moments(v):
            v = v.double()
            m = torch.zeros_like(v[:, :1]) if self.rms else v.mean(1, keepdim=True)
            return [m, 1 / torch.sqrt((v - m).square().mean(1, keepdim=True) + eps)]
        return [torch.cat(moments(z) + moments(h), 1).float() for z, h in zip(self.z, self.h)]

    def backward(self, dt, past=True, wanted=True):
        sizes, wide = [n * self.cols for n in self.rows], [self.cols] * self.p
        stats, dh = self.stats_of(), self.dh if past else None
        dz, dx = self.guards(sizes), self.guards(sizes)
        sums = {}
        if wanted:
            if self.post:
                sums["dpost_weight"] = self.guards(wide)
                if self.bias:
                    sums["dpost_bias"] = self.guards(wide)
            if self.pre:
                sums["dpre_weight"] = self.guards(wide)
                if self.bias:
                    sums["dpre_bias"] = self.guards(wide)
            if self.gate is not None:
                sums["dgate"] = self.guards(wide if self.gate_kind == "channel" else sizes)
        t = lambda gs: None if gs is None else [g.t for g in gs]
        need_z = self.post or "dgate" in sums
        dt.dt_block_norm_backward(self.dy, dh, self.z if need_z else None, self.h if self.pre else None, stats, t(dz), t(dx), gate=self.gate,
                                  scale=self.scale, post_weight=self.w1, post_bias=self.b1, pre_weight=self.w2, rms=self.rms,
                                  **{k: t(v) for k, v in sums.items()})
        torch.cuda.synchronize()
        cat = lambda v: None if v is None else torch.cat(v)
        first = lambda v: None if v is None else v[0]
        want = ref.block_backward(cat(self.dy), cat(dh), cat(self.z), cat(self.h), self.every_gate(), first(self.w1), first(self.b1),
                                  first(self.w2), torch.cat(stats), self.scale, self.rms)
        for gs in [dz, dx, *sums.values()]:
            for g in gs:
                g.check()
        ref.assert_close(torch.cat(t(dx)).view(-1, self.cols), *want["dx"], "dx")
        ref.assert_close(torch.cat(t(dz)).view(-1, self.cols), *want["dz"], "dz")
        for name, gs in sums.items():
            if name == "dgate" and self.gate_kind == "row":
                ref.assert_close(torch.cat(t(gs)).view(-1, self.cols), *want["dgate"], name)
                continue
            for q, g in enumerate(gs):
                ref.assert_close(g.t, *want["dgate_sum" if name == "dgate" else name], f"{name}[{q}]")
                assert torch.equal(g.t, gs[0].t)


SHAPES = [
    # rows per rank, cols, elements past an aligned start
    ([1], 1, 0), ([3], 2, 0), ([1, 0, 5], 7, 0), ([17, 4], 64, 0), ([2, 9, 1, 30], 100, 0), ([5, 3], 511, 0), ([4, 4], 1000, 0),
    ([8, 0, 3], 1001, 0), ([6, 2], 2048, 0), ([5, 5], 2048, 1), ([3, 2], 4096, 0), ([2, 3], 4104, 0), ([2, 2], 8192, 0), ([3], 8200, 3),
    ([2, 1], 11008, 0), ([2], 16385, 0), ([1, 1], 40000, 0), ([300, 411], 96, 0), ([7] * 16, 264, 0), ([700, 0, 650], 1024, 0),
]


@DTYPES
@pytest.mark.parametrize("rows,cols,offset", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_shapes(dt, rows, cols, offset, dtype):
    note(f"block rows={rows} cols={cols} offset={offset} {dtype}")
    for rms, gate in ((False, "channel"), (True, "row")):
        b = Block(rows, cols, dtype, gate=gate, rms=rms, scale=0.5, offset=offset, bias=not rms)
        b.forward(dt)
        b.backward(dt)


@DTYPES
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("post,pre,bias", [(True, True, False), (True, False, True), (False, True, True), (False, True, False)])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_forms(dt, post, pre, bias, gate, rms, dtype):
    """Every norm that may be missing, each gate, with and without what reaches h past y, in rows of registers and wide ones."""
    note(f"block post={post} pre={pre} bias={bias} gate={gate} rms={rms} {dtype}")
    for cols in (72, 1500, 20000):
        b = Block([5, 3], cols, dtype, post, pre, bias, gate, rms, scale=-0.75, seed=1)
        b.forward(dt)
        b.backward(dt)
        if pre:
            b.backward(dt, past=False)
        b.backward(dt, wanted=False)


def test_many_rows(dt):
    note("block with more rows than workgroups")
    for dtype, cols in ((torch.bfloat16, 520), (torch.float32, 129), (torch.bfloat16, 2056), (torch.bfloat16, 4104)):
        b = Block([2500, 1, 3001], cols, dtype, seed=2)
        b.forward(dt)
        b.backward(dt)


def test_a_large_mean_costs_no_digits(dt):
    note("block with a large mean")
    Block([40], 2048, torch.float32, seed=3, mean=1000.0).forward(dt)


def test_special_rows(dt):
    note("block of constant, infinite and NaN rows")
    b = Block([6], 512, torch.float32, gate="none", seed=4)
    b.z[0][1], b.z[0][2, 5], b.z[0][3, 7] = 3.0, float("inf"), float("nan")
    b.x[0][4, 9] = float("nan")
    h, y = [torch.zeros_like(b.z[0])], [torch.zeros_like(b.z[0])]
    dt.dt_block_norm(b.z, b.x, h, y, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, pre_bias=b.b2)
    torch.cuda.synchronize()
    assert torch.equal(h[0][1], b.x[0][1] + b.b1[0])   # no variance: the bias alone
    assert bool(h[0][2].isnan().all()) and bool(h[0][3].isnan().all())
    assert int(h[0][4].isnan().sum()) == 1 and bool(y[0][4].isnan().all())
    assert bool(y[0][0].isfinite().all()) and bool(y[0][1].isfinite().all()) and bool(y[0][5].isfinite().all())


def test_gradients_against_differences(dt):
    """dL for L = sum(y * dy) + sum(h * dh), by central differences of the 64-bit definition, through both norms."""
    note("block gradients by differences")
    for rms, gate in ((False, "channel"), (True, "row")):
        b = Block([2, 1], 24, torch.float32, gate=gate, rms=rms, scale=0.7, seed=6)
        like = lambda ts: [torch.empty_like(t) for t in ts]
        h, y, stats = like(b.z), like(b.z), [torch.empty(n, 4, device="cuda") for n in b.rows]
        dt.dt_block_norm(b.z, b.x, h, y, gate=b.gate, scale=b.scale, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, pre_bias=b.b2,
                         stats=stats, rms=rms)
        got = dict(z=like(b.z), x=like(b.x), gate=like(b.gate), w1=like(b.w1), b1=like(b.b1), w2=like(b.w2), b2=like(b.b2))
        dt.dt_block_norm_backward(b.dy, b.dh, b.z, h, stats, got["z"], got["x"], gate=b.gate, scale=b.scale, post_weight=b.w1,
                                  post_bias=b.b1, pre_weight=b.w2, dgate=got["gate"], dpost_weight=got["w1"], dpost_bias=got["b1"],
                                  dpre_weight=got["w2"], dpre_bias=got["b2"], rms=rms)
        torch.cuda.synchronize()
        at = dict(z=torch.cat(b.z).double(), x=torch.cat(b.x).double(), gate=b.every_gate().double(), w1=b.w1[0].double(), b1=b.b1[0].double(),
                  w2=b.w2[0].double(), b2=b.b2[0].double())

        def value(v):
            out = ref.block(v["z"], v["x"], v["gate"], v["w1"], v["b1"], v["w2"], v["b2"], b.scale, rms, 1e-5)
            return float((out["y"][0] * torch.cat(b.dy).double()).sum() + (out["h"][0] * torch.cat(b.dh).double()).sum())

        for name, ts in got.items():
            whole = torch.cat(ts).reshape(-1) if at[name].dim() > 1 else ts[0].reshape(-1)
            for i in range(0, whole.numel(), 5):
                up, dn = dict(at), dict(at)
                for v, s in ((up, 1e-5), (dn, -1e-5)):
                    v[name] = at[name].clone()
                    v[name].view(-1)[i] += s
                # third derivatives are O(1): 1e-10 of them, and the fp32 kernels' own error of some 100 U of sums of about 10
                assert abs((value(up) - value(dn)) / 2e-5 - float(whole[i])) < 2e-4, (name, i)


def test_no_rows_give_zero_gradients(dt):
    note("block without rows")
    for cols in (64, 20000):
        e, s = [torch.empty(0, cols, device="cuda")] * 2, [torch.empty(0, 4, device="cuda")] * 2
        w = [torch.ones(cols, device="cuda")] * 2
        assert dt.dt_block_norm(e, e, e, e, gate=w, post_weight=w, pre_weight=w, stats=s)[0].numel() == 0
        g = [[torch.full((cols,), 7.0, device="cuda") for _ in range(2)] for _ in range(3)]
        dt.dt_block_norm_backward(e, e, e, e, s, e, e, gate=w, post_weight=w, pre_weight=w, dgate=g[0], dpost_weight=g[1], dpre_weight=g[2])
        torch.cuda.synchronize()
        assert all(bool((t == 0).all()) for ts in g for t in ts)


def test_it_is_layer_norm_without_gate_and_scale(dt):
    """y of h = x + z is dt_layer_norm of the sum, bit for bit where the sum is exact."""
    note("block against layer norm")
    z, x = [torch.randint(-8, 9, (33, 640), device="cuda").float()], [torch.randint(-8, 9, (33, 640), device="cuda").float()]
    w, b = [torch.randn(640, device="cuda")], [torch.randn(640, device="cuda")]
    h, y, other = ([torch.empty_like(z[0])] for _ in range(3))
    dt.dt_block_norm(z, x, h, y, pre_weight=w, pre_bias=b)
    dt.dt_layer_norm([z[0] + x[0]], w, b, other)
    torch.cuda.synchronize()
    assert torch.equal(h[0], z[0] + x[0])
    want = ref.block(z[0], x[0], None, None, None, w[0], b[0], 1.0, False, 1e-5)["y"]
    ref.assert_close(y[0], *want, "y")
    ref.assert_close(other[0], *want, "layer norm")


def test_captured_and_replayed_and_on_another_stream(dt):
    note("block in a graph")
    b = Block([40, 25], 512, torch.bfloat16, seed=7)
    like = lambda ts: [torch.zeros_like(t) for t in ts]
    y, stats = like(b.z), [torch.zeros(n, 4, device="cuda") for n in b.rows]
    h, dz, dx = like(b.z), like(b.z), like(b.z)
    every = lambda: [torch.zeros(512, dtype=b.dtype, device="cuda") for _ in b.rows]
    dg, dw1, db1, dw2, db2 = every(), every(), every(), every(), every()
    outs = h + y + stats + dz + dx + dg + dw1 + db1 + dw2 + db2
    ws = torch.empty(dt.dt_block_norm_workspace(b.rows, 512, b.dtype), dtype=torch.uint8, device="cuda")

    def step(**kw):
        dt.dt_block_norm(b.z, b.x, h, y, gate=b.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, pre_bias=b.b2, stats=stats, **kw)
        dt.dt_block_norm_backward(b.dy, b.dh, b.z, h, stats, dz, dx, gate=b.gate, post_weight=b.w1, post_bias=b.b1, pre_weight=b.w2, dgate=dg,
                                  dpost_weight=dw1, dpost_bias=db1, dpre_weight=dw2, dpre_bias=db2, workspace=ws, **kw)

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
        assert all(torch.equal(u, v) for u, v in zip(outs, want))
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    step(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(outs, want))
