"""GPU: the model-step operators at sizes that take each of their kernels' larger
forms: the loss' tiles with a summed index that goes round the stages several
times, a plan of the exchange with more than 128 workgroups, layer norm with
more rows than workgroups.  The references are 64-bit, on the GPU."""

import pytest
import torch

import step_reference as ref
from gpu_util import Guarded, note

pytestmark = pytest.mark.gpu

U = ref.U


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# -------------------------------------------------------------------- loss --
def _close(got, want, err, what):
    """ref.assert_close on the GPU."""
    got = got.double()
    tol = err + what[1] * (want.abs() + err)
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), f"{what[0]}: {int(bad.sum())} of {bad.numel()} off"


def _loss(dt, tokens, cols, shards, dtype, seed=3):
    g, p, v = _gen(seed), len(shards), sum(shards)
    h = torch.randn(tokens, cols, generator=g, device="cuda").to(dtype)
    w = [(torch.randn(n, cols, generator=g, device="cuda") * (2.0 / cols ** 0.5)).to(dtype) for n in shards]
    t = torch.randint(0, v, (tokens,), generator=g, device="cuda")
    t[::11] = -100
    t[1], t[2] = v - 1, 0
    dl = torch.randn(tokens, generator=g, device="cuda")
    loss, lse = [[Guarded(tokens, torch.float32).poison() for _ in range(p)] for _ in range(2)]
    dh, dw = [Guarded(tokens * cols, dtype).poison() for _ in range(p)], [Guarded(n * cols, dtype).poison() for n in shards]
    dt.dt_vocab_loss([h] * p, w, [t] * p, [x.t for x in loss], [x.t for x in lse])
    dt.dt_vocab_loss_backward([h] * p, w, [t] * p, [x.t for x in lse], [dl] * p, [x.t for x in dh], [x.t for x in dw])
    torch.cuda.synchronize()
    for x in loss + lse + dh + dw:
        x.check()
    # the definitions and bounds of step_reference.loss
    x, wd = h.double(), torch.cat(w).double()
    use = t >= 0
    at = t.clamp(min=0)
    z = x @ wd.t().contiguous()
    ez = (cols + 8) * U * (x.abs() @ wd.abs().t().contiguous())
    l = torch.logsumexp(z, 1)
    spread = (z.amax(1) - z.amin(1)).clamp(max=100.0)
    el = ez.amax(1) + (v / 16.0 + 64 + 2 * spread) * U + 8 * U * l.abs()
    rows = torch.arange(tokens, device="cuda")
    f32, own = ref.half_step(torch.float32), ref.half_step(dtype)
    for q in range(p):
        _close(lse[q].t, l, el, ("lse", f32))
        _close(loss[q].t, torch.where(use, l - z[rows, at], 0.0), torch.where(use, el + ez[rows, at] + 4 * U * z[rows, at].abs(), 0.0), ("loss", f32))
    gr = torch.where(use, dl.double(), 0.0)[:, None]
    d = torch.softmax(z, 1)
    ed = d * (ez + el[:, None] + (8 + 2 * spread[:, None]) * U) * 1.01 * gr.abs()
    del z, ez
    size = d.clone()
    d[rows, at] -= 1.0
    size[rows, at] += 1.0
    d *= gr
    ed += 4 * U * size * gr.abs() + 1e-40
    del size
    if dtype == torch.bfloat16:
        ed = ed + own * (d.abs() + ed)
    want, err = d @ wd, ed @ wd.abs() + (v + 8) * U * (d.abs() @ wd.abs())
    for q in range(p):
        _close(dh[q].t.view(tokens, cols), want, err, ("dhidden", own))
    d, ed = d.t().contiguous(), ed.t().contiguous()
    want, err = d @ x, ed @ x.abs() + (tokens + 8) * U * (d.abs() @ x.abs())
    first = 0
    for q, n in enumerate(shards):
        _close(dw[q].t.view(n, cols), want[first:first + n], err[first:first + n], (f"dweight[{q}]", own))
        first += n


@pytest.mark.parametrize("tokens,cols,shards", [
    # 128 x 64 tiles: logits of 17 to 64 tokens, rows on 16-byte boundaries and off them; dhidden; dweight in one and two parts
    (48, 72, [9000, 0, 8001]), (48, 70, [17001]), (33, 16392, [120, 81]), (600, 16392, [50]), (33, 16390, [11, 39]),
    # 256 x 256 tiles: logits with d in one part and in two; dweight in two
    (600, 296, [10000, 9300]), (600, 300, [19300]), (300, 296, [28800]), (300, 300, [15000, 1, 13799]),
    # 256 x 256 tiles: dhidden and dweight, in one part and in two; logits in 128 x 128 tiles
    (2100, 6496, [1200, 1000]), (2100, 6500, [2200]), (500, 28700, [300, 200]),
    # 128 x 128 tiles: logits and dweight in two parts
    (500, 520, [6250]), (500, 522, [3125, 3125]),
], ids=str)
def test_bf16_loss_tiles(dt, tokens, cols, shards):
    note(f"loss tiles bf16 {tokens} x {cols}, {shards}")
    _loss(dt, tokens, cols, shards, torch.bfloat16)


@pytest.mark.parametrize("cols", [4100, 4097])
def test_fp32_loss_tiles(dt, cols):
    """33 x 33 tiles of 128 x 128 in all four products, rows on 16-byte boundaries and off them."""
    note(f"loss tiles fp32, {cols} columns")
    _loss(dt, 4099, cols, [2101, 2099], torch.float32)


# ---------------------------------------------------------------- exchange --
@pytest.mark.parametrize("rows,e,k,room", [([40000, 30001], 64, 2, 2.0), ([70000, 0, 1, 30000], 1000, 2, 0.9), ([150000], 8, 1, 1.0),
                                           ([44001] * 3, 96, 4, 1.1)], ids=str)
def test_a_plan_of_many_workgroups(dt, rows, e, k, room):
    """More than 131072 slots: the counts of the plan's workgroups are summed by a launch of their own."""
    note(f"plan of {sum(rows) * k} slots, {e} experts")
    p, cols, g = len(rows), 4, _gen(7)
    per, slots = e // p, sum(rows) * k
    assert slots > 131072
    cap = int(slots / p * room)
    lean = (torch.rand(e, generator=g, device="cuda") + 0.1).cumsum(0)
    ex = []
    for n in rows:
        x = torch.searchsorted(lean, torch.rand(n, k, generator=g, device="cuda") * lean[-1]).clamp(max=e - 1).to(torch.int32)
        x[torch.rand(n, k, generator=g, device="cuda") < 0.03] = -1
        ex.append(x)
    x = [torch.randint(-2 ** 31, 2 ** 31 - 1, (n, cols), generator=g, device="cuda", dtype=torch.int32) for n in rows]
    recv = [Guarded(cap * cols, torch.int32).poison() for _ in range(p)]
    pos = [Guarded(n * k, torch.int32).poison() for n in rows]
    off = [Guarded(per + 1, torch.int32).poison() for _ in range(p)]
    dt.dt_moe_dispatch(x, ex, [t.t for t in recv], [t.t for t in pos], [t.t for t in off], e)
    torch.cuda.synchronize()
    for t in recv + pos + off:
        t.check()
    flat, got = torch.cat(ex).reshape(-1), torch.cat([t.t for t in pos])
    token = torch.cat(x).repeat_interleave(k, 0)
    for q in range(p):
        mine = (flat // per == q) & (flat >= 0)
        at = mine.nonzero().reshape(-1)
        at = at[flat[at].sort(stable=True).indices][:cap]
        want = torch.full_like(flat, -1)
        want[at] = torch.arange(at.numel(), device="cuda", dtype=torch.int32)
        assert torch.equal(got[mine], want[mine]), f"positions of rank {q}"
        n = torch.bincount(flat[mine] - q * per, minlength=per).cumsum(0).clamp(max=cap)
        assert off[q].t.tolist() == [0] + n.tolist(), f"offsets[{q}]"
        rows_q = recv[q].t.view(cap, cols)
        assert torch.equal(rows_q[:at.numel()], token[at]), f"recv[{q}]"
        assert bool((rows_q[at.numel():].contiguous().view(torch.uint8) == 0xFF).all())
    assert bool((got[flat < 0] == -1).all())


# -------------------------------------------------------------- layer norm --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols,offset", [
    ([60000, 0, 1, 90000], 40, 0), ([140000], 37, 1),     # 16 lanes to a row, above 65536 rows
    ([9000, 0, 12001], 256, 0), ([18000, 500], 251, 0),   # a wave to a row, above 16384 rows
    ([4000, 2, 3000], 1024, 0), ([6001], 1023, 1),        # four waves, above 4096 rows
    ([300, 0, 0, 900], 4104, 0), ([1100], 4111, 0),       # four units a lane (bf16), above 512 rows
    ([4200, 300], 1504, 0), ([2100, 2300], 3001, 0),      # four waves with one and two units a lane (bf16), above 4096 rows
    ([700, 500], 16384, 0), ([1, 800], 16377, 0),         # sixteen waves, above 512 rows
    ([300, 301], 20000, 0), ([530], 20001, 1),            # four units a lane (bf16); too wide for the registers (fp32)
], ids=str)
def test_more_rows_than_workgroups(dt, rows, cols, offset, dtype):
    note(f"norm loops rows={rows} cols={cols} offset={offset} {dtype}")
    p, g, n = len(rows), _gen(9), sum(rows)

    def make(scale, mean):
        out = []
        for r in rows:
            t = torch.empty(offset + r * cols, dtype=dtype, device="cuda")
            t[offset:] = (torch.randn(r * cols, generator=g, device="cuda") * scale + mean).to(dtype)
            out.append(t[offset:].view(r, cols))
        return out

    x, dy = make(2.0, 0.5), make(0.3, 0.0)
    w = (torch.randn(cols, generator=g, device="cuda") * 0.2 + 1).to(dtype)
    b = torch.randn(cols, generator=g, device="cuda").to(dtype)
    guards = lambda sizes, kind: [Guarded(s, kind).poison() for s in sizes]
    sizes = [r * cols for r in rows]
    y, mean, rstd = guards(sizes, dtype), guards(rows, torch.float32), guards(rows, torch.float32)
    dx, dw, db = guards(sizes, dtype), guards([cols] * p, dtype), guards([cols] * p, dtype)
    dt.dt_layer_norm(x, [w] * p, [b] * p, [t.t for t in y], [t.t for t in mean], [t.t for t in rstd])
    dt.dt_layer_norm_backward(dy, x, [w] * p, [t.t for t in mean], [t.t for t in rstd], [t.t for t in dx], [t.t for t in dw], [t.t for t in db])
    torch.cuda.synchronize()
    for t in y + mean + rstd + dx + dw + db:
        t.check()
    xs, gs = torch.cat(x), torch.cat(dy)
    ms, rs = torch.cat([t.t for t in mean]), torch.cat([t.t for t in rstd])
    f32, own = ref.half_step(torch.float32), ref.half_step(dtype)
    want, err = ref.norm(xs, w, b, 1e-5)
    _close(torch.cat([t.t for t in y]).view(n, cols), want[0], err[0], ("y", own))
    _close(ms, want[1], err[1], ("mean", f32))
    _close(rs, want[2], err[2], ("rstd", f32))
    want, err = ref.norm_backward(gs, xs, w, ms, rs)
    _close(torch.cat([t.t for t in dx]).view(n, cols), want[0], err[0], ("dx", own))
    for q in range(p):
        _close(dw[q].t, want[1], err[1], ("dweight", own))
        _close(db[q].t, want[2], err[2], ("dbias", own))
