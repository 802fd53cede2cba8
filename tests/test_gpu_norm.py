"""GPU: layer norm over the ranks' rows, forward and backward, against the
64-bit definition, with canaries around every written buffer."""
import pytest
import torch

import step_reference as ref
import synth
from gpu_util import Guarded, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def _make(rows, cols, dtype, seed, offset=0, scale=1.0, mean=0.0):
    """Inputs per rank; `offset` elements past an aligned start."""
    out = []
    for r, n in enumerate(rows):
        buf = torch.empty(offset + n * cols, dtype=dtype, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed + r)
        buf[offset:] = (torch.randn(n * cols, generator=g, device="cuda") * scale + mean).to(dtype)
        out.append(buf[offset:].view(n, cols))
    return out


def _guards(sizes, dtype, offset=0):
    return [Guarded(n, dtype, offset_elems=offset).poison() for n in sizes]


CASES = [
    # rows per rank, cols, offset
    ([1], 1, 0), ([3], 2, 0), ([1, 0, 5], 7, 0), ([17, 4], 64, 0), ([2, 9, 1, 30], 100, 0), ([5, 3], 511, 0),
    ([4, 4], 1000, 0), ([8, 0, 3], 1001, 0), ([6, 2], 2048, 0), ([5, 5], 2048, 1), ([3, 2], 4096, 0), ([2, 3], 4104, 0),
    ([2, 2], 8192, 0), ([3], 8200, 3), ([2, 1], 11008, 0), ([2], 16385, 0), ([1, 1], 40000, 0), ([300, 411], 96, 0),
    ([7] * 16, 264, 0), ([700, 0, 650], 1024, 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols,offset", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_norm_and_its_gradients(dt, rows, cols, offset, dtype):
    note(f"norm rows={rows} cols={cols} offset={offset} {dtype}")
    p = len(rows)
    x = _make(rows, cols, dtype, 10, offset, scale=2.0, mean=1.5)
    dy = _make(rows, cols, dtype, 40, offset, scale=0.3)
    w = _make([1] * p, cols, dtype, 70, offset, scale=0.2, mean=1.0)
    b = _make([1], cols, dtype, 90, offset)[0].reshape(-1)
    w = [w[0].reshape(-1)] * p
    sizes = [n * cols for n in rows]
    y, mean, rstd = _guards(sizes, dtype, offset), _guards(rows, torch.float32), _guards(rows, torch.float32)
    dt.dt_layer_norm(x, w, [b] * p, [g.t for g in y], [g.t for g in mean], [g.t for g in rstd], eps=1e-5)
    dx, dw, db = _guards(sizes, dtype, offset), _guards([cols] * p, dtype, offset), _guards([cols] * p, dtype, offset)
    dt.dt_layer_norm_backward(dy, x, w, [g.t for g in mean], [g.t for g in rstd], [g.t for g in dx], [g.t for g in dw],
                              [g.t for g in db])
    torch.cuda.synchronize()
    for g in y + mean + rstd + dx + dw + db:
        g.check()
    xs, gs = torch.cat(x), torch.cat(dy)
    ms, rs = torch.cat([g.t for g in mean]), torch.cat([g.t for g in rstd])
    want, err = ref.norm(xs, w[0], b, 1e-5)
    ref.assert_close(torch.cat([g.t for g in y]).view(-1, cols), want[0], err[0], "y")
    ref.assert_close(ms, want[1], err[1], "mean")
    ref.assert_close(rs, want[2], err[2], "rstd")
    want, err = ref.norm_backward(gs, xs, w[0], ms, rs)
    ref.assert_close(torch.cat([g.t for g in dx]).view(-1, cols), want[0], err[0], "dx")
    for q in range(p):
        ref.assert_close(dw[q].t, want[1], err[1], f"dweight[{q}]")
        ref.assert_close(db[q].t, want[2], err[2], f"dbias[{q}]")
        assert torch.equal(dw[q].t, dw[0].t) and torch.equal(db[q].t, db[0].t)


def test_without_bias_and_statistics(dt):
    note("norm without bias")
    x = _make([33, 5], 640, torch.bfloat16, 1)
    w = _make([1], 640, torch.bfloat16, 2)[0].reshape(-1)
    y = [torch.empty_like(t) for t in x]
    dt.dt_layer_norm(x, [w] * 2, None, y, eps=1e-6)
    want, err = ref.norm(torch.cat(x), w, None, 1e-6)
    ref.assert_close(torch.cat(y), want[0], err[0], "y")
    mean = [want[1][:33].float().cuda(), want[1][33:].float().cuda()]
    rstd = [want[2][:33].float().cuda(), want[2][33:].float().cuda()]
    dw = [torch.empty_like(w) for _ in range(2)]
    dx = [torch.empty_like(t) for t in x]
    dt.dt_layer_norm_backward(x, x, [w] * 2, mean, rstd, dx, dw)
    want, err = ref.norm_backward(torch.cat(x), torch.cat(x), w, torch.cat(mean), torch.cat(rstd))
    ref.assert_close(torch.cat(dx), want[0], err[0], "dx")
    ref.assert_close(dw[1], want[1], err[1], "dw")


def test_no_rows_give_zero_gradients(dt):
    note("norm without rows")
    e = [torch.empty(0, 64, device="cuda")] * 2
    s = [torch.empty(0, device="cuda")] * 2
    w = [torch.ones(64, device="cuda")] * 2
    y = dt.dt_layer_norm(e, w, w, e, s, s)
    assert y[0].numel() == 0
    dw, db = [torch.full((64,), 7.0, device="cuda") for _ in range(2)], [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    dt.dt_layer_norm_backward(e, e, w, s, s, e, dw, db)
    torch.cuda.synchronize()
    assert all(bool((t == 0).all()) for t in dw + db)


def test_a_large_mean_costs_no_digits(dt):
    note("norm with a large mean")
    x = _make([64], 2048, torch.float32, 5, scale=1.0, mean=1000.0)
    w = [torch.ones(2048, device="cuda")]
    y = [torch.empty_like(x[0])]
    dt.dt_layer_norm(x, w, None, y)
    want, err = ref.norm(x[0], w[0], None, 1e-5)
    ref.assert_close(y[0], want[0], err[0], "y")
    assert float(err[0].max()) < 0.02  # the bound itself is meaningful here


def test_special_rows(dt):
    note("norm of constant, infinite and NaN rows")
    x = torch.randn(6, 512, device="cuda")
    x[1] = 3.0          # no variance: n = 0
    x[2] = 0.0
    x[3, 7] = float("inf")
    x[4, 9] = float("nan")
    w, b = torch.full((512,), 2.0, device="cuda"), torch.full((512,), 0.5, device="cuda")
    y = torch.empty_like(x)
    dt.dt_layer_norm([x], [w], [b], [y])
    torch.cuda.synchronize()
    assert bool((y[1] == 0.5).all()) and bool((y[2] == 0.5).all())
    assert bool(y[3].isnan().all()) and bool(y[4].isnan().all())
    assert bool(y[0].isfinite().all()) and bool(y[5].isfinite().all())


@pytest.mark.parametrize("cols", [7, 48])
def test_gradients_against_differences(dt, cols):
    """dL for L = sum(y * dy), by central differences of the 64-bit definition."""
    note(f"norm gradients by differences cols={cols}")
    x, dy = torch.randn(3, cols, device="cuda"), torch.randn(3, cols, device="cuda")
    w = torch.randn(cols, device="cuda")
    y, m, r = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dt.dt_layer_norm([x], [w], None, [y], [m], [r])
    dt.dt_layer_norm_backward([dy], [x], [w], [m], [r], [dx], [dw])
    torch.cuda.synchronize()

    def value(xx, ww):
        return float((ref.norm(xx, ww, None, 1e-5)[0][0] * dy.double()).sum())

    h = 1e-5
    for i in range(3):
        for c in range(0, cols, max(1, cols // 7)):
            up, dn = x.double().clone(), x.double().clone()
            up[i, c] += h
            dn[i, c] -= h
            # third derivatives are O(|dy| r^3): h^2 of them and the fp32 kernel's own error stay below 1e-4
            assert abs((value(up, w) - value(dn, w)) / (2 * h) - float(dx[i, c])) < 1e-4
    for c in range(0, cols, max(1, cols // 7)):
        up, dn = w.double().clone(), w.double().clone()
        up[c] += h
        dn[c] -= h
        assert abs((value(x, up) - value(x, dn)) / (2 * h) - float(dw[c])) < 1e-4
