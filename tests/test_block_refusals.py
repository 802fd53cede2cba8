"""CPU: the expert block's entry points refuse what they cannot do, with a status
and a message, before anything is queued (the pointers here are not memory), and
the binding refuses lists that are not one tensor per rank."""
import ctypes
import types

import pytest
import torch

import collective_communication_primitives_amd as dt

ARG, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from collective_communication_primitives_amd import _lib
    return _lib.load()


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*v)


def sizes(*v):
    return (ctypes.c_size_t * len(v))(*v)


A, B, C, D, E, F, G, H, W, I, J, K, L, M, N, O, P, Q = (0x100000 * i for i in range(1, 19))
two = lambda at: ptrs(at, at + 4096)


def call(fn, defaults, order, kw):
    a = dict(defaults)
    a.update(kw)
    return fn(*[a[k] for k in order.split()], None)


def linear(lib, **kw):
    return call(lib.dt_linear, dict(x=two(A), w=two(B), b=two(C), r=two(D), o=two(E), y=two(F), pre=two(G), p=2, rows=sizes(4, 5), runs=2, cols=8,
                                    outs=6, act=3, gated=0, dtype=0), "x w b r o y pre p rows runs cols outs act gated dtype", kw)


def linear_back(lib, **kw):
    return call(lib.dt_linear_backward, dict(dy=two(A), x=two(B), w=two(C), pre=two(D), o=two(E), dx=two(F), dw=two(G), db=two(H), p=2, rows=sizes(4, 5),
                                             runs=2, cols=8, outs=6, act=3, gated=0, dtype=0, ws=W, n=1 << 16),
                "dy x w pre o dx dw db p rows runs cols outs act gated dtype ws n", kw)


def layer(lib, **kw):
    return call(lib.dt_moe_layer, dict(x=two(A), e=two(B), g=two(C), wi=two(D), bi=two(E), wo=two(F), bo=two(G), r=two(H), out=two(I), p=2, n=sizes(4, 5),
                                       cols=8, inner=6, ne=4, k=2, act=3, gated=1, dtype=0, ws=W, wn=1 << 16),
                "x e g wi bi wo bo r out p n cols inner ne k act gated dtype ws wn", kw)


def block(lib, **kw):
    return call(lib.dt_block_norm, dict(z=two(A), x=two(B), g=two(C), w1=two(D), b1=two(E), w2=two(F), b2=two(G), h=two(H), y=two(I), s=two(J), p=2,
                                        rows=sizes(4, 5), cols=8, per=0, scale=1.0, rms=0, eps=1e-5, dtype=0),
                "z x g w1 b1 w2 b2 h y s p rows cols per scale rms eps dtype", kw)


def block_back(lib, **kw):
    return call(lib.dt_block_norm_backward, dict(dy=two(A), dh=two(B), z=two(C), h=two(D), g=two(E), w1=two(F), b1=two(G), w2=two(H), s=two(I), dz=two(J),
                                                 dx=two(K), dg=two(L), dw1=two(M), db1=two(N), dw2=two(O), db2=two(P), p=2, rows=sizes(4, 5), cols=8,
                                                 per=0, scale=1.0, rms=0, dtype=0, ws=Q, n=1 << 16),
                "dy dh z h g w1 b1 w2 s dz dx dg dw1 db1 dw2 db2 p rows cols per scale rms dtype ws n", kw)


NAN = float("nan")


@pytest.mark.parametrize("fn,kw,status,word", [
    (linear, dict(p=0), ARG, "nranks"), (linear, dict(p=17), ARG, "nranks"), (linear, dict(dtype=2), UNSUPPORTED, "int32"),
    (linear, dict(dtype=9), ARG, "dtype"), (linear, dict(rows=None), ARG, "rows"), (linear, dict(rows=sizes(1 << 30, 0)), ARG, "rows"),
    (linear, dict(cols=0), ARG, "cols"), (linear, dict(cols=1 << 19), ARG, "cols"), (linear, dict(outs=0), ARG, "outs"),
    (linear, dict(outs=1 << 19), ARG, "outs"), (linear, dict(act=4), ARG, "act"), (linear, dict(act=-1), ARG, "act"), (linear, dict(runs=0), ARG, "runs"),
    (linear, dict(runs=513), ARG, "runs"), (linear, dict(o=None), ARG, "offsets"), (linear, dict(o=ptrs(E, 0)), ARG, "offsets[1]"),
    (linear, dict(x=None), ARG, "x is NULL"), (linear, dict(y=ptrs(0, F)), ARG, "y[0]"), (linear, dict(w=ptrs(B, B + 2)), ARG, "aligned"),
    (linear, dict(y=two(A)), ARG, "overlap"), (linear, dict(y=two(D)), ARG, "overlap"), (linear, dict(y=ptrs(F, F + 16)), ARG, "overlap"),
    (linear, dict(pre=two(F)), ARG, "overlap"), (linear, dict(y=ptrs(E + 8, F)), ARG, "overlap"), (linear, dict(b=ptrs(0, C)), ARG, "bias[0]"),
    (linear, dict(cols=1 << 18, outs=1 << 11, dtype=0), ARG, "2 GiB"), (linear, dict(cols=1 << 18, outs=1 << 11, gated=1, dtype=1), ARG, "2 GiB"),
    (linear_back, dict(p=-1), ARG, "nranks"), (linear_back, dict(dtype=2), UNSUPPORTED, "int32"), (linear_back, dict(pre=None), ARG, "pre"),
    (linear_back, dict(pre=None, act=0, gated=1), ARG, "pre"), (linear_back, dict(n=64), ARG, "workspace"), (linear_back, dict(ws=W + 64), ARG, "256"),
    (linear_back, dict(ws=0), ARG, "workspace"), (linear_back, dict(dx=two(B)), ARG, "overlap"), (linear_back, dict(dw=two(C)), ARG, "overlap"),
    (linear_back, dict(db=ptrs(H, H)), ARG, "overlap"), (linear_back, dict(ws=F), ARG, "overlap"), (linear_back, dict(dw=None), ARG, "dweight"),
    (linear_back, dict(o=None), ARG, "offsets"), (linear_back, dict(runs=600), ARG, "runs"), (linear_back, dict(act=7), ARG, "act"),
    (layer, dict(p=3), ARG, "divide"), (layer, dict(n=sizes(200, 57)), ARG, "tokens"), (layer, dict(dtype=2), UNSUPPORTED, "int32"),
    (layer, dict(cols=0), ARG, "cols"), (layer, dict(inner=0), ARG, "inner"), (layer, dict(inner=1 << 19), ARG, "inner"), (layer, dict(k=5), ARG, "topk"),
    (layer, dict(ne=0), ARG, "nexperts"), (layer, dict(act=5), ARG, "act"), (layer, dict(wn=32), ARG, "workspace"), (layer, dict(out=two(A)), ARG, "overlap"),
    (layer, dict(out=two(H)), ARG, "overlap"), (layer, dict(out=ptrs(I, I)), ARG, "overlap"), (layer, dict(ws=I), ARG, "overlap"),
    (layer, dict(wi=None), ARG, "w_in"), (layer, dict(wo=ptrs(F, 0)), ARG, "w_out[1]"), (layer, dict(g=ptrs(C + 1, C)), ARG, "aligned"),
    (layer, dict(cols=1 << 18, inner=1 << 12), ARG, "2 GiB"),
    (block, dict(w1=None, b1=None, w2=None, b2=None, y=None), ARG, "neither"), (block, dict(w1=None), ARG, "post_bias"), (block, dict(w2=None, y=None), ARG, "pre_bias"),
    (block, dict(y=None), ARG, "y and pre_weight"), (block, dict(w2=None, b2=None), ARG, "y and pre_weight"), (block, dict(g=None, per=1), ARG, "gate_per_row"),
    (block, dict(scale=NAN), ARG, "scale"), (block, dict(scale=float("inf")), ARG, "scale"), (block, dict(eps=-1.0), ARG, "eps"), (block, dict(eps=NAN), ARG, "eps"),
    (block, dict(dtype=2), UNSUPPORTED, "int32"), (block, dict(cols=0), ARG, "cols"), (block, dict(h=two(B)), ARG, "overlap"), (block, dict(h=two(A)), ARG, "overlap"),
    (block, dict(y=two(H)), ARG, "overlap"), (block, dict(s=two(H)), ARG, "overlap"), (block, dict(z=ptrs(A, 0)), ARG, "z[1]"), (block, dict(rows=None), ARG, "rows"),
    (block_back, dict(dy=None), ARG, "dy and pre_weight"), (block_back, dict(w2=None), ARG, "dy and pre_weight"),
    (block_back, dict(w2=None, dy=None), ARG, "not there"), (block_back, dict(w1=None, b1=None), ARG, "not there"), (block_back, dict(g=None), ARG, "dgate"),
    (block_back, dict(z=None), ARG, "z is NULL"), (block_back, dict(h=None), ARG, "h is NULL"), (block_back, dict(s=None), ARG, "stats"),
    (block_back, dict(dx=two(B)), ARG, "overlap"), (block_back, dict(dz=two(K)), ARG, "overlap"), (block_back, dict(dw1=ptrs(M, M)), ARG, "overlap"),
    (block_back, dict(n=8), ARG, "workspace"), (block_back, dict(ws=L), ARG, "overlap"), (block_back, dict(dtype=2), UNSUPPORTED, "int32"),
    (block_back, dict(scale=NAN), ARG, "scale"),
])
def test_refused(lib, fn, kw, status, word):
    assert fn(lib, **kw) == status
    assert word in lib.dt_last_error().decode()


def test_workspace_sizes_refuse_like_the_calls(lib):
    assert lib.dt_linear_backward_workspace(0, sizes(1), 1, 4, 3, 0, 1, 0) == 0 and lib.dt_last_error()
    assert lib.dt_linear_backward_workspace(1, sizes(1), 1, 4, 9, 0, 1, 0) == 0 and lib.dt_last_error()
    assert lib.dt_linear_backward_workspace(1, sizes(9), 1, 4, 0, 0, 0, 0) == 0 and not lib.dt_last_error()   # dz is dy, and no sums
    small, large = (lib.dt_linear_backward_workspace(1, sizes(n), 1, 40, 3, 1, 1, 1) for n in (100, 1000))
    assert 0 < small < large
    assert lib.dt_moe_layer_workspace(1, sizes(257), 8, 8, 4, 2, 0) == 0 and lib.dt_last_error()
    assert lib.dt_moe_layer_workspace(1, sizes(0), 8, 8, 4, 2, 0) == 0 and not lib.dt_last_error()
    assert lib.dt_moe_layer_workspace(1, sizes(7), 8, 8, 4, 2, 0) > 0
    assert lib.dt_block_norm_workspace(1, sizes(4), 8, 2) == 0 and lib.dt_last_error()
    assert lib.dt_block_norm_workspace(1, sizes(4), 8, 1) > 0


def test_calls_without_rows_do_nothing(lib):
    none = ptrs(0, 0)
    assert linear(lib, rows=sizes(0, 0), x=none, w=none, b=none, r=none, o=none, y=none, pre=none) == 0
    assert layer(lib, n=sizes(0, 0)) == 0
    assert block(lib, rows=sizes(0, 0), z=none, x=none, h=none, y=none) == 0


# ---------------------------------------------------------------- the binding --
R = 3


@pytest.fixture
def reached(monkeypatch):
    """The names of the library's functions that were called; CPU tensors pass for the GPU's."""
    calls = []

    def entry(name):
        def run(*args):
            calls.append(name)
            return 256 if name.endswith("_workspace") else 0
        return run

    monkeypatch.setattr(dt, "_L", types.SimpleNamespace(**{n: entry(n) for n in dt._lib.EXPORTS}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(dt, "_current_stream_handle", lambda: 0)
    monkeypatch.setattr(dt, "_workspace", lambda *a: torch.empty(256, dtype=torch.uint8))
    return calls


def tensors(*shape, dtype=torch.float32, n=R):
    return [torch.zeros(*shape, dtype=dtype) for _ in range(n)]


i32 = torch.int32
LINEAR = dict(x=tensors(4, 8), weight=tensors(2, 6, 8), y=tensors(4, 6), bias=tensors(2, 6), residual=tensors(4, 6), pre=tensors(4, 6), offsets=tensors(3, dtype=i32))
LINEAR_BACK = dict(dy=tensors(4, 6), x=tensors(4, 8), weight=tensors(2, 6, 8), dx=tensors(4, 8), dweight=tensors(2, 6, 8), pre=tensors(4, 6), dbias=tensors(2, 6),
                   offsets=tensors(3, dtype=i32))
LAYER = dict(x=tensors(4, 8), experts=tensors(4, 2, dtype=i32), weights=tensors(4, 2), w_in=tensors(2, 12, 8), w_out=tensors(2, 8, 6), out=tensors(4, 8),
             b_in=tensors(2, 12), b_out=tensors(2, 8), residual=tensors(4, 8))
BLOCK = dict(z=tensors(4, 8), x=tensors(4, 8), h=tensors(4, 8), y=tensors(4, 8), gate=tensors(8), post_weight=tensors(8), post_bias=tensors(8),
             pre_weight=tensors(8), pre_bias=tensors(8), stats=tensors(4, 4))
BLOCK_BACK = dict(dy=tensors(4, 8), dh=tensors(4, 8), z=tensors(4, 8), h=tensors(4, 8), stats=tensors(4, 4), dz=tensors(4, 8), dx=tensors(4, 8), gate=tensors(8),
                  post_weight=tensors(8), post_bias=tensors(8), pre_weight=tensors(8), dgate=tensors(8), dpost_weight=tensors(8), dpost_bias=tensors(8),
                  dpre_weight=tensors(8), dpre_bias=tensors(8))
CALLS = dict(dt_linear=LINEAR, dt_linear_backward=LINEAR_BACK, dt_moe_layer=LAYER, dt_block_norm=BLOCK, dt_block_norm_backward=BLOCK_BACK)


@pytest.mark.parametrize("name,which", [(n, k) for n, kw in CALLS.items() for k in kw])
def test_every_list_has_one_tensor_per_rank(reached, name, which):
    fn, kw = getattr(dt, name), CALLS[name]
    fn(**kw)
    assert reached[-1] == name
    for bad in (kw[which][:-1], kw[which] + kw[which][:1], kw[which][:-1] + [None], kw[which][:-1] + [kw[which][0].double()],
                kw[which][:-1] + [torch.zeros(5, dtype=kw[which][0].dtype)]):
        reached.clear()
        with pytest.raises((ValueError, TypeError)):
            fn(**dict(kw, **{which: bad}))
        assert name not in reached


@pytest.mark.parametrize("name,kw", [
    ("dt_linear", dict(weight=tensors(6, 8))), ("dt_linear", dict(weight=tensors(2, 6, 9))), ("dt_linear", dict(offsets=None)), ("dt_linear", dict(act="tanh")),
    ("dt_linear", dict(weight=tensors(2, 7, 8), gated=True)), ("dt_linear", dict(gated=True)), ("dt_linear", dict(weight=tensors(2, 0, 8))),
    ("dt_moe_layer", dict(w_in=tensors(2, 6, 8))), ("dt_moe_layer", dict(gated=False)), ("dt_moe_layer", dict(w_out=tensors(2, 9, 6))),
    ("dt_moe_layer", dict(w_out=tensors(16, 6))), ("dt_block_norm", dict(post_weight=None, pre_weight=None)), ("dt_block_norm", dict(gate=tensors(3, 8))),
    ("dt_block_norm_backward", dict(post_weight=None, pre_weight=None)),
])
def test_shapes_that_do_not_fit(reached, name, kw):
    with pytest.raises((ValueError, KeyError)):
        getattr(dt, name)(**dict(CALLS[name], **kw))
    assert name not in reached


def test_workspace_functions_of_the_binding():
    with pytest.raises(dt.DtError):
        dt.dt_moe_layer_workspace([300], 8, 8, 4, 2)
    with pytest.raises(dt.DtError):
        dt.dt_linear_backward_workspace([4], 0, 8)
    with pytest.raises(dt.DtError):
        dt.dt_block_norm_workspace([4], 0)
    assert dt.dt_linear_backward_workspace([4, 4], 2, 8) == 0
    assert dt.dt_linear_backward_workspace([4, 4], 2, 8, "silu", True, True, torch.float32) > 0
    assert dt.dt_moe_layer_workspace([4], 8, 8, 4, 2) > 0 and dt.dt_block_norm_workspace([4], 8) > 0
