"""GPU: the loss over a sharded vocabulary and its gradients against the
64-bit definition."""
import pytest
import torch

import step_reference as ref
from gpu_util import Guarded, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def _make(tokens, cols, shards, dtype, seed, offset=0, replicas=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = sum(shards)

    def rows(n, std):
        t = torch.empty(n * cols + offset, dtype=dtype, device="cuda")
        t[offset:] = (torch.randn(n * cols, generator=g, device="cuda") * std).to(dtype)
        return t[offset:].view(n, cols)

    weight = [rows(n, 2.0 / cols ** 0.5) for n in shards]
    hidden = rows(tokens, 1.0)
    targets = torch.randint(0, v, (tokens,), generator=g, device="cuda")
    if tokens > 3:
        targets[1] = -100
        targets[tokens - 1] = v - 1
        targets[2] = 0
    dloss = torch.randn(tokens, generator=g, device="cuda")
    p = len(shards)
    if replicas:
        return [hidden.clone() if offset == 0 else hidden for _ in range(p)], weight, [targets.clone() for _ in range(p)], [
            dloss.clone() for _ in range(p)]
    return [hidden] * p, weight, [targets] * p, [dloss] * p


def _run(dt, hidden, weight, targets, dloss, offset=0, **kw):
    p, (tokens, cols), dtype = len(hidden), hidden[0].shape, hidden[0].dtype
    loss = [Guarded(tokens, torch.float32).poison() for _ in range(p)]
    lse = [Guarded(tokens, torch.float32).poison() for _ in range(p)]
    dh = [Guarded(tokens * cols, dtype, offset_elems=offset).poison() for _ in range(p)]
    dw = [Guarded(w.numel(), dtype, offset_elems=offset).poison() for w in weight]
    ign = {k: v for k, v in kw.items() if k == "ignore_index"}
    dt.dt_vocab_loss(hidden, weight, targets, [g.t for g in loss], [g.t for g in lse], **ign)
    dt.dt_vocab_loss_backward(hidden, weight, targets, [g.t for g in lse], dloss, [g.t for g in dh], [g.t for g in dw], **kw)
    torch.cuda.synchronize()
    for g in loss + lse + dh + dw:
        g.check()
    return loss, lse, dh, dw


def _check(dt, hidden, weight, targets, dloss, offset=0, **kw):
    loss, lse, dh, dw = _run(dt, hidden, weight, targets, dloss, offset, **kw)
    cols = hidden[0].shape[1]
    want = ref.loss(hidden[0], weight, targets[0], dloss[0], kw.get("ignore_index", -100))
    for q in range(len(hidden)):
        ref.assert_close(lse[q].t, *want["lse"], f"lse[{q}]")
        ref.assert_close(loss[q].t, *want["loss"], f"loss[{q}]")
        ref.assert_close(dh[q].t.view(-1, cols), *want["dhidden"], f"dhidden[{q}]")
        ref.assert_close(dw[q].t.view(-1, cols), want["dweight"][0][q], want["dweight"][1][q], f"dweight[{q}]")


CASES = [
    # tokens, cols, shards, piece
    (1, 1, [1], 0), (1, 8, [2], 0), (3, 16, [5, 0, 4], 0), (5, 64, [130], 0), (2, 128, [100, 300], 0), (17, 100, [70, 33], 0),
    (64, 256, [128, 128], 0), (65, 72, [257], 100), (130, 512, [200, 120, 77], 64), (129, 1000, [333, 1, 400], 0),
    (300, 136, [260, 250], 96), (33, 1024, [1000], 0), (7, 33, [64] * 16, 0), (260, 40, [520, 10], 300), (16, 4096, [300, 500], 0),
    (257, 320, [700, 513], 256), (1, 2048, [5000, 3001], 0), (4, 520, [1030], 0),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tokens,cols,shards,piece", CASES, ids=lambda v: str(v).replace(" ", "")[:24])
def test_loss_and_its_gradients(dt, tokens, cols, shards, piece, dtype):
    note(f"loss tokens={tokens} cols={cols} shards={shards} piece={piece} {dtype}")
    _check(dt, *_make(tokens, cols, shards, dtype, 5), piece_rows=piece)


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_off_alignment(dt, dtype, off):
    note(f"loss off alignment {off} {dtype}")
    _check(dt, *_make(70, 136, [190, 45], dtype, 6, offset=off), offset=off)


def test_all_tokens_left_out(dt):
    note("loss all ignored")
    h, w, t, g = _make(9, 64, [40, 30], torch.bfloat16, 7)
    for bad in (-100, 70, 2 ** 40, -1):
        t = [torch.full_like(x, bad) for x in t]
        loss, lse, dh, dw = _run(dt, h, w, t, g)
        assert all(bool((v.t == 0).all()) for v in loss + dh + dw)
        assert all(bool(v.t.isfinite().all()) for v in lse)


def test_ignore_index_inside_the_vocabulary(dt):
    note("loss ignore_index 3")
    h, w, t, g = _make(40, 96, [50, 30], torch.float32, 8)
    t = [x.clone() for x in t]
    for x in t:
        x[::3] = 3
    _check(dt, h, w, t, g, ignore_index=3)


def test_no_tokens_give_zero_weight_gradients(dt):
    note("loss without tokens")
    h, w, t, g = _make(0, 64, [40, 30], torch.float32, 9)
    loss, lse, dh, dw = _run(dt, h, w, t, g)
    assert all(bool((v.t == 0).all()) for v in dw)


def test_large_logits_do_not_overflow(dt):
    note("loss large logits")
    h, w, t, g = _make(30, 64, [100, 28], torch.float32, 10)
    h = [x * 300 for x in h]
    _check(dt, h, w, t, g)


def test_nan_stays_in_its_token(dt):
    note("loss NaN row")
    h, w, t, g = _make(20, 64, [100, 28], torch.bfloat16, 11, replicas=False)
    h[0][4, 3] = float("nan")
    loss, lse, dh, dw = _run(dt, h, w, t, g)
    bad = lse[0].t.isnan()
    assert bool(bad[4]) and int(bad.sum()) == 1
    rows = dh[0].t.view(20, 64).isnan().any(1)
    assert bool(rows[4]) and int(rows.sum()) == 1


@pytest.mark.parametrize("piece", [1, 7, 64, 1000])
def test_pieces_give_one_result(dt, piece):
    """The piece changes only how dhidden's sum is cut."""
    note(f"loss piece {piece}")
    _check(dt, *_make(50, 96, [120, 60], torch.float32, 12), piece_rows=piece)


def test_gradients_against_differences(dt):
    note("loss gradients by differences")
    h, w, t, g = _make(4, 24, [9, 6], torch.float32, 13)
    _, _, dh, dw = _run(dt, h, w, t, g)
    use = t[0] >= 0

    def value(x, ws):
        z = x @ torch.cat(ws).t()
        at = t[0].clamp(min=0)
        return float(((torch.logsumexp(z, 1) - z.gather(1, at[:, None])[:, 0]) * use * g[0].double()).sum())

    e = 1e-5
    x, ws = h[0].double(), [s.double() for s in w]
    for i in range(4):
        for c in range(0, 24, 5):
            up, dn = x.clone(), x.clone()
            up[i, c] += e
            dn[i, c] -= e
            assert abs((value(up, ws) - value(dn, ws)) / (2 * e) - float(dh[0].t.view(4, 24)[i, c])) < 2e-5
    for v in range(9):
        up, dn = [s.clone() for s in ws], [s.clone() for s in ws]
        up[0][v, 3] += e
        dn[0][v, 3] -= e
        assert abs((value(x, up) - value(x, dn)) / (2 * e) - float(dw[0].t.view(9, 24)[v, 3])) < 2e-5


@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 34), (torch.bfloat16, 1002), (torch.bfloat16, 35), (torch.float32, 33),
                                        (torch.float32, 131), (torch.float32, 64)], ids=str)
def test_an_infinite_weight_stays_in_its_row(dt, dtype, cols):
    """A vocabulary row that -inf takes out (all hidden values of that column
    positive) leaves the rows beside it alone, wherever a row ends."""
    note(f"loss row of -inf, {cols} columns {dtype}")
    h, w, t, g = _make(70, cols, [200, 90], dtype, 14, replicas=False)
    h[0][:, 0] = h[0][:, 0].abs() + 0.5
    t[0].clamp_(min=10)
    gone = [3, 4, 199]
    for v in gone:
        w[0][v] = 0
        w[0][v, 0] = -float("inf")
    t[0][torch.isin(t[0], torch.tensor(gone, device="cuda"))] = 11
    loss, lse, dh, dw = _run(dt, h, w, t, g)
    keep = [v for v in range(200) if v not in gone]
    want = ref.loss(h[0], [w[0][keep], w[1]], t[0] - (t[0] > 3).long() - (t[0] > 4).long() - (t[0] > 199).long(), g[0])
    for q in range(2):
        ref.assert_close(lse[q].t, *want["lse"], f"lse[{q}]")
        ref.assert_close(loss[q].t, *want["loss"], f"loss[{q}]")
    mine = dw[0].t.view(200, cols)
    ref.assert_close(mine[keep], want["dweight"][0][0], want["dweight"][1][0], "dweight[0]")
    ref.assert_close(dw[1].t.view(90, cols), want["dweight"][0][1], want["dweight"][1][1], "dweight[1]")
    assert bool((mine[gone] == 0).all())


@pytest.mark.parametrize("tokens", [1, 12, 65, 300, 512])
def test_few_tokens_lose_nothing_to_the_rounded_gradient(dt, tokens):
    """bf16, few tokens: the gradients are off by their own rounding and, relative to the terms' magnitudes, by 2^-16 (the
    logits' gradient in two bf16 parts), 350 * 2^-24 (logits of 256 terms of up to 16 in all, in fp32) and the sums' 40 *
    2^-24: under 2^-14 together.  One bf16 part would add 2^-8."""
    note(f"loss in two parts, {tokens} tokens")
    h, w, t, g = _make(tokens, 256, [300, 213], torch.bfloat16, 15, replicas=False)
    _, _, dh, dw = _run(dt, h, w, t, g)
    x, v = h[0].double(), torch.cat(w).double()
    use = (t[0] >= 0).double()[:, None] * g[0].double()[:, None]
    p = (x @ v.t()).softmax(1)
    hot = torch.zeros_like(p).scatter_(1, t[0].clamp(min=0)[:, None], 1.0)
    d, size = (p - hot) * use, (p + hot) * use.abs()
    for q in range(2):
        ref.assert_close(dh[q].t.view(-1, 256), d @ v, 2.0 ** -14 * (size @ v.abs()), f"dhidden[{q}]")
    got = torch.cat([s.t.view(-1, 256) for s in dw])
    ref.assert_close(got, d.t() @ x, 2.0 ** -14 * (size.t() @ x.abs()), "dweight")


def test_odd_rows_copied_in_several_pieces(dt):
    """bf16 rows of odd width are copied piece by piece; these need three pieces, which cut the shards."""
    note("loss, odd bf16 rows in three pieces")
    _check(dt, *_make(2000, 33, [25000, 0, 15001], torch.bfloat16, 16, replicas=False))


def test_as_many_tokens_as_the_call_takes(dt):
    """2^22 tokens: the forward pass needs more than one launch for 20000 rows.  Sampled tokens against the definition; a
    logit of 8 terms and the sum of 20000 exponentials in fp32."""
    note("loss of 2^22 tokens")
    tokens, cols, shards = 1 << 22, 8, [9000, 11000]
    g = torch.Generator(device="cuda").manual_seed(17)
    h = torch.randn(tokens, cols, generator=g, device="cuda").bfloat16()
    w = [(torch.randn(n, cols, generator=g, device="cuda") / 2).bfloat16() for n in shards]
    t = torch.randint(0, sum(shards), (tokens,), generator=g, device="cuda")
    loss, lse = [[torch.empty(tokens, device="cuda") for _ in range(2)] for _ in range(2)]
    dt.dt_vocab_loss([h] * 2, w, [t] * 2, loss, lse)
    at = torch.cat([torch.arange(300, device="cuda"), torch.randint(0, tokens, (2000,), generator=g, device="cuda"),
                    torch.arange(tokens - 300, tokens, device="cuda")])
    want = ref.loss(h[at], w, t[at], None)
    for q in range(2):
        ref.assert_close(lse[q][at], *want["lse"], f"lse[{q}]")
        ref.assert_close(loss[q][at], *want["loss"], f"loss[{q}]")
    assert torch.equal(lse[0], lse[1]) and bool(lse[0].isfinite().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_every_rank_gets_the_same_bits(dt, dtype):
    note(f"loss, sixteen ranks' bits {dtype}")
    h, w, t, g = _make(600, 64, [300] * 16, dtype, 18, replicas=False)
    loss, lse, dh, _ = _run(dt, h, w, t, g)
    for outs in (loss, lse, dh):
        assert all(torch.equal(o.t, outs[0].t) for o in outs)


@pytest.mark.parametrize("dloss", ["mean", "one large", "infinite", "zero", "masked NaN"])
def test_gradients_of_the_loss_scaled(dt, dloss):
    """More tokens than are kept in two parts: the logits' gradient is relative to the largest finite dloss."""
    note(f"loss, dloss {dloss}")
    tokens = 700
    h, w, t, g = _make(tokens, 96, [180, 130], torch.bfloat16, 19, replicas=False)
    if dloss == "mean":
        g[0].fill_(1.0 / tokens)
    elif dloss == "one large":
        g[0][5] = 3e30
    elif dloss == "zero":
        g[0].zero_()
    if dloss in ("mean", "one large", "zero"):
        _check(dt, h, w, t, g)
    if dloss == "mean":
        # the rounding of 1 / tokens itself must not be in the result: its half step would shift the whole norm by up to
        # 2^-9, the results' and the other terms' roundings are independent of it and leave its average near 0
        _, _, dh, _ = _run(dt, h, w, t, g)
        want = ref.loss(h[0], w, t[0], g[0])["dhidden"][0].cuda()
        got = dh[0].t.view(tokens, 96).double()
        assert abs(float((got * want).sum() / want.square().sum()) - 1) < 2.0 ** -12
    if dloss == "infinite":
        g[0][5] = float("inf")
        _, _, dh, _ = _run(dt, h, w, t, g)
        ok = dh[0].t.view(tokens, 96).isfinite().all(1)
        assert int((~ok).sum()) == 1 and not bool(ok[5])
    if dloss == "masked NaN":
        t[0][7] = -100
        g[0][7] = float("nan")
        clean = g[0].clone()
        clean[7] = 0
        a, b = _run(dt, h, w, t, g), _run(dt, h, w, t, [clean] * 2)
        for x, y in zip(a[2] + a[3], b[2] + b[3]):
            assert torch.equal(x.t, y.t)
