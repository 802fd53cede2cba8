"""GPU: tokens that their target leaves out of the loss may hold anything in
their hidden rows (a padded batch): no gradient takes anything from them."""
import pytest
import torch

from gpu_util import Guarded, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


def _gradients(dt, h, w, t, dl, p):
    tokens, cols = h.shape
    loss, lse = [[torch.empty(tokens, device="cuda") for _ in range(p)] for _ in range(2)]
    dh = [Guarded(h.numel(), h.dtype).poison() for _ in range(p)]
    dw = [Guarded(x.numel(), h.dtype).poison() for x in w]
    dt.dt_vocab_loss([h] * p, w, [t] * p, loss, lse)
    dt.dt_vocab_loss_backward([h] * p, w, [t] * p, lse, [dl] * p, [x.t for x in dh], [x.t for x in dw])
    torch.cuda.synchronize()
    for x in dh + dw:
        x.check()
    return [x.t.view(-1, cols) for x in dh], [x.t.view(-1, cols) for x in dw], loss


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tokens,cols,offset", [(1, 64, 0), (9, 33, 0), (40, 136, 1), (130, 512, 0), (700, 96, 0), (700, 34, 2)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_what_padding_holds_reaches_no_gradient(dt, tokens, cols, offset, dtype, value):
    note(f"loss, padded rows of {value}, {tokens} x {cols} + {offset} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(31)
    flat = torch.empty(offset + tokens * cols, dtype=dtype, device="cuda")
    flat[offset:] = torch.randn(tokens * cols, generator=g, device="cuda").to(dtype)
    h = flat[offset:].view(tokens, cols)
    w = [(torch.randn(n, cols, generator=g, device="cuda") / cols ** 0.5).to(dtype) for n in (70, 55)]
    t = torch.randint(0, 125, (tokens,), generator=g, device="cuda")
    out = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    out[::3] = True
    t[::3] = -100
    t[::6] = 125
    dl = torch.rand(tokens, generator=g, device="cuda")
    h[out] = 0
    dh0, dw0, loss0 = _gradients(dt, h, w, t, dl, 2)
    h[out] = value
    dh, dw, loss = _gradients(dt, h, w, t, dl, 2)
    for a, b in zip(dw + loss, dw0 + loss0):
        assert torch.equal(a, b) and bool(a.isfinite().all())
    for a, b in zip(dh, dh0):
        assert torch.equal(a, b) and bool((a[out] == 0).all())
    h0 = h.clone()
    assert torch.equal(h0.nan_to_num(), h.nan_to_num())  # the input is as it was
