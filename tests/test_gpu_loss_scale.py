"""GPU: the loss' gradients where one token's dloss is many orders above the
others': each token's gradient keeps its own size."""
import pytest
import torch

import step_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [1e38, 1e-30, 1.0])
@pytest.mark.parametrize("rest", [1.0, 1e-3])
def test_a_token_far_above_the_others(top, rest):
    import collective_communication_primitives_amd as dt
    note(f"loss, one dloss of {top}, the others {rest} below it")
    tokens, cols, shards = 600, 64, [90, 110]
    g = torch.Generator(device="cuda").manual_seed(21)
    h = torch.randn(tokens, cols, generator=g, device="cuda").bfloat16()
    w = [(torch.randn(n, cols, generator=g, device="cuda") / 4).bfloat16() for n in shards]
    t = torch.randint(0, 200, (tokens,), generator=g, device="cuda")
    dl = torch.full((tokens,), min(top, 1.0) * rest * 0.7, device="cuda")
    dl[5] = top
    loss, lse = [[torch.empty(tokens, device="cuda") for _ in range(2)] for _ in range(2)]
    dh, dw = [torch.empty_like(h) for _ in range(2)], [torch.empty_like(x) for x in w]
    dt.dt_vocab_loss([h] * 2, w, [t] * 2, loss, lse)
    dt.dt_vocab_loss_backward([h] * 2, w, [t] * 2, lse, [dl] * 2, dh, dw)
    want = ref.loss(h, w, t, dl)
    for q in range(2):
        ref.assert_close(dh[q], *want["dhidden"], f"dhidden[{q}]")
        ref.assert_close(dw[q], want["dweight"][0][q], want["dweight"][1][q], f"dweight[{q}]")
