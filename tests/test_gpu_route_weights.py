"""GPU: renormalised sigmoid weights of very negative logits: a share of the
sum keeps its digits where the score itself leaves fp32's range."""
import pytest
import torch

import step_reference as ref
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("e,k", [(8, 4), (200, 4), (600, 4), (40, 20)])
def test_shares_of_scores_that_underflow(e, k, dtype):
    import collective_communication_primitives_amd as dt
    note(f"route weights of negative logits, {k} of {e} {dtype}")
    x = torch.full((8, e), -3e4, device="cuda")
    for row, top in enumerate((-40.0, -55.0, -59.5, -60.0, -60.5, -90.0, -2.0, 30.0)):
        x[row, :k] = torch.linspace(top, top - 80.0, k, device="cuda")
    x = x.to(dtype)
    ex, w = torch.empty(8, k, dtype=torch.int32, device="cuda"), torch.empty(8, k, device="cuda")
    dt.dt_moe_route([x], [ex], [w], score="sigmoid")
    want, _, _ = ref.route(x, k, score="sigmoid")
    assert torch.equal(ex.long().cpu(), want)
    # the definition's own shares, s / sum in 64 bits (e^-140 is far inside them)
    s = torch.sigmoid(x[:, :k].double().cpu())
    share = s / s.sum(1, keepdim=True)
    ref.assert_close(w, share, (2 * 200 + ref.chain(e) + 24) * ref.U * share + 1e-37, "weights")
    g, dl = torch.rand(8, k, device="cuda") + 0.5, torch.empty_like(x)
    dt.dt_moe_route_backward([x], [ex], [g], [dl], score="sigmoid")
    gd = g.double().cpu()
    mean = (gd * share).sum(1, keepdim=True)
    dx = torch.zeros(8, e, dtype=torch.float64)
    dx[:, :k] = share * (gd - mean) * (1 - s)
    size = torch.zeros_like(dx)
    size[:, :k] = share * (gd + mean)
    ref.assert_close(dl, dx, (4 * 200 + 2 * ref.chain(e) + 40) * ref.U * size + 1e-37, "dlogits")
