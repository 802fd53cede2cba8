"""GPU: infinite weights of the experts' second product.  A finite value that is not
zero times an infinite weight is an infinity of the product's sign, whatever bits the
value has between the products."""
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


# tokens, cols, inner, experts, choices: 8 and 16 waves to a workgroup, 16 and 64 tokens at a time, split and whole rows
SHAPES = [(5, 72, 40, 4, 1), (9, 70, 41, 6, 2), (40, 256, 64, 2, 2), (130, 64, 96, 8, 2), (20, 2048, 512, 16, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tokens,cols,inner,experts,topk", SHAPES)
def test_an_infinite_weight_gives_an_infinity(dt, tokens, cols, inner, experts, topk, dtype):
    note(f"layer with infinite weights, {tokens} tokens of {cols}, {topk} of {experts} experts of {inner} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(70 + tokens)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    # the first product gives whole numbers of up to 24, of which the second bf16 part is zero; the first choice's weight takes
    # a little off them, and the second part has the other sign (7.99 rounds to 8)
    x = torch.zeros(tokens, cols, device="cuda")
    x[:, 0] = torch.randint(1, 4, (tokens,), generator=g, device="cuda") * torch.where(new(tokens) > 0, 1.0, -1.0)
    w_in, b_in = torch.zeros(experts, inner, cols, device="cuda"), torch.zeros(experts, inner, device="cuda")
    w_in[:, :, 0] = torch.randint(1, 9, (experts, inner), generator=g, device="cuda").float()
    share = torch.ones(tokens, topk, device="cuda")
    share[:, 0] = 0.99875   # 8 times it is 7.99
    chosen = torch.rand(tokens, experts, generator=g, device="cuda").topk(topk, 1).indices
    w_out = new(experts, cols, inner)
    at = torch.randint(0, inner, (experts, cols), generator=g, device="cuda")
    sign = torch.where(new(experts, cols) > 0, 1.0, -1.0)
    some = torch.rand(experts, cols, generator=g, device="cuda") < 0.5   # half of the rows have an infinity
    row = torch.full((), float("inf"), device="cuda") * sign
    w_out.scatter_(2, at[:, :, None], torch.where(some, row, w_out.gather(2, at[:, :, None])[:, :, 0])[:, :, None])
    out = torch.empty(tokens, cols, dtype=dtype, device="cuda")
    to = lambda t: [t.to(dtype)]
    dt.dt_moe_layer(to(x), [chosen.int()], [share], to(w_in), to(w_out), [out], b_in=to(b_in), act="none", gated=False)
    torch.cuda.synchronize()
    want = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    for j in range(topk):
        h = (w_in[chosen[:, j], :, 0] * x[:, :1]).double() * share[:, j:j + 1].double()
        want += (w_out.to(dtype)[chosen[:, j]].double() * h[:, None, :]).sum(2)
    assert int(want.isinf().sum()) > 0 and int(want.isfinite().sum()) > 0
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.isposinf(), want.isposinf()) and torch.equal(out.isneginf(), want.isneginf())
