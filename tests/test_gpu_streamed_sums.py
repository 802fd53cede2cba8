"""GPU: fp32 sums of many terms where few rows meet many weights.  A sum runs over
512 terms at most, and these sums are added up apart, as in the products of many
rows: the error does not grow with every term of a long sum."""
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


# A term just above 1 whose excess is rounded away, the same way each time, beside a
# sum of 2^14 or more.  One sum of n such terms is off by thousands of U, in any
# order that adds them to it one by one (5300 and 6700 U with the 32768 terms of a
# quarter).
TERMS = [1 + 0.45 * 2.0 ** -10, 1 + 0.9 * 2.0 ** -10]


def allowed(n):
    """Every value of `terms` terms in all, split among 4 waves or more: 512 roundings in a run, one for each run of a wave's
    share, one for each of up to 16 waves; each of at most U of the whole sum, as all terms are positive.  8 for what follows."""
    return (512 + n // 4 // 512 + 16 + 8) * U


@pytest.mark.parametrize("rows", [1, 17, 40], ids=["16_waves", "32_rows_at_a_time", "64_rows_at_a_time"])
@pytest.mark.parametrize("cols", [131072, 131070])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_products(dt, gated, cols, rows):
    note(f"streamed fp32 sums, {rows} rows of {cols} gated={gated}")
    for term in TERMS:
        x, w = torch.ones(rows, cols, device="cuda"), torch.full((32, cols), term, device="cuda")
        outs = 16 if gated else 32
        y, pre = torch.empty(rows, outs, device="cuda"), torch.empty(rows, 32, device="cuda")
        dt.dt_linear([x], [w], [y], pre=[pre], gated=gated)
        torch.cuda.synchronize()
        want = float(w[0, 0].double()) * cols
        assert float((pre.double() / want - 1).abs().max()) <= allowed(cols), term


def test_the_experts_layer(dt):
    """Many tokens to an expert, so that four waves share the first product's sum, and as many terms in the second's."""
    for cols, inner in ((131072, 16), (131070, 16), (16, 131072)):
        note(f"streamed fp32 sums, layer cols={cols} inner={inner}")
        for term in TERMS:
            t = 40
            x, experts, one = torch.ones(t, cols, device="cuda"), torch.zeros(t, 1, dtype=torch.int32, device="cuda"), torch.ones(t, 1, device="cuda")
            # the first product's terms are summed where cols is long, the second's where inner is; the others' sums are exact:
            # one term that is not 0
            w_in, w_out = torch.zeros(1, inner, cols, device="cuda"), torch.zeros(1, cols, inner, device="cuda")
            if cols > inner:
                w_in[:] = term
                w_out[:, :, 0] = 1
            else:
                w_in[:, :, 0] = 1
                w_out[:] = term
            out = torch.empty_like(x)
            dt.dt_moe_layer([x], [experts], [one], [w_in], [w_out], [out], act="none", gated=False)
            torch.cuda.synchronize()
            n = max(cols, inner)
            want = float(torch.tensor(term).double()) * n
            assert float((out.double() / want - 1).abs().max()) <= allowed(n), (cols, inner, term)
