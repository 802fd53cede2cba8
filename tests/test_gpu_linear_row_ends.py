"""GPU: dx in parts where a workgroup goes from one part to the next.  The last part's
rows end earlier than the others', inside 16 bytes, and what is masked behind their
end must not be masked in the part before.

A workgroup takes several tiles of such a product only where the runs are longer
than all rows, which offsets that decrease make them: those are not allowed, and a
row in several runs gets any of their values.  Here all runs have the same weight,
so there is one value."""
import pytest
import torch

import block_reference as ref
from gpu_util import Guarded, note
from test_gpu_linear import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    import collective_communication_primitives_amd as m
    return m


# outs: the parts take 20 steps each (16 terms of fp32, 32 of bf16), the last one 16.9 of them
@pytest.mark.parametrize("dtype,outs", [(torch.float32, 1230), (torch.bfloat16, 2458)], ids=["fp32", "bf16"])
def test_a_part_s_terms_are_all_met(dt, dtype, outs):
    note(f"linear parts' row ends {dtype}")
    rows, cols, runs = 1024, 64, 6
    g = torch.Generator(device="cuda").manual_seed(60)
    x, dy, one = (normal(g, dtype, *s) for s in ((rows, cols), (rows, outs), (outs, cols)))
    w = one.expand(runs, outs, cols).contiguous()
    off = [torch.tensor([0, rows, 0, rows, 0, rows, 0], dtype=torch.int32, device="cuda")]
    dx, dw = Guarded(rows * cols, dtype).poison(), Guarded(runs * outs * cols, dtype).poison()
    dt.dt_linear_backward([dy], [x], [w], [dx.t], [dw.t], offsets=off)
    torch.cuda.synchronize()
    for t in (dx, dw):
        t.check()
    want, err = ref.linear_backward(dy, x, one, None, "none", False)
    ref.assert_close(dx.t.view(rows, cols), want[0], err[0], "dx")
    for e in range(runs):
        got = dw.t.view(runs, outs, cols)[e]
        if e % 2 == 0:
            ref.assert_close(got, want[1], err[1], f"dweight {e}")
        else:
            assert bool((got == 0).all())
