"""GPU: the norms around a block through the C ABI where ranks hold no rows and
list NULL for them, and where only some of the shared gradients are asked for,
against the 64-bit definition."""
import ctypes
import itertools

import pytest
import torch

import block_reference as ref
from gpu_util import Guarded, note
from test_gpu_block import DTYPES, Block

pytestmark = pytest.mark.gpu


def pointers(ts, rows, all_ranks=False):
    """The list as C takes it: NULL for a rank without rows, unless every rank gets the buffer."""
    if ts is None:
        return None
    return (ctypes.c_void_p * len(rows))(*[t.data_ptr() if n > 0 or all_ranks else None for t, n in zip(ts, rows)])


def backward(b, wanted):
    """The gradients named in `wanted`, dx and dz, checked."""
    from collective_communication_primitives_amd import _lib
    lib = _lib.load()
    sizes, wide, stats = [n * b.cols for n in b.rows], [b.cols] * b.p, b.stats_of()
    dz, dx = b.guards(sizes), b.guards(sizes)
    sums = {name: b.guards(sizes if name == "dgate" and b.gate_kind == "row" else wide) for name in wanted}
    t = lambda gs: None if gs is None else [g.t for g in gs]
    of = lambda ts: pointers(ts, b.rows)
    out = lambda name: pointers(t(sums.get(name)), b.rows, name != "dgate" or b.gate_kind == "channel")
    rows = (ctypes.c_size_t * b.p)(*b.rows)
    code = {torch.float32: 0, torch.bfloat16: 1}[b.dtype]
    need = lib.dt_block_norm_workspace(b.p, rows, b.cols, code)
    space = torch.empty(need, dtype=torch.uint8, device="cuda")
    status = lib.dt_block_norm_backward(of(b.dy), of(b.dh), of(b.z), of(b.h), of(b.gate), of(b.w1), of(b.b1), of(b.w2), of(stats), of(t(dz)), of(t(dx)),
                                        out("dgate"), out("dpost_weight"), out("dpost_bias"), out("dpre_weight"), out("dpre_bias"), b.p, rows, b.cols,
                                        int(b.gate_kind == "row"), b.scale, int(b.rms), code, space.data_ptr(), need,
                                        torch.cuda.current_stream().cuda_stream)
    assert status == 0, lib.dt_last_error().decode()
    torch.cuda.synchronize()
    want = ref.block_backward(torch.cat(b.dy), torch.cat(b.dh), torch.cat(b.z), torch.cat(b.h), b.every_gate(), b.w1[0], b.b1[0], b.w2[0],
                              torch.cat(stats), b.scale, b.rms)
    for gs in [dz, dx, *sums.values()]:
        for g in gs:
            g.check()
    ref.assert_close(torch.cat(t(dx)).view(-1, b.cols), *want["dx"], "dx")
    ref.assert_close(torch.cat(t(dz)).view(-1, b.cols), *want["dz"], "dz")
    for name, gs in sums.items():
        if name == "dgate" and b.gate_kind == "row":
            ref.assert_close(torch.cat(t(gs)).view(-1, b.cols), *want["dgate"], name)
        else:
            for q, g in enumerate(gs):
                ref.assert_close(g.t, *want["dgate_sum" if name == "dgate" else name], f"{name}[{q}]")


# a width of each way that a row is held: lanes, waves, two passes, read again
WIDTHS = [40, 100, 700, 1999, 4000, 9000, 40000]


@DTYPES
@pytest.mark.parametrize("gate", ["channel", "row"])
@pytest.mark.parametrize("rows", [[0, 7, 3], [0, 0, 5], [4, 0, 2]], ids=lambda v: str(v).replace(" ", ""))
def test_the_gate_s_gradient_sees_the_bias_of_the_ranks_with_rows(rows, gate, dtype):
    """dgate without the biases' gradients: post_bias is an input of dgate all the same, wherever the rows are."""
    note(f"block, NULL for ranks without rows, rows={rows} gate={gate} {dtype}")
    for cols in WIDTHS:
        b = Block(rows, cols, dtype, gate=gate, scale=0.75, seed=50)
        backward(b, ["dgate"])
        backward(b, ["dgate", "dpre_weight"])


NAMES = ["dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"]


@pytest.mark.parametrize("cols", WIDTHS)
def test_any_of_the_gradients_may_be_left_out(cols):
    note(f"block, every choice of gradients, cols={cols}")
    for i, wanted in enumerate(itertools.chain.from_iterable(itertools.combinations(NAMES, n) for n in range(6))):
        b = Block([[0, 6, 5], [3, 4, 0]][i % 2], cols, (torch.bfloat16, torch.float32)[i // 2 % 2], gate=("channel", "row")[i % 3 % 2], rms=i % 5 == 0, seed=i)
        backward(b, wanted)
