"""The host helper of the binding: what it takes, what it hands back, what it
leaves for the caller to refuse.  Needs no GPU (a CPU tensor's device is -1)."""
import ctypes
import sys

import pytest
import torch

import collective_communication_primitives_amd as dt
from collective_communication_primitives_amd import _marshal


def pointers(packed):
    return list((ctypes.c_void_p * (len(packed) // 8)).from_buffer_copy(packed))


@pytest.mark.parametrize("seq", [list, tuple])
@pytest.mark.parametrize("p", [1, 3, 16])
def test_pointers_and_stash(seq, p):
    tensors = seq(torch.zeros(r + 1, 4) for r in range(p))
    stash = ["before"]
    packed = _marshal.buffers(tensors, [4 * (r + 1) for r in range(p)], torch.float32, -1, stash)
    assert pointers(packed) == [t.data_ptr() for t in tensors]
    assert stash[0] == "before" and len(stash) == p + 1 and all(a is b for a, b in zip(stash[1:], tensors))


def test_views_and_empty_tensors():
    base = torch.zeros(10)
    packed = _marshal.buffers([base[3:], base[:0]], [7, 0], torch.float32, -1, [])
    assert pointers(packed)[0] == base.data_ptr() + 12
    assert _marshal.buffers([torch.nn.Parameter(base)], [10], torch.float32, -1, []) is not None


@pytest.mark.parametrize("tensors, sizes", [
    ([torch.zeros(4)], [5]), ([torch.zeros(4)], [4, 4]), ([torch.zeros(4, dtype=torch.bfloat16)], [4]),
    ([torch.zeros(4, 4).t()], [16]), ([torch.zeros(8)[::2]], [4]), ([None], [4]), ([4], [4]), (torch.zeros(1, 4), [4]),
    (None, [4]), ([torch.zeros(4).to_sparse()], [4]),
])
def test_refused_lists_leave_the_stash(tensors, sizes):
    stash = []
    try:
        assert _marshal.buffers(tensors, sizes, torch.float32, -1, stash) is None
    except RuntimeError:  # torch's own refusal of a layout without that property
        pass
    assert stash == []
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        dt._buffers("x", tensors, sizes, torch.float32, -1, stash)


def test_a_tensor_elsewhere_is_refused():
    with pytest.raises(ValueError, match="current GPU"):
        dt._buffers("x", [torch.zeros(4)], [4], torch.float32, 0, [])


def test_counts():
    tensors = [torch.zeros(3, 8), torch.zeros(0, 8), torch.zeros(2, 2, 8)]
    sizes, rows, slots, packed = _marshal.counts(tensors, 8, 3)
    assert (sizes, rows, slots) == ([24, 0, 32], [3, 0, 4], [9, 0, 12])
    assert list((ctypes.c_size_t * 3).from_buffer_copy(packed)) == rows
    for bad in ([torch.zeros(7)], [None], None, 5):
        assert _marshal.counts(bad, 8, 1) is None
    assert _marshal.counts(tensors, 0, 1) is None
    with pytest.raises(ValueError, match="whole rows of 8"):
        dt._row_counts([torch.zeros(7)], 8, "x")


def test_wrong_arguments_raise():
    for args in ((), ([], (), torch.float32, -1, []), ([], [], "float32", -1, []), ([], [], torch.float32, None, [])):
        with pytest.raises(TypeError):
            _marshal.buffers(*args)


def test_no_reference_is_lost_or_kept():
    t = torch.zeros(4, 8)
    before = sys.getrefcount(t)
    for _ in range(100):
        stash = []
        _marshal.buffers([t, t], [32, 32], torch.float32, -1, stash)
        _marshal.buffers([t, t], [32, 31], torch.float32, -1, stash)
        _marshal.counts([t], 8, 2)
        _marshal.counts([t], 7, 2)
    del stash
    assert sys.getrefcount(t) == before
