"""Lists of tensors that the binding of the model-step operators hands to the
C ABI: one tensor per rank in each of them, or a refusal before the call.
Needs no GPU: a CPU tensor's device is -1, and the library is a stub."""
import types

import pytest
import torch

import collective_communication_primitives_amd as dt

P, TOKENS, COLS, EXPERTS, TOPK, CAPACITY = 4, 3, 8, 8, 2, 5


@pytest.fixture
def reached(monkeypatch):
    """The names of the library's functions that were called."""
    calls = []

    def entry(name):
        def call(*args):
            calls.append(name)
            return 256 if name.endswith("_workspace") else 0
        return call

    names = [n for n in dt._lib.EXPORTS]
    monkeypatch.setattr(dt, "_L", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(dt, "_current_stream_handle", lambda: 0)
    monkeypatch.setattr(dt, "_workspace", lambda *a: torch.empty(256, dtype=torch.uint8))
    return calls


def exchange_calls():
    """name -> call(p, length of one list): the exchange's calls with that list one tensor per rank, or not."""
    tok = lambda n=P: [torch.zeros(TOKENS, COLS) for _ in range(n)]
    held = lambda n=P: [torch.zeros(CAPACITY, COLS) for _ in range(n)]
    slots = lambda dtype, n=P: [torch.zeros(TOKENS, TOPK, dtype=dtype) for _ in range(n)]
    i32, f32 = torch.int32, torch.float32
    offsets = lambda n=P: [torch.zeros(EXPERTS // P + 1, dtype=i32) for _ in range(n)]
    return {
        "dispatch recv": lambda n: dt.dt_moe_dispatch(tok(), slots(i32), held(n), slots(i32), offsets(), EXPERTS),
        "dispatch experts": lambda n: dt.dt_moe_dispatch(tok(), slots(i32, n), held(), slots(i32), offsets(), EXPERTS),
        "dispatch positions": lambda n: dt.dt_moe_dispatch(tok(), slots(i32), held(), slots(i32, n), offsets(), EXPERTS),
        "dispatch offsets": lambda n: dt.dt_moe_dispatch(tok(), slots(i32), held(), slots(i32), offsets(n), EXPERTS),
        "combine y": lambda n: dt.dt_moe_combine(held(n), slots(i32), slots(i32), None, tok(), EXPERTS),
        "combine weights": lambda n: dt.dt_moe_combine(held(), slots(i32), slots(i32), slots(f32, n), tok(), EXPERTS),
        "backward y and dy": lambda n: dt.dt_moe_combine_backward(tok(), held(n), slots(i32), slots(i32), slots(f32), held(n), slots(f32),
                                                                 EXPERTS),
        "backward y": lambda n: dt.dt_moe_combine_backward(tok(), held(n), slots(i32), slots(i32), slots(f32), held(), slots(f32), EXPERTS),
        "backward dy": lambda n: dt.dt_moe_combine_backward(tok(), held(), slots(i32), slots(i32), slots(f32), held(n), slots(f32), EXPERTS),
        "backward dweights": lambda n: dt.dt_moe_combine_backward(tok(), held(), slots(i32), slots(i32), slots(f32), held(), slots(f32, n),
                                                                 EXPERTS),
    }


@pytest.mark.parametrize("name", sorted(exchange_calls()))
def test_an_exchange_takes_one_tensor_per_rank(reached, name):
    call = exchange_calls()[name]
    call(P)
    assert [n for n in reached if not n.endswith("_workspace")] == ["dt_moe_" + {"dispatch": "dispatch", "combine": "combine",
                                                                                "backward": "combine_backward"}[name.split()[0]]]
    for n in (P - 1, 1, P + 1):
        reached.clear()
        with pytest.raises(ValueError):
            call(n)
        assert reached == []
