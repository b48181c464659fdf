"""A holder made for the current device stays on it, whichever is current later (no GPU needed: the machine of
test_binding_devices.py)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests.test_binding_devices import _Gpu0, _Gpu1, machine  # noqa: E402,F401

M, K, E, TOP_K, I = 4, 256, 8, 2, 128


@pytest.fixture
def memory(machine, monkeypatch):  # noqa: F811
    """torch.empty puts what is asked for on "cuda" on the current device; the sizes come from the library."""
    lib, load = MM._lib, MM.load
    empty = torch.empty

    def on_device(*a, device=None, **k):
        d = torch.device(device)
        kind = (_Gpu0, _Gpu1)[machine.current if d.index is None else d.index]
        return empty(*a, **k).as_subclass(kind)
    monkeypatch.setattr(torch, "empty", on_device)
    monkeypatch.setattr(MM, "_lib", None)
    real = load()
    monkeypatch.setattr(MM, "_lib", lib)
    for module in (MM, H):
        monkeypatch.setattr(module, "load", lambda: real)
    return machine


def at_1(*shape, t):
    return torch.zeros(shape, dtype=t).as_subclass(_Gpu1)


IDS, PROBS = at_1(M, TOP_K, t=torch.int32), at_1(M, TOP_K, t=torch.float32)


def int8(holder):
    moe = holder(M, K, E, TOP_K, I)
    moe.scale1, moe.scale2 = at_1(E, 2 * I, t=torch.float32), at_1(E, K, t=torch.float32)
    return moe, torch.float16, ("forward", "forward_few")


def mxfp4(holder):
    return holder(M, K, E, TOP_K, I), torch.float16, ("forward",)


def half(holder):
    moe = holder(M, K, E, TOP_K, I)
    moe.load_weights(at_1(E, 2 * I, K, t=torch.bfloat16), at_1(E, K, I, t=torch.bfloat16))
    return moe, torch.bfloat16, ("forward", "forward_rows")


@pytest.mark.parametrize("holder, make", [(MM.MegaMoE, int8), (MM.MegaMoEMXFP4, mxfp4), (H.MegaMoEHalf, half)])
def test_stays_on_the_device_it_was_made_on(memory, holder, make):
    memory.current = 1
    moe, t, forms = make(holder)
    memory.current = 0
    for form in forms:
        del memory.calls[:]
        result = getattr(moe, form)(at_1(M, K, t=t), IDS, PROBS)
        assert memory.calls and all(where == 1 for _, where, _ in memory.calls)
    if holder is H.MegaMoEHalf:
        del memory.calls[:]
        moe.combine(result)
        moe.backward(result, at_1(M, K, t=t))
        assert len(memory.calls) == 6 and all(where == 1 for _, where, _ in memory.calls)
    assert moe.device == torch.device("cuda", 1)
