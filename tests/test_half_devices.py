"""The binding of include/megamoe/half.h: complete, and every entry point starts on its tensors' device and that device's
stream, whichever is current (no GPU needed: tensors that name a device, and a library that records calls)."""
from __future__ import annotations

import os
import re
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests.test_binding_devices import _Gpu0, _Gpu1, handle, machine  # noqa: E402,F401
from tests.test_half_refusals import ARGS, B, D  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_library_and_binding_agree():
    src = open(os.path.join(ROOT, "include", "megamoe", "half.h")).read()
    declared = set(re.findall(r"\b(megamoe_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert declared == set(H.EXPORTED) and len(H.EXPORTED) == len(declared)
    assert not declared & set(MM.EXPORTED)
    for name in declared:
        assert hasattr(MM.load(), name) and hasattr(H, name)
    assert set(ARGS) == {n for n in declared if not n.endswith("_bytes")}


def on(kind, name, **changed):
    return {k: (changed.get(k, kind))._make_subclass(changed.get(k, kind), v) for k, v in ARGS[name].items()}


@pytest.mark.parametrize("name", sorted(ARGS))
@pytest.mark.parametrize("kind", [_Gpu0, _Gpu1], ids=["current", "other"])
def test_runs_on_the_tensors_device(machine, name, kind):  # noqa: F811
    getattr(H, name)(B, **on(kind, name))
    assert machine.calls == [(name, kind.where, handle(kind.where))]
    assert machine.current == 0


@pytest.mark.parametrize("name", sorted(ARGS))
def test_stream_given(machine, name):  # noqa: F811
    stream = SimpleNamespace(cuda_stream=77, device_index=1)
    getattr(H, name)(B, **on(_Gpu1, name), stream=stream)
    assert machine.calls == [(name, 1, 77)]
    with pytest.raises(ValueError, match="stream"):
        getattr(H, name)(B, **on(_Gpu0, name), stream=stream)
    assert len(machine.calls) == 1


@pytest.mark.parametrize("name", sorted(ARGS))
def test_tensors_of_two_devices_are_refused(machine, name):  # noqa: F811
    for key in ARGS[name]:
        with pytest.raises(ValueError, match="one device"):
            getattr(H, name)(B, **on(_Gpu0, name, **{key: _Gpu1}))
    assert machine.calls == []


OPTIONAL = {"probs", "bias", "dprobs", "gate", "w_after", "w_before", "expanded_row_idx", "rows", "x", "dr", "dh", "s", "r",
            "h", "ds", "dw_after", "dw_before", "dgate"}  # which of them may be missing together is the library's to say


@pytest.mark.parametrize("name", sorted(ARGS))
def test_nothing_for_a_tensor(name):
    """None is a null pointer, which the library refuses with its own error."""
    if torch.cuda.device_count():
        pytest.skip("passes host addresses; host-only")
    for key in ARGS[name]:
        if key == "workspace" or (key in OPTIONAL and name in ("megamoe_norm", "megamoe_norm_grad")):
            continue
        if key in ("probs", "bias", "dprobs") and name != "megamoe_forward_half" and (name, key) != ("megamoe_route_grad", "probs"):
            continue
        with pytest.MonkeyPatch.context() as patch:
            patch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
            patch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
            with pytest.raises(MM.MegaMoEError) as err:
                getattr(H, name)(B, **{**on(_Gpu0, name), key: None})
            assert err.value.status == 1, key


def test_dims_are_the_placeholder_ones():
    assert MM.megamoe_check_dims(D) == 0 and MM.megamoe_check_dims(B) == 0
