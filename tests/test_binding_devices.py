"""The binding starts every entry point on its tensors' device and that device's stream, whichever
device is current (no GPU needed: tensors that name a device, and a library that records calls)."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402


class _Gpu0(torch.Tensor):
    """A CPU tensor that says it lives on GPU 0."""
    where = 0

    def get_device(self):
        return self.where

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.where))


class _Gpu1(_Gpu0):
    where = 1


M, K, E, TOP_K, I = 4, 256, 8, 2, 128
R = M * TOP_K
I8, I32, U8, F16, F32, BF = (torch.int8, torch.int32, torch.uint8, torch.float16, torch.float32, torch.bfloat16)
W1P, W2P = (E * K * 256,), (E * I * 256,)
WS = (U8, (64,))
X, IDS, PROBS, OUT = (F16, (M, K)), (I32, (M, TOP_K)), (F32, (M, TOP_K)), (BF, (M, K))
S1, S2, ROWS, EXPERTS = (F32, (E, 2 * I)), (F32, (E, K)), (I32, (R,)), (I32, (E,))
SORT = [X, IDS, (I8, (R, K)), (F32, (R,)), ROWS, ROWS, EXPERTS, EXPERTS]
W1Q, W1S, W2Q, W2S = ((U8, (E, 2 * I, K // 2)), (U8, (E, 2 * I, K // 32)), (U8, (E, K, I // 2)), (U8, (E, K, I // 32)))

# entry point -> takes dims?, its tensors
CALLS = {
    "megamoe_prepack_w1": (True, [(I8, (E, K, 2 * I)), (I8, W1P)]),
    "megamoe_prepack_w2": (True, [(I8, (E, I, K)), (I8, W2P)]),
    "megamoe_forward": (True, [X, IDS, PROBS, (I8, W1P), S1, (I8, W2P), S2, OUT, WS]),
    "megamoe_permute": (True, SORT + [WS]),
    "megamoe_permute_tokens": (True, SORT + [WS]),
    "megamoe_permute_noalloc": (True, SORT + [(I32, (4,))]),
    "megamoe_permute_tokens_paired": (True, SORT + [ROWS, WS]),
    "megamoe_gmm1": (True, [(I8, (R, K)), EXPERTS, (I8, W1P), S1, (F16, (R, 2 * I))]),
    "megamoe_gmm1_gather": (True, [(I8, (M, K)), ROWS, EXPERTS, (I8, W1P), S1, (F16, (R, 2 * I))]),
    "megamoe_gmm1_gather_split": (True, [(I8, (M, K)), ROWS, EXPERTS, (I8, W1P), S1, (F16, (R, 2 * I)), WS]),
    "megamoe_swiglu_quant": (True, [(F16, (R, 2 * I)), (F32, (R,)), EXPERTS, (I8, (R, I)), (F32, (R,))]),
    "megamoe_swiglu_quant_paired": (True, [(F16, (R, 2 * I)), (F32, (R,)), EXPERTS, ROWS, (I8, (R, I)), (F32, (R,))]),
    "megamoe_gmm2": (True, [(I8, (R, I)), EXPERTS, (I8, W2P), S2, (F16, (R, K))]),
    "megamoe_gmm2_paired": (True, [(I8, (R, I)), EXPERTS, (I8, W2P), S2, (F16, (R, K))]),
    "megamoe_unpermute": (True, [(F16, (R, K)), (F32, (R,)), ROWS, PROBS, OUT]),
    "megamoe_last_error": (False, [WS]),
    "megamoe_route": (True, [(F32, (M, E)), IDS, PROBS]),
    "megamoe_forward_few": (True, [X, IDS, PROBS, (I8, W1P), S1, (I8, W2P), S2, OUT, WS]),
    "megamoe_mxfp4_quant": (False, [X, (U8, (M, K // 2)), (U8, (M, K // 32))]),
    "megamoe_mxfp4_dequant": (False, [(U8, (M, K // 2)), (U8, (M, K // 32)), X]),
    "megamoe_mxfp4_gmm1": (True, [(U8, (M, K // 2)), (U8, (M, K // 32)), ROWS, EXPERTS, W1Q, W1S, (BF, (R, I))]),
    "megamoe_mxfp4_gmm2": (True, [(U8, (R, I // 2)), (U8, (R, I // 32)), EXPERTS, W2Q, W2S, (F16, (R, K))]),
    "megamoe_forward_mxfp4": (True, [X, IDS, PROBS, W1Q, W1S, W2Q, W2S, OUT, WS]),
}


def handle(dev):
    return 0x1000 + dev


@pytest.fixture
def machine(monkeypatch):
    """Two devices, 0 current, and a library that notes the current device and the stream of every call."""
    state = SimpleNamespace(current=0, calls=[])

    @contextlib.contextmanager
    def device(dev):
        before, state.current = state.current, dev
        try:
            yield
        finally:
            state.current = before

    def current_stream(dev=None):
        return SimpleNamespace(cuda_stream=handle(state.current if dev is None else dev))

    class Library:
        def __getattr__(self, name):
            def entry(*args):
                stream = args[1] if name == "megamoe_last_error" else args[-1]
                state.calls.append((name, state.current, getattr(stream, "value", stream)))
                return 0
            return entry

    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", handle, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state.current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(MM, "_lib", Library())
    return state


def arguments(name, kinds):
    dims, specs = CALLS[name]
    ts = [torch.zeros(shape, dtype=dtype).as_subclass(kind) for (dtype, shape), kind in zip(specs, kinds)]
    return ([MM.dims(M, K, E, TOP_K, I)] if dims else []) + ts


def test_every_entry_point_is_here():
    sizes = {n for n in MM.EXPORTED if n.endswith("_bytes")}
    assert set(CALLS) == set(MM.EXPORTED) - sizes - {"megamoe_strerror", "megamoe_check_dims", "megamoe_set_overlap"}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("kind", [_Gpu0, _Gpu1], ids=["current", "other"])
def test_runs_on_the_tensors_device(machine, name, kind):
    getattr(MM, name)(*arguments(name, [kind] * len(CALLS[name][1])))
    assert machine.calls == [(name, kind.where, handle(kind.where))]
    assert machine.current == 0


@pytest.mark.parametrize("name", sorted(CALLS))
def test_stream_given(machine, name):
    n = len(CALLS[name][1])
    stream = SimpleNamespace(cuda_stream=77, device_index=1)
    getattr(MM, name)(*arguments(name, [_Gpu1] * n), stream=stream)
    assert machine.calls == [(name, 1, 77)]
    with pytest.raises(ValueError, match="stream"):
        getattr(MM, name)(*arguments(name, [_Gpu0] * n), stream=stream)
    assert len(machine.calls) == 1


@pytest.mark.parametrize("name", sorted(set(CALLS) - {"megamoe_last_error"}))
def test_tensors_of_two_devices_are_refused(machine, name):
    n = len(CALLS[name][1])
    for at in range(n):
        kinds = [_Gpu1 if i == at else _Gpu0 for i in range(n)]
        with pytest.raises(ValueError, match="one device"):
            getattr(MM, name)(*arguments(name, kinds))
    assert machine.calls == []


SIZED_BY = {("megamoe_mxfp4_quant", 0), ("megamoe_mxfp4_dequant", 2)}  # no sizes without these


@pytest.mark.parametrize("name", sorted(CALLS))
def test_nothing_for_a_tensor(name):
    """None is a null pointer, which the library refuses with its own error."""
    n = len(CALLS[name][1])
    if torch.cuda.device_count():
        pytest.skip("passes host addresses; host-only")
    for at in range(n):
        if CALLS[name][1][at] is WS or (name, at) in SIZED_BY:
            continue
        with pytest.MonkeyPatch.context() as patch:
            patch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
            patch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
            args = arguments(name, [_Gpu0] * n)
            args[at + CALLS[name][0]] = None
            with pytest.raises(MM.MegaMoEError) as err:
                getattr(MM, name)(*args)
            assert err.value.status == 1, at
