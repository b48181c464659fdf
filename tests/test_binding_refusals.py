"""The Python names of the router, the few-token layer and the MXFP4 entry points refuse a tensor of
another shape, type, layout or place, argument by argument, before the library is called: on the CPU
with tensors that say they live on a GPU, and with GPU tensors."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests.test_binding_devices import (BF, F16, F32, I32, I8, IDS, OUT, PROBS, S1, S2, U8, W1P, W1Q, W1S, W2P, W2Q, W2S,  # noqa: E402
                                        X, E, EXPERTS, I, K, M, R, ROWS, TOP_K, _Gpu0, _Gpu1)

# entry point -> its tensors by name; None for the types: fp32, fp16 and bf16
ANY = None
FORWARD = dict(x=X, expert_idx=IDS, probs=PROBS)
CALLS = {
    "megamoe_route": dict(logits=(ANY, (M, E)), expert_idx=IDS, probs=PROBS, bias=(F32, (E,))),
    "megamoe_forward_few": dict(FORWARD, w1p=(I8, W1P), scale1=S1, w2p=(I8, W2P), scale2=S2, out=OUT),
    "megamoe_mxfp4_quant": dict(x=(ANY, (M, K)), q=(U8, (M, K // 2)), scale=(U8, (M, K // 32)), valid_rows=(I32, (1,))),
    "megamoe_mxfp4_dequant": dict(q=(U8, (M, K // 2)), scale=(U8, (M, K // 32)), x=(ANY, (M, K)), valid_rows=(I32, (1,))),
    "megamoe_mxfp4_gmm1": dict(xq=(U8, (M, K // 2)), xs=(U8, (M, K // 32)), sorted_route=ROWS, expert_cumsum=EXPERTS,
                               w1q=W1Q, w1s=W1S, y=(BF, (R, I))),
    "megamoe_mxfp4_gmm2": dict(yq=(U8, (R, I // 2)), ys=(U8, (R, I // 32)), expert_cumsum=EXPERTS, w2q=W2Q, w2s=W2S,
                               gmm2_out=(F16, (R, K))),
    "megamoe_forward_mxfp4": dict(FORWARD, w1q=W1Q, w1s=W1S, w2q=W2Q, w2s=W2S, out=OUT),
}
WORKSPACE = {"megamoe_forward_few": MM.megamoe_few_workspace_bytes, "megamoe_forward_mxfp4": MM.megamoe_mxfp4_workspace_bytes}
ARGS = [(name, arg) for name in CALLS for arg in CALLS[name]]
ids = [f"{name}-{arg}" for name, arg in ARGS]


class Refusals:
    """make(shape, dtype): a tensor in its place; elsewhere: tensors that live elsewhere."""

    def call(self, name, **changed):
        good = {a: self.make(shape, dtype or F16) for a, (dtype, shape) in CALLS[name].items()}
        if name in WORKSPACE:
            d = MM.dims(M, K, E, TOP_K, I)
            good["workspace"] = self.make((WORKSPACE[name](d),), U8)
        first = () if name in ("megamoe_mxfp4_quant", "megamoe_mxfp4_dequant") else (MM.dims(M, K, E, TOP_K, I),)
        getattr(MM, name)(*first, **{**good, **changed})

    @pytest.mark.parametrize("name,arg", ARGS, ids=ids)
    def test_shape(self, called, name, arg):
        dtype, shape = CALLS[name][arg]
        sized = name.startswith("megamoe_mxfp4_") and arg == "x"  # every [rows, cols] is one
        bad = [shape[:-1] + (shape[-1] * 2,), (1,) + shape]
        if len(shape) > 1:
            bad += [(shape[0] - 1,) + shape[1:], (shape[0] + 1,) + shape[1:]]
        if arg in ("w1p", "w2p"):  # flat or not, and longer: packed weights of more experts
            bad = [(shape[0] - 16,), (16,)]
        if arg == "valid_rows":  # one element of any shape
            bad = [(2,), (0,), (1, 3)]
        for s in bad:
            other = "q|scale" if sized and len(s) == 2 else arg  # what no longer fits
            with pytest.raises(ValueError, match=f"^({other}): "):
                self.call(name, **{arg: self.make(s, dtype or F16)})
        assert called == []

    @pytest.mark.parametrize("name,arg", ARGS, ids=ids)
    def test_type(self, called, name, arg):
        dtype, shape = CALLS[name][arg]
        for t in (torch.float64, I8 if dtype is U8 else U8, F32 if dtype in (F16, BF) else torch.int64):
            with pytest.raises(TypeError, match="expected" if dtype is ANY else f"^{arg}: expected"):
                self.call(name, **{arg: self.make(shape, t)})
        assert called == []

    @pytest.mark.parametrize("name,arg", [a for a in ARGS if a[1] != "valid_rows"],
                             ids=[i for i in ids if "valid" not in i])
    def test_layout(self, called, name, arg):
        dtype, shape = CALLS[name][arg]
        bad = self.make(shape[:-1] + (2 * shape[-1],), dtype or F16)[..., ::2]
        with pytest.raises(ValueError, match=f"^{arg}: .*contiguous"):
            self.call(name, **{arg: bad})
        assert called == []

    @pytest.mark.parametrize("name,arg", ARGS, ids=ids)
    def test_place(self, called, name, arg):
        dtype, shape = CALLS[name][arg]
        for bad, why in self.elsewhere(shape, dtype or F16):
            with pytest.raises(ValueError, match=why):
                self.call(name, **{arg: bad})
        assert called == []

    @pytest.mark.parametrize("name", sorted(WORKSPACE))
    def test_workspace(self, called, name):
        need = WORKSPACE[name](MM.dims(M, K, E, TOP_K, I))
        for bad, why in self.elsewhere((need,), U8):
            with pytest.raises(ValueError, match=why):
                self.call(name, workspace=bad)
        with pytest.raises(ValueError, match="^workspace: .*contiguous"):
            self.call(name, workspace=self.make((2 * need,), U8)[::2])
        assert called == []

    def test_the_good_call_is_made(self, called):
        for name in CALLS:
            self.call(name)
        assert called == list(CALLS)


class TestCpu(Refusals):
    def make(self, shape, dtype):
        return torch.zeros(shape, dtype=dtype).as_subclass(_Gpu0)

    def elsewhere(self, shape, dtype):
        t = torch.zeros(shape, dtype=dtype)
        return [(t, "GPU|one device"), (t.as_subclass(_Gpu1), "one device")]

    @pytest.fixture
    def called(self, monkeypatch):
        names = []

        class Library:
            def __getattr__(self, name):
                def entry(*args):
                    names.append(name)
                    return 0
                return entry if not name.endswith("_bytes") else getattr(real, name)

        real = MM.load()
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
        monkeypatch.setattr(MM, "_lib", Library())
        return names


@pytest.mark.gpu
class TestGpu(Refusals):
    def make(self, shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    def elsewhere(self, shape, dtype):
        return [(torch.zeros(shape, dtype=dtype), "GPU|one device")]

    @pytest.fixture
    def called(self, monkeypatch):
        if not torch.cuda.is_available():
            pytest.skip("no GPU")
        names, launch = [], MM._launch
        monkeypatch.setattr(MM, "_launch", lambda name, *args: (names.append(name), launch(name, *args)))
        return names

    def test_workspace_size(self, called):
        for name in sorted(WORKSPACE):
            need = WORKSPACE[name](MM.dims(M, K, E, TOP_K, I))
            with pytest.raises(MM.MegaMoEError) as err:
                self.call(name, workspace=self.make((need - 1,), U8))
            assert err.value.status == 3
