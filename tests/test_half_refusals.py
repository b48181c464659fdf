"""Host-side refusals of the 16-bit products, SwiGLU, the norms and the router's gradient (no GPU needed): every bad
argument is answered by its status, or by the binding's exception, with nothing launched."""
from __future__ import annotations

import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402

GOOD, ODD = 0x10000, 0x10004
P, SZ, I64, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
D = MM.dims(16, 256, 4, 2, 128)

# the entry points below are given placeholder addresses
pytestmark = pytest.mark.skipif(torch.cuda.device_count() != 0,
                                reason="passes placeholder device addresses; host-only")

# arguments after the dims: "p" a pointer, "n" a nullable one, "t" a 16-bit type, "w" the weights' type, "l" any type,
# "0" a plain integer, "s" the workspace's size
_CALLS = {
    "megamoe_sort_routes": "pppppps",
    "megamoe_half_gmm1": "ptpppp",
    "megamoe_half_gmm1_swiglu": "ptppnpp",
    "megamoe_half_gmm2": "ptppp",
    "megamoe_half_gmm1_dgrad": "ptppp",
    "megamoe_half_gmm2_dgrad": "ptpppp",
    "megamoe_half_gmm1_wgrad": "pptpppw0",
    "megamoe_half_gmm2_wgrad": "pptpppw0",
    "megamoe_half_swiglu": "ptppnp",
    "megamoe_half_swiglu_grad": "pptpppnpn",
    "megamoe_route_grad": "pln0pppp",
    "megamoe_forward_half": "ptpppppps",
}


def call(name, d=D, change=None):
    args = []
    for i, kind in enumerate(_CALLS[name]):
        v = {"p": GOOD, "n": GOOD, "t": 2, "w": 2, "l": 0, "0": 1, "s": 1 << 40}[kind]
        v = change[i] if change and i in change else v
        args.append((P(v) if v else None) if kind in "pn" else SZ(v) if kind == "s" else v)
    return getattr(MM.load(), name)(None if d is None else ctypes.byref(d), *args, None)


@pytest.mark.parametrize("name", sorted(_CALLS))
def test_pointers_types_and_dims(name):
    for i, kind in enumerate(_CALLS[name]):
        if kind == "p":
            assert call(name, change={i: 0}) == 1 and call(name, change={i: ODD}) == 1
        elif kind == "n":
            assert call(name, change={i: ODD}) == 1
        elif kind == "t":
            for v in (-1, 0, 3):
                assert call(name, change={i: v}) == 1
        elif kind == "l":
            for v in (-1, 3):
                assert call(name, change={i: v}) == 1
        elif kind == "w":
            for v in (-1, 1, 3):  # the rows are bf16: neither fp16 nor a type that is none
                assert call(name, change={i: v}) == 1
    assert call(name, d=None) == 1
    for bad, code in ((MM.dims(0, 256, 4, 2, 128), 1), (MM.dims(4, 200, 4, 2, 128), 2), (MM.dims(4, 256, 4, 5, 128), 2),
                      (MM.dims(4, 256, 300, 2, 128), 2), (MM.dims(4, 256, 4, 2, 192), 2),
                      (MM.dims(1 << 20, 32768, 8, 8, 128), 2)):
        assert call(name, d=bad) == code


def test_weight_gradients_limit():
    """Their rows end 64 rows before the other entry points' do."""
    d = MM.dims((1 << 31) // 32768 - 64, 32768, 8, 1, 128)
    assert MM.megamoe_check_dims(d) == 0
    for name in ("megamoe_half_gmm1_wgrad", "megamoe_half_gmm2_wgrad"):
        assert call(name, d=d) == 2


def test_workspaces():
    lib = MM.load()
    for name, size in (("megamoe_sort_routes", MM.megamoe_permute_workspace_bytes(D)),
                       ("megamoe_forward_half", H.megamoe_half_workspace_bytes(D))):
        assert call(name, change={_CALLS[name].index("s"): size - 1}) == 3
    assert H.megamoe_half_workspace_bytes(D) >= 32 * 128 * 2 + 32 * 256 * 2
    for fn in (lib.megamoe_half_workspace_bytes, lib.megamoe_norm_grad_workspace_bytes):
        assert fn(ctypes.byref(D), None) == 1
        n = SZ(0)
        assert fn(ctypes.byref(MM.dims(4, 200, 4, 2, 128)), ctypes.byref(n)) == 2


def norm(d=D, x=GOOD, x_type=2, rows=GOOD, rows_type=2, idx=GOOD, w_after=GOOD, gate=GOOD, gate_type=0, gate_rows=1,
         gate_cols=1, alpha=1.0, w_before=GOOD, eps=1e-6, s=GOOD, r=GOOD, h=GOOD, h_type=2):
    q = lambda v: P(v) if v else None
    return MM.load().megamoe_norm(ctypes.byref(d), q(x), x_type, q(rows), rows_type, q(idx), q(w_after), q(gate), gate_type,
                                  I64(gate_rows), I64(gate_cols), F(alpha), q(w_before), F(eps), q(s), q(r), q(h), h_type, None)


def test_norm():
    for key in ("x", "rows", "idx", "w_after", "gate", "w_before", "s", "r", "h"):
        assert norm(**{key: ODD}) == 1, key
    assert norm(x=0, rows=0, idx=0, w_after=0, gate=0, s=0) == 1          # nothing to read
    assert norm(s=0, r=0, h=0, w_before=0) == 1                           # nothing to write
    assert norm(h=0) == 1 and norm(w_before=0) == 1                       # one without the other
    for key in ("idx", "w_after", "gate", "s"):                           # parts of a block that is not there
        rest = dict(idx=0, w_after=0, gate=0, s=0, rows=0)
        rest[key] = GOOD
        assert norm(**rest) == 1, key
    for key in ("x_type", "rows_type", "h_type", "gate_type"):
        assert norm(**{key: 3}) == 1 and norm(**{key: -1}) == 1
    for rows, cols in ((2, 1), (1, 2), (0, 1), (16, 255), (15, 256), (1, 0), (1 << 32 | 1, 1)):
        assert norm(gate_rows=rows, gate_cols=cols) == 1
    for eps in (0.0, -1e-6, math.inf, math.nan):
        assert norm(eps=eps) == 1
    assert norm(alpha=math.nan) == 1 and norm(alpha=math.inf) == 1
    assert norm(d=MM.dims(16, 200, 4, 2, 128)) == 2


def grad(d=D, dr=GOOD, r=GOOD, x_type=2, dh=GOOD, h_type=2, idx=GOOD, s=GOOD, rows_type=2, w_after=GOOD, gate=GOOD,
         gate_type=0, gate_rows=1, gate_cols=1, alpha=1.0, w_before=GOOD, eps=1e-6, dx=GOOD, ds=GOOD, dw_after=GOOD,
         dw_before=GOOD, dgate=GOOD, ws=GOOD, size=1 << 40):
    q = lambda v: P(v) if v else None
    return MM.load().megamoe_norm_grad(ctypes.byref(d), q(dr), q(r), x_type, q(dh), h_type, q(idx), q(s), rows_type,
                                       q(w_after), q(gate), gate_type, I64(gate_rows), I64(gate_cols), F(alpha), q(w_before),
                                       F(eps), q(dx), q(ds), q(dw_after), q(dw_before), q(dgate), q(ws), SZ(size), None)


def test_norm_grad():
    for key in ("dr", "r", "dh", "idx", "s", "w_after", "gate", "w_before", "dx", "ds", "dw_after", "dw_before", "dgate", "ws"):
        assert grad(**{key: ODD}) == 1, key
    for key in ("r", "dh", "w_before", "dx", "ds", "s", "dw_after", "dw_before", "dgate", "gate", "w_after", "ws"):
        assert grad(**{key: 0}) == 1, key                                 # something that the rest asks for
    assert grad(dr=0, dh=0, w_before=0, dw_before=0, r=0, idx=0) == 1     # no gradient at all
    assert grad(dh=0, w_before=0, dw_before=0, r=0) == 1                  # rows of a gradient that is not there
    for key in ("x_type", "rows_type", "h_type", "gate_type"):
        assert grad(**{key: 3}) == 1 and grad(**{key: -1}) == 1
    assert grad(gate_rows=2) == 1 and grad(gate_cols=128) == 1
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert grad(eps=eps) == 1
    assert grad(alpha=math.inf) == 1
    assert grad(size=H.megamoe_norm_grad_workspace_bytes(D) - 1) == 3
    assert grad(d=MM.dims(16, 200, 4, 2, 128)) == 2


# ---------------------------------------------------------------------------------------------
# the binding: tensors of another shape, type, layout or place, on the CPU

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
M, K, E, k, I = 4, 256, 8, 2, 128
R = M * k
B = MM.dims(M, K, E, k, I)


def z(*shape, t=BF):
    return torch.zeros(shape, dtype=t)


ROUTE, END, ROWOF, PROBS = z(R, t=I32), z(E, t=I32), z(R, t=I32), z(M, k, t=F32)
ARGS = {
    "megamoe_half_gmm1": dict(x=z(M, K), sorted_route=ROUTE, expert_cumsum=END, w1=z(E, 2 * I, K), c=z(R, 2 * I)),
    "megamoe_half_gmm1_swiglu": dict(x=z(M, K), sorted_route=ROUTE, expert_cumsum=END, w1=z(E, 2 * I, K), y=z(R, I), probs=PROBS),
    "megamoe_half_gmm2": dict(y=z(R, I), expert_cumsum=END, w2=z(E, K, I), gmm2_out=z(R, K)),
    "megamoe_half_gmm1_dgrad": dict(dc=z(R, 2 * I), expert_cumsum=END, w1=z(E, 2 * I, K), dx_rows=z(R, K)),
    "megamoe_half_gmm2_dgrad": dict(dout=z(M, K), sorted_route=ROUTE, expert_cumsum=END, w2=z(E, K, I), dy=z(R, I)),
    "megamoe_half_gmm1_wgrad": dict(dc=z(R, 2 * I), x=z(M, K), sorted_route=ROUTE, expert_cumsum=END, dw1=z(E, 2 * I, K)),
    "megamoe_half_gmm2_wgrad": dict(dout=z(M, K), y=z(R, I), sorted_route=ROUTE, expert_cumsum=END, dw2=z(E, K, I)),
    "megamoe_half_swiglu": dict(c=z(R, 2 * I), sorted_route=ROUTE, expert_cumsum=END, y=z(R, I), probs=PROBS),
    "megamoe_half_swiglu_grad": dict(c=z(R, 2 * I), dy=z(R, I), sorted_route=ROUTE, expanded_row_idx=ROWOF, expert_cumsum=END,
                                     dc=z(R, 2 * I), probs=PROBS, dprobs=PROBS),
    "megamoe_sort_routes": dict(expert_idx=z(M, k, t=I32), expanded_row_idx=ROWOF, sorted_route=ROUTE, tokens_per_expert=END,
                                expert_cumsum=END, workspace=z(1 << 16, t=torch.uint8)),
    "megamoe_route_grad": dict(logits=z(M, E), expert_idx=z(M, k, t=I32), probs=PROBS, dprobs=PROBS, dlogits=z(M, E),
                               bias=z(E, t=F32)),
    "megamoe_forward_half": dict(x=z(M, K), expert_idx=z(M, k, t=I32), probs=PROBS, w1=z(E, 2 * I, K), w2=z(E, K, I),
                                 out=z(M, K), workspace=z(1 << 20, t=torch.uint8)),
    "megamoe_norm": dict(x=z(M, K), rows=z(R, K), expanded_row_idx=ROWOF, w_after=z(K, t=F32), gate=z(M, 1, t=F32),
                         w_before=z(K, t=F32), s=z(M, K), r=z(M, K), h=z(M, K)),
    "megamoe_norm_grad": dict(r=z(M, K), workspace=z(1 << 20, t=torch.uint8), dr=z(M, K), dh=z(R, K), expanded_row_idx=ROWOF,
                              s=z(M, K), w_after=z(K, t=F32), gate=z(M, 1, t=F32), w_before=z(K, t=F32), dx=z(M, K),
                              ds=z(M, K), dw_after=z(K, t=F32), dw_before=z(K, t=F32), dgate=z(M, 1, t=F32)),
}


class Answered(Exception):
    """The library was called."""


@pytest.fixture
def as_if_on_gpu(monkeypatch):
    """The binding's checks with CPU tensors in the place of GPU ones: they report device 0, and a call that passes
    every check ends before the library."""
    class Fake(torch.Tensor):
        def get_device(self):
            return 0

    def launch(*a):
        raise Answered
    monkeypatch.setattr(H, "_launch", launch)
    return lambda t: t.as_subclass(Fake)


@pytest.mark.parametrize("name", sorted(ARGS))
def test_binding(name, as_if_on_gpu):
    fn = getattr(H, name)
    with pytest.raises(ValueError, match="GPU"):
        fn(B, **ARGS[name])
    good = {key: as_if_on_gpu(v) for key, v in ARGS[name].items()}
    with pytest.raises(Answered):
        fn(B, **good)
    loose = {"megamoe_norm_grad": ("workspace",), "megamoe_sort_routes": ("workspace",), "megamoe_forward_half": ("workspace",)}
    for key, v in good.items():
        if key in loose.get(name, ()):
            continue
        for bad in (torch.zeros((*v.shape[:-1], v.shape[-1] + 1), dtype=v.dtype), torch.zeros((1, *v.shape), dtype=v.dtype)):
            with pytest.raises(ValueError):
                fn(B, **{**good, key: as_if_on_gpu(bad)})
        with pytest.raises(TypeError):
            fn(B, **{**good, key: as_if_on_gpu(torch.zeros(v.shape, dtype=torch.int64))})
        if v.dim() > 1 and v.shape[-1] > 1:
            wide = torch.zeros((*v.shape[:-1], 2 * v.shape[-1]), dtype=v.dtype)[..., ::2]
            with pytest.raises(ValueError, match="contiguous"):
                fn(B, **{**good, key: as_if_on_gpu(wide)})


def test_mixed_types(as_if_on_gpu):
    """fp16 rows with bf16 weights, and x of one type with r of another."""
    f = as_if_on_gpu
    good = {key: f(v) for key, v in ARGS["megamoe_half_gmm2"].items()}
    with pytest.raises(TypeError):
        H.megamoe_half_gmm2(B, **{**good, "y": f(z(R, I, t=torch.float16))})
    with pytest.raises(TypeError):
        H.megamoe_half_gmm2(B, **{**good, "y": f(z(R, I, t=F32))})
    good = {key: f(v) for key, v in ARGS["megamoe_norm"].items()}
    with pytest.raises(TypeError):
        H.megamoe_norm(B, **{**good, "r": f(z(M, K, t=F32))})
    with pytest.raises(TypeError):
        H.megamoe_norm(B, **{**good, "s": f(z(M, K, t=F32))})
    good = {key: f(v) for key, v in ARGS["megamoe_half_gmm1_wgrad"].items()}
    with pytest.raises(TypeError):
        H.megamoe_half_gmm1_wgrad(B, **{**good, "dw1": f(z(E, 2 * I, K, t=torch.float16))})
    with pytest.raises(Answered):
        H.megamoe_half_gmm1_wgrad(B, **{**good, "dw1": f(z(E, 2 * I, K, t=F32))})


def test_holder():
    with pytest.raises(TypeError):
        H.MegaMoEHalf(4, 256, 8, 2, 128, dtype=torch.float32, device="cpu")
    with pytest.raises(MM.MegaMoEError):
        H.MegaMoEHalf(4, 200, 8, 2, 128, device="cpu")
