"""Host-side refusals of the router, the few-token layer and the MXFP4 entry points
(no GPU needed): every bad argument is answered by its status, with nothing launched."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402

GOOD, ODD = 0x10000, 0x10004
P, SZ, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64

# pointer positions (after the dims), which of them are nullable
_CALLS = {
    "megamoe_forward_few": (9, (), True),
    "megamoe_forward_mxfp4": (9, (), True),
    "megamoe_mxfp4_gmm1": (7, (), False),
    "megamoe_mxfp4_gmm2": (6, (), False),
}

# the entry points below are given placeholder addresses
pytestmark = pytest.mark.skipif(torch.cuda.device_count() != 0,
                                reason="passes placeholder device addresses; host-only")


@pytest.mark.parametrize("name", sorted(_CALLS))
def test_null_and_misaligned_pointers(name):
    n, nullable, sized = _CALLS[name]
    fn = getattr(MM.load(), name)
    d = MM.dims(16, 256, 4, 2, 128)
    for pos in range(n):
        for bad in (0, ODD):
            ptrs = [GOOD] * n
            ptrs[pos] = bad
            args = [ctypes.byref(d)] + [P(v) if v else None for v in ptrs]
            args += [SZ(1 << 40)] if sized else []
            assert fn(*args, None) == 1, (name, pos, bad)
    assert fn(None, *([P(GOOD)] * n), *([SZ(1 << 40)] if sized else []), None) == 1


@pytest.mark.parametrize("name", sorted(_CALLS))
def test_dims(name):
    n, _, sized = _CALLS[name]
    fn = getattr(MM.load(), name)
    for bad, code in ((MM.dims(0, 256, 4, 2, 128), 1), (MM.dims(4, 200, 4, 2, 128), 2),
                      (MM.dims(4, 256, 4, 5, 128), 2), (MM.dims(4, 256, 300, 2, 128), 2),
                      (MM.dims(4, 256, 4, 2, 192), 2)):
        args = [ctypes.byref(bad)] + [P(GOOD)] * n + ([SZ(1 << 40)] if sized else [])
        assert fn(*args, None) == code, bad


def test_route_refusals():
    fn = MM.load().megamoe_route
    d = MM.dims(16, 256, 4, 2, 128)

    def call(logits=GOOD, kind=0, bias=0, ids=GOOD, probs=GOOD, dims=d):
        q = [P(v) if v else None for v in (logits, bias, ids, probs)]
        return fn(ctypes.byref(dims), q[0], kind, q[1], 1, q[2], q[3], None)

    for key in ("logits", "ids", "probs"):
        assert call(**{key: 0}) == 1 and call(**{key: ODD}) == 1
    assert call(bias=ODD) == 1
    for kind in (-1, 3, 99):
        assert call(kind=kind) == 1
    assert call(dims=MM.dims(16, 256, 4, 5, 128)) == 2


def test_few_limits():
    lib = MM.load()
    for bad in (MM.dims(17, 256, 64, 2, 128), MM.dims(16, 256, 64, 33, 128)):
        n = SZ(0)
        assert lib.megamoe_few_workspace_bytes(ctypes.byref(bad), ctypes.byref(n)) == 2
        assert lib.megamoe_forward_few(ctypes.byref(bad), *([P(GOOD)] * 9), SZ(1 << 40), None) == 2
    d = MM.dims(16, 256, 64, 32, 128)
    need = MM.megamoe_few_workspace_bytes(d)
    assert need >= 512 * 128 * 4 + 512 * 8 * 4 + 4
    assert lib.megamoe_forward_few(ctypes.byref(d), *([P(GOOD)] * 9), SZ(need - 1), None) == 3
    assert lib.megamoe_few_workspace_bytes(ctypes.byref(d), None) == 1


def test_mxfp4_workspace():
    lib = MM.load()
    d = MM.dims(64, 256, 8, 2, 128)
    need = MM.megamoe_mxfp4_workspace_bytes(d)
    assert need >= 64 * 136 + 128 * 68 + 128 * 256 * 2  # quantised x and y, the second product's rows
    assert lib.megamoe_forward_mxfp4(ctypes.byref(d), *([P(GOOD)] * 9), SZ(need - 1), None) == 3
    assert lib.megamoe_mxfp4_workspace_bytes(ctypes.byref(d), None) == 1


@pytest.mark.parametrize("back", [False, True])
def test_mxfp4_rows_refusals(back):
    lib = MM.load()

    def call(a=GOOD, b=GOOD, c=GOOD, valid=0, kind=1, rows=4, cols=64):
        a, b, c, v = (P(x) if x else None for x in (a, b, c, valid))
        if back:
            return lib.megamoe_mxfp4_dequant(a, b, I64(rows), I64(cols), v, c, kind, None)
        return lib.megamoe_mxfp4_quant(a, kind, I64(rows), I64(cols), v, b, c, None)

    for key in ("a", "b", "c"):
        assert call(**{key: 0}) == 1 and call(**{key: ODD}) == 1
    assert call(valid=0x10002) == 1
    for kind in (-1, 3):
        assert call(kind=kind) == 1
    for rows, cols, code in ((0, 64, 1), (-1, 64, 1), (4, 0, 1), (4, -32, 1), (4, 48, 2), (4, 16, 2),
                             (1 << 40, 64, 2), (1, 1 << 30, 2), ((1 << 63) - 1, 32, 2)):
        assert call(rows=rows, cols=cols) == code, (rows, cols)


def test_binding_checks_shapes_and_types():
    """The Python names refuse tensors of another shape, type or place before any call."""
    d = MM.dims(4, 256, 8, 2, 128)
    x, ids, pr = torch.zeros(4, 256).half(), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):  # on the CPU
        MM.megamoe_route(d, torch.zeros(4, 8), ids, pr)
    with pytest.raises(ValueError):
        MM.megamoe_route(d, torch.zeros(4, 9), ids, pr)
    with pytest.raises(ValueError):
        MM.megamoe_mxfp4_quant(x, torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 7, dtype=torch.uint8))
    with pytest.raises(ValueError):
        MM.megamoe_mxfp4_quant(x[0], torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8))
    with pytest.raises(ValueError):
        MM.megamoe_mxfp4_gmm2(d, torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8),
                              torch.zeros(8, dtype=torch.int32), torch.zeros(8, 256, 64, dtype=torch.uint8),
                              torch.zeros(8, 255, 4, dtype=torch.uint8), torch.zeros(8, 256).half())
    with pytest.raises(ValueError):
        MM.megamoe_forward_few(d, x[:3], ids, pr, None, None, None, None, x, x)
