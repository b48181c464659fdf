"""Gradients of the weights where a workgroup has more tiles than it looks up at a time: the list is filled again while
the copies of stages to come are under way, tiles of one stage and of several among them, and experts without rows."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from tests import half64 as P  # noqa: E402
from tests import test_gpu_half as G  # noqa: E402

pytestmark = pytest.mark.gpu
_gpu = G._gpu

COUNTS = [1, 130, 0, 64, 97, 33, 2, 65, 0, 128, 63]
K, I = 8192, 8192


@pytest.fixture(scope="module", params=sorted(G.T))
def case(request):
    c = G.Case(sum(COUNTS), K, len(COUNTS), 1, I, G.counted(COUNTS), G.T[request.param])
    c.w1 = c.w2 = None
    torch.cuda.empty_cache()
    yield c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("accumulate", [False, True], ids=["written", "added"])
@pytest.mark.parametrize("out", ["16", "fp32"])
@pytest.mark.parametrize("first", [True, False], ids=["gmm1", "gmm2"])
def test_weight_gradients_of_many_tiles(case, first, out, accumulate):
    c, t = case, case.t if out == "16" else torch.float32
    rows, cols = (2 * I, K) if first else (K, I)
    full = sum(n > 0 for n in COUNTS) * (rows // 256) * (cols // 256)
    assert full > 33 * 256  # with rows, of 256 workgroups at most: past the first filling of the list
    dw = torch.full((c.E, rows, cols), math.nan, dtype=t, **G.CU)
    if accumulate:
        for e in range(c.E):
            dw[e] = torch.randn((rows, cols), generator=c.g, **G.CU)
    old = dw.clone()
    if first:
        H.megamoe_half_gmm1_wgrad(c.d, c.dc, c.x, c.route, c.end, dw, accumulate=accumulate)
    else:
        H.megamoe_half_gmm2_wgrad(c.d, c.dout, c.y, c.route, c.end, dw, accumulate=accumulate)
    for e, n in enumerate(COUNTS):
        if n == 0:
            assert G.same_bits(dw[e], old[e]) if accumulate else not dw[e].any()
    for lo in range(0, rows, 1024):  # all of it, some rows at a time
        at = slice(lo, lo + 1024)
        if first:
            v, b = P.weights(c.dc[:, at], None, c.x, c.token, c.end, c.E)
        else:
            v, b = P.weights(c.dout[:, at], c.token, c.y, None, c.end, c.E)
        if accumulate:  # one more fp32 addition
            v = v + old[:, at].double()
            b = b + v.abs() * P.U * 2
        G.near("wgrad", dw[:, at], v, b, t)
