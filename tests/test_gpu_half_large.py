"""What the smaller problems of test_gpu_half.py and test_gpu_norm.py do not reach: workgroups that look up their tiles several
times, and that go on to further tokens at every width."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from tests import half64 as P  # noqa: E402
from tests import test_gpu_half as G  # noqa: E402
from tests import test_gpu_norm as N  # noqa: E402

pytestmark = pytest.mark.gpu
_gpu = G._gpu


@pytest.mark.parametrize("counts", [[9000, 0, 31, 7900, 300], [6000, 6001, 5200]])
def test_products_of_many_tiles(counts):
    """More than 32 tiles to each of 256 workgroups, of every size, an incomplete last round among them."""
    c = G.Case(sum(counts), 128, len(counts), 1, 16384, G.counted(counts), torch.bfloat16)
    assert sum((n + 255) // 256 for n in counts) * 128 > 32 * 256
    out, y = c.out(2 * c.I), c.out(c.I)
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, out)
    H.megamoe_half_gmm1_swiglu(c.d, c.x, c.route, c.end, c.w1, y, probs=c.probs)
    v, b = P.product(c.x, c.token, c.w1, c.end, c.R)
    for i in range(0, c.R, 1000):
        near = slice(i, i + 1000)
        G.near("gmm1", out[near], v[near], b[near], c.t)
        w, e = P.swiglu(v[near], c.p[near], b[near])
        G.near("gmm1_swiglu", y[near], w, e, c.t)
    del v, b, out, y
    # as many tiles the other way: the weights' gradient, all of whose rows are there
    dw = torch.full((c.E, 2 * c.I, c.K), math.nan, dtype=c.t, device="cuda")
    H.megamoe_half_gmm1_wgrad(c.d, c.dc, c.x, c.route, c.end, dw)
    v, b = P.weights(c.dc, None, c.x, c.token, c.end, c.E)
    G.near("gmm1_wgrad", dw, v, b, c.t)


@pytest.mark.parametrize("M,K,x,rows,h,k,after,gate,with_dr,before", [
    (600, 7168, "bf16", "bf16", "bf16", 3, True, "channel", True, True),
    (530, 8192, "fp32", "fp16", "bf16", 0, True, "token", True, True),
    (300, 12288, "bf16", "bf16", "bf16", 2, True, "channel", True, True),
    (1500, 4096, "fp32", "bf16", "bf16", 2, True, "one", True, True),
    (2200, 2048, "fp16", "fp16", "fp16", 2, True, "channel", True, True),
    (2100, 512, "bf16", "bf16", "fp32", 1, True, "element", False, True),
])
def test_norm_gradients_over_several_tokens(M, K, x, rows, h, k, after, gate, with_dr, before):
    N.test_norm_gradients(M, K, x, rows, h, k, after, gate, with_dr, before)


EDGES = [[63, 64, 65], [0, 0, 127, 128, 129, 0], [191, 192, 193], [255, 256, 257], [511, 512, 513, 0], [40, 1, 300, 31, 33]]


def _wide(K, I):
    for t in ("bf16", "fp16"):
        for c in EDGES:
            yield pytest.param(lambda c=c, t=t: G.Case(sum(c), K, len(c), 1, I, G.counted(c), G.T[t]),
                               id=f"{t}-K{K}-I{I}-rows-" + "-".join(map(str, c)))
        for how in ("drop", "zipf", "one", "none", "twice"):
            yield pytest.param(lambda how=how, t=t: G.Case(130, K, 5, 2, I, G.make_ids(130, 5, 2, how, 7), G.T[t]),
                               id=f"{t}-K{K}-I{I}-{how}")


# so wide that few rows make many tiles, and the other way about: each product meets the kernel of many tiles in one of them
WIDE = list(_wide(256, 8192)) + list(_wide(8192, 256))


@pytest.mark.parametrize("case", WIDE)
def test_wide_products(case):
    G.test_products(case)


@pytest.mark.parametrize("case", WIDE)
def test_wide_row_gradients(case):
    G.test_row_gradients(case)


@pytest.mark.parametrize("case", WIDE)
def test_wide_weight_gradients(case):
    G.test_weight_gradients(case)


@pytest.mark.parametrize("t", sorted(G.T))
@pytest.mark.parametrize("M,K,I", [(200, 256, 8192), (200, 8192, 256), (40, 2048, 256)])
def test_nothing_leaks_between_wide_groups(M, K, I, t, monkeypatch):
    case = G.Case
    monkeypatch.setattr(G, "Case", lambda m, k, E, top_k, i, ids, kind: case(M, K, E, top_k, I, ids[:M].contiguous(), kind))
    G.test_nothing_leaks_between_groups(t)


@pytest.mark.parametrize("M", [70, 200])
def test_largest_widths(M):
    """K and I at their limits: an expert's weights are 2^31 bytes."""
    case = G.Case(M, 32768, 2, 1, 16384, G.counted([M // 2 - 3, M - M // 2 + 3]), torch.bfloat16)
    G.test_products(lambda: case)
    torch.cuda.empty_cache()
    G.test_row_gradients(lambda: case)
    torch.cuda.empty_cache()
    # the weights' gradient, whole rows of it: an expert's in 64 bits would be 8 GiB each for values and bounds
    dw = torch.full((2, 2 * case.I, case.K), math.nan, dtype=case.t, device="cuda")
    H.megamoe_half_gmm1_wgrad(case.d, case.dc, case.x, case.route, case.end, dw)
    assert torch.isfinite(dw).all()
    for rows in (slice(0, 300), slice(16300, 16500), slice(32468, 32768)):
        v, b = P.weights(case.dc[:, rows], None, case.x, case.token, case.end, 2)
        G.near("gmm1_wgrad", dw[:, rows], v, b, case.t)


def test_rows_of_nearly_2_to_32_bytes():
    case = G.Case(65000, 32768, 5, 1, 128, G.counted([20000, 3, 0, 24997, 20000]), torch.bfloat16)
    assert 0.98 * 2 ** 31 < case.R * case.K < 2 ** 31
    out = case.out(2 * case.I)
    H.megamoe_half_gmm1(case.d, case.x, case.route, case.end, case.w1, out)
    v, b = P.product(case.x, case.token, case.w1, case.end, case.R)
    G.near("gmm1", out, v, b, case.t)
    dw = torch.full((5, 2 * case.I, case.K), math.nan, dtype=case.t, device="cuda")
    H.megamoe_half_gmm1_wgrad(case.d, case.dc, case.x, case.route, case.end, dw)
    v, b = P.weights(case.dc, None, case.x, case.token, case.end, 5)
    G.near("gmm1_wgrad", dw, v, b, case.t)
    dy = case.out(case.I)
    H.megamoe_half_gmm2_dgrad(case.d, case.dout, case.route, case.end, case.w2, dy)
    v, b = P.product(case.dout, case.token, case.w2, case.end, case.R, transposed=True)
    G.near("gmm2_dgrad", dy, v, b, case.t)
    dx = case.out(case.K)
    H.megamoe_half_gmm1_dgrad(case.d, case.dc, case.end, case.w1, dx)
    for lo, hi in ((0, 300), (19990, 20010), (44900, 45100), (64700, 65000)):
        end = (case.end - lo).clamp(0, hi - lo)
        v, b = P.product(case.dc[lo:hi], None, case.w1, end, hi - lo, transposed=True)
        G.near("gmm1_dgrad", dx[lo:hi], v, b, case.t)
