"""Products of fp16 rows that are subnormal, as small gradients are: they count, and how exactly.

A matrix instruction takes a subnormal operand as it is stored, 0.f times 2^-14, and adds the products aligned to their
exponents before it rounds: a product with a subnormal operand is as exact as one with 2^-14 in its place.  So the bound of
half64.py holds with S = sum max(|a|, 2^-14) max(|b|, 2^-14) over the products that are not 0."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from tests import half64 as P  # noqa: E402
from tests import test_gpu_half as G  # noqa: E402

pytestmark = pytest.mark.gpu
_gpu = G._gpu


def magnitude(v):
    a = v.double().abs()
    return torch.where(a > 0, a.clamp_min(2.0 ** -14), a)


def bound(a, b, n):
    """Of a [., n] times b [n, .]."""
    return (magnitude(a) @ magnitude(b)) * ((n / 16 + 17) * 2 * P.U)


def subnormal(g, *shape):
    return (torch.randint(-1023, 1024, shape, generator=g, device="cuda").double() * 2.0 ** -24).half()


# few tiles, few rows an expert, many tiles
@pytest.mark.parametrize("M,K,E,k,I", [(200, 256, 4, 2, 256), (80, 2048, 16, 2, 1024), (130, 256, 5, 2, 8192), (130, 8192, 5, 2, 256)])
def test_subnormal_rows(M, K, E, k, I):
    c = G.Case(M, K, E, k, I, G.make_ids(M, E, k, "drop", M), torch.float16)
    c.x, c.dout = subnormal(c.g, M, K), subnormal(c.g, M, K)
    c.y, c.dc = subnormal(c.g, c.R, I), subnormal(c.g, c.R, 2 * I)
    c.y[c.n:], c.dc[c.n:] = math.nan, math.nan
    # the second factors are large enough for results that are not subnormal themselves
    c.w1, c.w2 = c.w1 * 64, c.w2 * 64
    x1 = (torch.randn((M, K), generator=c.g, device="cuda") * 4).half()
    y1 = (torch.randn((c.R, I), generator=c.g, device="cuda") * 4).half()
    out = dict(gmm1=c.out(2 * I), gmm2=c.out(K), d1=c.out(K), d2=c.out(I))
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, out["gmm1"])
    H.megamoe_half_gmm2(c.d, c.y, c.end, c.w2, out["gmm2"])
    H.megamoe_half_gmm1_dgrad(c.d, c.dc, c.end, c.w1, out["d1"])
    H.megamoe_half_gmm2_dgrad(c.d, c.dout, c.route, c.end, c.w2, out["d2"])
    dw1, dw2 = torch.full((E, 2 * I, K), math.nan, device="cuda"), torch.full((E, K, I), math.nan, device="cuda")
    H.megamoe_half_gmm1_wgrad(c.d, c.dc, x1, c.route, c.end, dw1)
    H.megamoe_half_gmm2_wgrad(c.d, c.dout, y1, c.route, c.end, dw2)
    for e, b, n in P.groups(c.end):
        t = c.token[b:n]
        for name, a, w in (("gmm1", c.x[t], c.w1[e].t()), ("gmm2", c.y[b:n], c.w2[e].t()), ("d1", c.dc[b:n], c.w1[e]),
                           ("d2", c.dout[t], c.w2[e])):
            want = a.double() @ w.double()
            assert want.abs().max() > 2.0 ** -14
            G.near(name, out[name][b:n], want, bound(a, w, a.shape[1]), torch.float16)
        for name, a, w, got in (("w1", c.dc[b:n].t(), x1[t], dw1[e]), ("w2", c.dout[t].t(), y1[b:n], dw2[e])):
            G.near(name, got, a.double() @ w.double(), bound(a, w, n - b), torch.float32)
