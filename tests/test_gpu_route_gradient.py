"""The router's gradient on the GPU, every expert's against a bound of its own: experts of small weight, which are most of
many, have to be right by their own size."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests import half64 as P  # noqa: E402

CU = dict(device="cuda")
T = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def exact(x, bias, ids, dprobs, renormalize):
    """dlogits [M, E] in 64 bits from the definition w[e] (g[e] - sum w g), and the bound of its fp32 arithmetic.

    u = 2^-24.  A weight's exponent x - most is rounded, multiplied by a rounded log2(e) and rounded again: 3 u of its
    magnitude, at most the spread D of the row, and the exponential is off by 2 u.  The sum of the exponentials inherits
    (3 D + 2) u and adds 16 u (8 in a lane, at most 8 across lanes), the quotient 3 u: (6 D + 24) u of the weight.  An exponent
    below -126 may give 0: 2^-126.  The dot product over k slots inherits the weights' errors and adds (k + 2) u of its
    magnitudes; the difference and its product are rounded once each."""
    M, E = x.shape
    k = ids.shape[1]
    x, g1 = x.double(), dprobs.double()
    part = (x if bias is None else x + bias.double()) > -math.inf
    slots = (ids >= 0) & (ids < E)
    rows = torch.arange(M, device=x.device).unsqueeze(1).expand(M, k)
    if renormalize:
        part = torch.zeros_like(part)
        part[rows[slots], ids.long()[slots]] = True
    x = torch.where(part, x, -math.inf)
    some = part.any(1, keepdim=True)
    w = torch.where(some, torch.softmax(torch.where(some, x, 0.0), 1), 0.0)
    g = torch.zeros_like(x)
    g.index_put_((rows[slots], ids.long()[slots]), g1[slots], accumulate=True)
    dot, size = (w * g).sum(1, keepdim=True), (w * g.abs()).sum(1, keepdim=True)
    most, least = x.amax(1, keepdim=True), torch.where(part, x, math.inf).amin(1, keepdim=True)
    spread = torch.where(some, most - least, 0.0)
    rel = (6 * spread + 24) * P.U
    want = w * (g - dot)
    bound = want.abs() * (rel + 3 * P.U) + w * size * (rel + (k + 2) * P.U) + torch.where(part, 2.0 ** -126 * (g.abs() + size), 0.0)
    return want, bound, part


def held_to(got, want, bound, t):
    """Where got is off by more than its bound and one rounding to t."""
    return (got.double() - want).abs() > bound + P.half_step(want.abs() + bound, t)


def problem(M, E, k, t, scale, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)
    x = (torch.randn((M, E), generator=g, device=device) * scale).to(t)
    x[M // 2, ::2] = -math.inf
    x[M // 3] = -math.inf
    bias = torch.randn(E, generator=g, device=device) * 0.5
    bias[E // 2] = -math.inf
    return x, bias, torch.randn((M, k), generator=g, device=device)


@pytest.mark.parametrize("renormalize", [True, False])
def test_the_bound_is_tight(renormalize):
    """On the CPU: a kernel that loses an expert of small weight, or takes the sum from another row, is found in nearly
    every place; the exact result passes."""
    x, bias, dp = problem(40, 256, 8, torch.float32, 3.0, 0, "cpu")
    score = torch.where(torch.isnan(x + bias), -math.inf, x + bias)
    top, ids = torch.sort(score, 1, descending=True)
    ids = torch.where(top[:, :8] > -math.inf, ids[:, :8], -1).int()
    want, bound, part = exact(x, bias, ids, dp, renormalize)
    assert not held_to(want, want, bound, torch.float32).any()
    part = part & (want != 0)
    lost = held_to(torch.zeros_like(want), want, bound, torch.float32)[part]
    shifted = held_to(want * (1 + 1e-3), want, bound, torch.float32)[part]
    assert lost.float().mean() > 0.99 and shifted.float().mean() > 0.95


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.3, 3.0, 30.0])
@pytest.mark.parametrize("kind", sorted(T))
@pytest.mark.parametrize("M,E,k", [(3, 8, 2), (130, 32, 8), (70, 33, 4), (257, 64, 6), (130, 255, 7), (300, 256, 8), (40, 256, 70),
                                   (65, 65, 65)])
def test_every_experts_gradient(M, E, k, kind, scale):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, bias, dp = problem(M, E, k, T[kind], scale, M + E, "cuda")
    d = MM.dims(M, 128, E, k, 128)
    for b in (None, bias):
        for renormalize in (True, False):
            ids, probs = torch.empty((M, k), dtype=torch.int32, **CU), torch.empty((M, k), **CU)
            MM.megamoe_route(d, x, ids, probs, bias=b, renormalize=renormalize)
            out = torch.full((M, E), math.nan, dtype=T[kind], **CU)
            H.megamoe_route_grad(d, x, ids, probs, dp, out, bias=b, renormalize=renormalize)
            want, bound, part = exact(x, b, ids, dp, renormalize)
            assert torch.isfinite(out).all() and (out[~part] == 0).all()
            off = held_to(out, want, bound, T[kind])
            assert not off.any(), (int(off.sum()), ((out.double() - want).abs() / bound)[off].max().item())
