"""Norms of rows whose squares pass fp32's range: 0 for that row, as the header says, and nothing for the others."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402

pytestmark = pytest.mark.gpu
CU = dict(device="cuda")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [128, 4096, 8320])
def test_norm_past_the_range_of_squares(t, K):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    M, d = 4, MM.dims(4, K, 4, 1, 128)
    g = torch.Generator(device="cuda").manual_seed(K)
    x, rows = torch.randn((M, K), generator=g, **CU).to(t), torch.randn((M, K), generator=g, **CU).to(t)
    w = torch.ones(K, **CU)
    out = lambda: [torch.full((M, K), math.nan, dtype=t, **CU) for _ in range(3)]
    want, got = out(), out()
    H.megamoe_norm(d, x=x, rows=rows, w_after=w, w_before=w, s=want[0], r=want[1], h=want[2])
    rows[1], x[2] = 1e25, -1e25
    H.megamoe_norm(d, x=x, rows=rows, w_after=w, w_before=w, s=got[0], r=got[1], h=got[2])
    for a, b in zip(got, want):
        assert torch.equal(a[[0, 3]], b[[0, 3]])
    assert torch.equal(got[0], rows) and torch.equal(got[1][1], x[1])  # the norm after: 0
    assert not got[2][2].any() and torch.isfinite(got[2]).all()        # the norm before: 0
