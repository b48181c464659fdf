"""The few-token layer and the MXFP4 layer at the sizes where their kernels go round more than once:
several runs of experts, several tiles to a workgroup, several row blocks to an expert; and the MXFP4
layer against the whole layer in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from oracle import oracle as O  # noqa: E402
from tests import gpu_helpers as H  # noqa: E402
from tests.test_gpu_operators import (CU, U24, drop_some, few_case, groups, mx_forward, mx_layer, mx_values64,  # noqa: E402
                                      one_expert, run_few, run_gmm, run_quant, same_bits)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


# ---------------------------------------------------------------------------------------------
# few tokens, with 32 output columns to a workgroup (K >= 6144)

FEW_WIDE = [
    (16, 7168, 32, 8, 2048, "uniform", None),      # 128 pairs, 32 rows to a buffer: runs of experts
    (16, 6144, 48, 24, 512, "uniform", None),      # 384 pairs: past the eight early channel scales of a thread
    (16, 6272, 64, 32, 640, "zipf", drop_some),    # 512 routes, columns that are no multiple of the XCDs
    (13, 6144, 12, 8, 4224, "zipf", None),        # runs of experts, each in chunks of the reduction
    (16, 8192, 4, 4, 2048, "uniform", None),       # sixteen rows of every expert
    (16, 7168, 8, 2, 2048, "uniform", one_expert),
    (2, 8192, 160, 120, 128, "uniform", None),     # many experts of few rows
]


@pytest.mark.parametrize("M,K,E,top_k,I,routing,spoil", FEW_WIDE,
                         ids=lambda v: v.__name__ if callable(v) else None)
def test_few_wide_equals_forward(M, K, E, top_k, I, routing, spoil):
    w, inp, dev, d, w1p, w2p = few_case(M, K, E, top_k, I, routing, seed=M + I, spoil=spoil)
    ref, dropped = H.run_forward(w, dev, w1p, w2p)
    for fill in (0xFF, 0x3C):
        out, bad = run_few(d, dev, w1p, w2p, fill)
        assert same_bits(out, ref) and bad == dropped


def test_few_wide_against_oracle():
    w, inp, dev, d, w1p, w2p = few_case(16, 6144, 24, 12, 2048, "zipf", seed=5, spoil=drop_some)
    ref = O.forward(inp, E=w.E)
    out, bad = run_few(d, dev, w1p, w2p)
    H.assert_out_close(H.bf16_f32(out), ref["out_f32"])
    assert bad == ref["dropped"]


# ---------------------------------------------------------------------------------------------
# the MXFP4 layer and its stages


def ids_of(counts, M, top_k, seed):
    """Expert ids that give expert e counts[e] rows, in a random order; the rest dropped."""
    route, _ = groups(counts, M, top_k, seed)
    flat = torch.full((M * top_k,), -1, dtype=torch.int32, **CU)
    experts = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(torch.int32).cuda()
    flat[route[: sum(counts)].long()] = experts
    return flat.view(M, top_k)


def by_stages(d, x, ids, probs, w1, w2):
    """The layer's stages one by one; y and the second product's rows beside the result."""
    M, K, E, top_k = d.M, d.K, d.E, d.top_k
    R = M * top_k
    qx, pts1 = torch.empty((M, K), dtype=torch.int8, **CU), torch.empty(R, **CU)
    eri, srt = torch.empty(R, dtype=torch.int32, **CU), torch.empty(R, dtype=torch.int32, **CU)
    cnt, cum = torch.empty(E, dtype=torch.int32, **CU), torch.empty(E, dtype=torch.int32, **CU)
    ws = torch.empty(MM.megamoe_permute_workspace_bytes(d), dtype=torch.uint8, **CU)
    MM.megamoe_permute_tokens(d, x, ids, qx, pts1, eri, srt, cnt, cum, ws)
    y = run_gmm(True, d, *run_quant(x), srt, cum, *w1)
    g2 = run_gmm(False, d, *run_quant(y, int(cum[-1])), srt, cum, *w2)
    out = torch.empty((M, K), dtype=torch.bfloat16, **CU)
    MM.megamoe_unpermute(d, g2, torch.ones(R, **CU), eri, probs, out)
    return out, cnt


def check_layer(counts, M, K, top_k, I, seed):
    d, x, _, w1, w2 = mx_layer(M, K, len(counts), top_k, I, seed)
    ids = ids_of(counts, M, top_k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    probs = torch.softmax(torch.randn((M, top_k), generator=g, **CU), 1)
    out, dropped = mx_forward(d, x, ids, probs, w1, w2)
    want, cnt = by_stages(d, x, ids, probs, w1, w2)
    assert cnt.tolist() == counts and dropped == M * top_k - sum(counts)
    assert torch.isfinite(want.float()).all() and (want != 0).any()
    assert same_bits(out, want)
    assert same_bits(mx_forward(d, x, ids, probs, w1, w2, 0xFF)[0], out)


# Wide tiles: up to four tiles of every height to a workgroup; three to seven stages of K, the last one
# whole or half, so that the next tile's copies start in this one's last stages (from four on) or after it.
@pytest.mark.parametrize("K", [256, 640, 768, 896, 1024, 1152, 1536, 1664])
def test_mxfp4_layer_wide_tiles(K):
    check_layer([300, 0, 520, 70, 40, 513, 900, 257], 1305, K, 2, 8192, seed=K)


# Several tiles of both products to a workgroup, and experts of more rows than a tile has.
@pytest.mark.parametrize("K,I", [(4096, 1152), (7168, 2048)])
def test_mxfp4_layer_prompt(K, I):
    check_layer([260, 31, 700, 0, 129, 512, 64, 65, 1, 190, 400, 257], 900, K, 3, I, seed=I)


# Narrow tiles (few rows to an expert on average): of up to 32 rows, of up to 64, several to an expert.
@pytest.mark.parametrize("K", [128, 256, 384, 640, 1152, 2048])
@pytest.mark.parametrize("I", [128, 384, 2048])
def test_mxfp4_layer_narrow_tiles(K, I):
    check_layer([50, 100, 33, 64, 1, 0, 2, 130, 32, 0, 0, 0, 0, 0, 7, 0, 0, 16], 250, K, 2, I, seed=K + I)


# The first product narrow, the second too or wide, on either side of the rules' borders: 28 and 48 mean rows.
@pytest.mark.parametrize("mean", [27, 28, 29, 47, 48, 49])
def test_mxfp4_layer_at_the_borders(mean):
    counts = [2 * mean, 0, mean + 20, mean - 20]
    check_layer(counts, 2 * mean, 896, 2, 640, seed=mean)


# ---------------------------------------------------------------------------------------------
# the MXFP4 layer in 64 bits

GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def mx_round64(v, e):
    """v [.., 32] to MXFP4 values under the scale 2^e [.., 1]: nearest, ties to the even code, 6 at most."""
    grid = GRID.to(v.device)
    s = torch.exp2(e.double())
    m = (v.abs() / s).clamp_max(6.0)
    hi = torch.searchsorted(grid, m.contiguous()).clamp_max(7)
    lo = (hi - 1).clamp_min(0)
    up, down = grid[hi] - m, m - grid[lo]
    code = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.sign(v) * grid[code] * s


def mx_exponent(most):
    return (torch.frexp(most).exponent - 3).clamp_min(-127)


def mx_between(lo, hi):
    """The least and the largest MXFP4 value of anything between lo and hi (rows of bf16 values), and
    the value of nothing but lo = hi.  Rounding is monotone under a scale; the scale may be either of
    those of the block's least and largest maximum (they are at most a step apart where lo and hi are)."""
    lo, hi = lo.unflatten(-1, (-1, 32)), hi.unflatten(-1, (-1, 32))
    most_hi = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True)
    inside = torch.where((lo <= 0) & (hi >= 0), 0.0, torch.minimum(lo.abs(), hi.abs()))
    most_lo = inside.amax(-1, keepdim=True)
    a, b = mx_exponent(most_lo), mx_exponent(most_hi)
    least = torch.minimum(mx_round64(lo, a), mx_round64(lo, b))
    largest = torch.maximum(mx_round64(hi, a), mx_round64(hi, b))
    assert (b - a <= 1).all()
    return least.flatten(-2), largest.flatten(-2)


def layer64(x, ids, probs, w1, w2, I):
    """The layer from its definition in 64 bits, and how far the kernels may be from it.  The roundings
    that belong to the definition are made: x and y to MXFP4, y to bf16 before that, the second
    product's rows to fp16 and bf16."""
    M, K = x.shape
    b = x.double().unflatten(-1, (-1, 32))
    xv = mx_round64(b, mx_exponent(b.abs().amax(-1, keepdim=True))).flatten(-2)
    out, tol = torch.zeros((M, K), dtype=torch.float64, **CU), torch.zeros((M, K), dtype=torch.float64, **CU)
    for e in range(w1[0].shape[0]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if len(tok) == 0:
            continue
        a, w = xv[tok], mx_values64(w1[0][e], w1[1][e]).t().contiguous()
        p, ab = a @ w, a.abs() @ w.abs()
        # an fp32 sum of K exact products: K roundings of 2^-24 of the terms' sizes, twice (a block's
        # terms may be added truncated)
        dp = K * 2 * U24 * ab
        u, gate, du, dg = p[:, :I], p[:, I:], dp[:, :I], dp[:, I:]
        sl = torch.sigmoid(u) * u
        y = sl * gate
        # |silu'| <= 1.1; silu itself (3 |u| + 8) roundings of 2^-24, the product one more
        dy = 1.1 * du * gate.abs() + sl.abs() * dg + 1.1 * du * dg + (3 * u.abs().clamp_max(104) + 9) * U24 * y.abs()
        mid = y.bfloat16().double()
        # rounding to bf16 through fp32, as .bfloat16() of a double does, keeps the order
        least, largest = mx_between((y - dy).bfloat16().double(), (y + dy).bfloat16().double())
        val, _ = mx_between(mid, mid)
        dq = torch.maximum(largest - val, val - least)
        assert (dq >= 0).all()
        w = mx_values64(w2[0][e], w2[1][e]).t().contiguous()
        g = val @ w
        # what y's codes may differ by, and the fp32 sum of the second product
        dg2 = dq @ w.abs() + I * 2 * U24 * ((val.abs() + dq) @ w.abs())
        row = g.half().double().bfloat16().double()
        # the kernel's row, from anywhere in g +- dg2: fp16 half a step (2^-11, 2^-25 below its normal
        # range) and bf16 half a step (2^-8) on either side
        drow = dg2 + 2 * (2.0 ** -11 + 2.0 ** -8) * (g.abs() + dg2) * 1.01 + 2.0 ** -24
        pr = probs[tok, slot].double().unsqueeze(1)
        for s in slot.unique().tolist():       # a token at most once in each addition
            at = slot == s
            out[tok[at]] += row[at] * pr[at]
            tol[tok[at]] += (drow[at] + ids.shape[1] * 2 * U24 * (row[at].abs() + drow[at])) * pr[at]
    return out, tol + 2.0 ** -8 * (out.abs() + tol)


@pytest.mark.parametrize("counts,M,K,top_k,I", [
    ([1, 0, 1, 0], 1, 256, 2, 128), ([3, 0, 9, 4, 2, 0], 9, 640, 2, 384), ([40, 3, 0, 64, 20], 64, 1152, 2, 256),
    ([300, 0, 70, 129], 250, 768, 2, 640), ([900, 257, 5, 0], 400, 512, 3, 256)])
def test_mxfp4_layer_against_64_bits(counts, M, K, top_k, I):
    d, x, _, w1, w2 = mx_layer(M, K, len(counts), top_k, I, seed=7 * M)
    ids = ids_of(counts, M, top_k, seed=M)
    g = torch.Generator(device="cuda").manual_seed(M)
    probs = torch.softmax(torch.randn((M, top_k), generator=g, **CU), 1)
    out, dropped = mx_forward(d, x, ids, probs, w1, w2)
    ref, tol = layer64(x, ids, probs, w1, w2, I)
    assert dropped == M * top_k - sum(counts)
    off = (out.double() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp_min(1e-300)).max())
    # the bound is a small part of the values, so that it can tell a wrong layer from a right one
    live = (ids >= 0).any(1)
    assert (tol[live].norm() <= 0.3 * ref[live].norm()) and (out[~live] == 0).all()
