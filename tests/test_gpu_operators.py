"""The router, the few-token layer, MXFP4 rows and the MXFP4 products on the GPU.

Each against a plain 64-bit implementation (tests/plain64.py, torch in float64), the few-token
layer also bit for bit against megamoe_forward, at the sizes and values where it can go wrong."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import inputs as W  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from oracle import oracle as O  # noqa: E402
from tests import gpu_helpers as H  # noqa: E402
from tests import plain64 as P64  # noqa: E402

pytestmark = pytest.mark.gpu
CU = dict(device="cuda")
U24 = 2.0 ** -24
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


def same_bits(a, b):
    v = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(v), b.contiguous().view(v))


# ---------------------------------------------------------------------------------------------
# router


def route_dims(M, E, top_k):
    return MM.dims(M, 128, E, top_k, 128)


def run_route(logits, top_k, bias=None, renormalize=True):
    M, E = logits.shape
    ids = torch.full((M, top_k), -7, dtype=torch.int32, **CU)
    probs = torch.full((M, top_k), -7.0, **CU)
    MM.megamoe_route(route_dims(M, E, top_k), logits, ids, probs, bias=bias, renormalize=renormalize)
    return ids, probs


def check_route(logits, top_k, bias=None, renormalize=True):
    ids, probs = run_route(logits, top_k, bias, renormalize)
    rid, rw = P64.route(logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(),
                        top_k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # one weight is exp(x - most) / total.  The exponent's argument carries three roundings (the
    # difference, the constant, the product), each |x - most| 2^-24; the exponential 2 ulp, the sum
    # of up to 256 terms at most 24 additions deep (16 in a lane, 4 across lanes, margin), the
    # quotient a half.  Twice that: numerator and total.
    lf = logits.float().cpu().numpy().astype(np.float64)
    fin = np.where(np.isfinite(lf), lf, 0)
    spread = min(float(fin.max() - fin.min()), 104.0)  # further down a weight is under 2^-149
    rtol = 2 * (3 * spread + 4 + 24 + 1) * U24
    got = probs.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - rw) <= rtol * rw + 2.0 ** -126), np.abs(got - rw).max()
    return ids, probs


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("M,E,top_k", [(1, 1, 1), (1, 32, 8), (3, 7, 7), (17, 33, 4), (5, 64, 64),
                                       (130, 65, 6), (33, 128, 9), (4, 129, 3), (257, 256, 8),
                                       (2, 256, 256), (31, 251, 1)])
def test_route_shapes(kind, M, E, top_k):
    g = torch.Generator(device="cuda").manual_seed(M * 1000 + E)
    logits = (torch.randn((M, E), generator=g, **CU) * 3).to(TYPES[kind])
    bias = torch.randn(E, generator=g, **CU) * 0.5
    for b in (None, bias):
        for renorm in (True, False):
            check_route(logits, top_k, b, renorm)


@pytest.mark.parametrize("E", [8, 100, 256])
def test_route_ties_and_zeros(E):
    """Equal scores go to the lowest index first; +0 and -0 are equal."""
    same = torch.zeros((3, E), **CU)
    same[1] = 1.5
    same[2, ::2] = -0.0
    ids, _ = check_route(same, 6)
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5]] * 3
    few = torch.randint(-2, 3, (64, E), generator=torch.Generator().manual_seed(E)).float().cuda()
    check_route(few.bfloat16(), min(E, 20))
    check_route(few, E, renormalize=False)


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_route_masks_and_extremes(kind):
    """Empty rows, -inf, NaN, the type's lowest value, +inf, and biases that switch experts off."""
    t, inf = TYPES[kind], float("inf")
    E, k = 40, 6
    x = torch.randn((9, E), generator=torch.Generator().manual_seed(1)).to(t)
    x[0] = -inf                                 # nothing takes part
    x[1] = float("nan")
    x[2] = -inf
    x[2, 17] = 0.5                              # one expert
    x[3] = torch.finfo(t).min                   # the lowest value is a value
    x[4, :30] = torch.finfo(t).min
    x[5, ::3] = float("nan")
    x[6, 5] = x[6, 33] = inf                    # an equal share each, the rest 0
    x[7, :35] = -inf                            # fewer than top_k
    x[8] = torch.finfo(t).max
    x = x.cuda()
    for renorm in (True, False):
        ids, probs = check_route(x, k, renormalize=renorm)
        assert ids[0].tolist() == [-1] * k and probs[0].abs().sum() == 0
        assert ids[1].tolist() == [-1] * k
        assert ids[2].tolist() == [17] + [-1] * (k - 1) and probs[2, 0] == 1
        assert ids[3].tolist() == list(range(k))
        assert ids[6, :2].tolist() == [5, 33] and probs[6, 0] == 0.5 and probs[6, 2] == 0
        assert ids[7, 5].item() == -1
    bias = torch.zeros(E, **CU)
    bias[::2] = -inf
    bias[1] = float("nan")
    bias[3] = inf
    ids, _ = check_route(x[5:6], k, bias, True)
    # odd experts only; expert 3's bias is +inf, but its logit is NaN here, so it takes no part
    assert (ids % 2 == 1)[ids >= 0].all() and 3 not in ids[0].tolist()
    assert check_route(x[8:9], k, bias, True)[0][0, 0] == 3


# ---------------------------------------------------------------------------------------------
# few tokens


def few_case(M, K, E, top_k, I, routing="uniform", seed=0, spoil=None):
    w = W.custom(M, K, E, top_k, I, routing=routing)
    inp = W.generate(w, seed)
    if spoil:
        spoil(inp)
    dev = H.to_dev(inp)
    d = MM.dims(M, K, E, top_k, I)
    w1p, w2p = H.prepack(d, dev)
    return w, inp, dev, d, w1p, w2p


def run_few(d, dev, w1p, w2p, fill=0xA5):
    ws = torch.full((MM.megamoe_few_workspace_bytes(d),), fill, dtype=torch.uint8, **CU)
    out = torch.full((d.M, d.K), float("nan"), dtype=torch.bfloat16, **CU)
    MM.megamoe_forward_few(d, dev["x"], dev["expert_idx"], dev["probs"], w1p, dev["scale1"], w2p,
                           dev["scale2"], out, ws)
    return out, MM.megamoe_last_error(ws)


def drop_some(inp):
    inp["expert_idx"][:, ::3] = -1
    inp["expert_idx"][0, -1] = 1 << 30


def drop_all(inp):
    inp["expert_idx"][:] = -5


def twice(inp):  # a token names an expert in several slots
    inp["expert_idx"][:] = inp["expert_idx"][:, :1]


def one_expert(inp):
    inp["expert_idx"][:] = -1
    inp["expert_idx"][:, 1] = 2


def zero_rows(inp):
    inp["x"][::2] = 0


def not_finite(inp):
    inp["x"][0, 5] = np.inf
    inp["x"][-1, 7] = np.nan
    inp["x"][1 % len(inp["x"]), 3] = -np.inf


FEW = [
    (1, 128, 1, 1, 128, "uniform", None), (1, 256, 4, 2, 128, "uniform", None),
    (2, 384, 16, 4, 256, "uniform", None), (3, 1024, 8, 8, 384, "uniform", drop_some),
    (5, 4096, 64, 6, 1408, "zipf", drop_some), (7, 640, 13, 3, 640, "zipf", None),
    (16, 896, 200, 8, 256, "zipf_empty", None), (16, 256, 256, 32, 128, "uniform", None),
    (4, 256, 8, 4, 128, "uniform", drop_all), (6, 512, 8, 5, 256, "uniform", twice),
    (16, 8192, 4, 3, 256, "uniform", one_expert),   # 16 rows of one expert: two passes over it
    (16, 32768, 3, 2, 128, "uniform", None),        # one quantised row fits at a time
    (16, 128, 4, 2, 16384, "uniform", None),        # the second reduction in chunks
    (16, 256, 5, 4, 4224, "uniform", drop_some),
    (3, 256, 6, 3, 256, "uniform", zero_rows), (4, 256, 6, 3, 256, "uniform", not_finite),
    (1, 7168, 32, 8, 2048, "uniform", None),
]


@pytest.mark.parametrize("M,K,E,top_k,I,routing,spoil", FEW,
                         ids=lambda v: v.__name__ if callable(v) else None)
def test_few_equals_forward(M, K, E, top_k, I, routing, spoil):
    w, inp, dev, d, w1p, w2p = few_case(M, K, E, top_k, I, routing, seed=K + M, spoil=spoil)
    ref, dropped = H.run_forward(w, dev, w1p, w2p)
    for fill in (0, 0xA5, 0xFF):
        out, bad = run_few(d, dev, w1p, w2p, fill)
        assert same_bits(out, ref), f"{w.describe()}, workspace of {fill:#x}"
        assert bad == dropped


@pytest.mark.parametrize("M,K,E,top_k,I,routing,spoil", FEW[1:6], ids=lambda v: v.__name__ if callable(v) else None)
def test_few_against_oracle(M, K, E, top_k, I, routing, spoil):
    w, inp, dev, d, w1p, w2p = few_case(M, K, E, top_k, I, routing, seed=11, spoil=spoil)
    ref = O.forward(inp, E=w.E)
    out, bad = run_few(d, dev, w1p, w2p)
    H.assert_out_close(H.bf16_f32(out), ref["out_f32"])
    assert bad == ref["dropped"]


# ---------------------------------------------------------------------------------------------
# MXFP4 rows


def mx_values64(q, s):
    """Packed codes and scale bytes (GPU tensors) -> float64 values on the GPU."""
    t = torch.tensor(list(P64.GRID) + [-v for v in P64.GRID], dtype=torch.float64, **CU)
    v = torch.stack((t[(q & 15).long()], t[(q >> 4).long()]), dim=-1).flatten(-2)
    sc = torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))
    return v * sc.repeat_interleave(32, dim=-1)


def run_quant(x, valid=None):
    rows, cols = x.shape
    q = torch.full((rows, cols // 2), 0x5A, dtype=torch.uint8, **CU)
    s = torch.full((rows, cols // 32), 0x5A, dtype=torch.uint8, **CU)
    v = None if valid is None else torch.tensor([valid], dtype=torch.int32, **CU)
    MM.megamoe_mxfp4_quant(x, q, s, valid_rows=v)
    return q, s


def mx_input(rows, cols, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, **CU) * torch.exp(2 * torch.randn((rows, 1), generator=g, **CU))
    x[:, ::17] = torch.round(x[:, ::17] * 4) / 4   # on and next to borders
    return x.to(t)


@pytest.mark.parametrize("kind", sorted(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (7, 160), (128, 128), (33, 4064), (1000, 64)])
def test_quant_shapes(kind, rows, cols):
    x = mx_input(rows, cols, TYPES[kind], rows + cols)
    q, s = run_quant(x)
    code, scale = P64.mx_quant(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), P64.pack(code))


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_quant_special_blocks(kind):
    t = TYPES[kind]
    f = torch.finfo(t)
    tiny = f.tiny * f.eps  # the smallest subnormal
    x = torch.zeros((16, 64), dtype=t)
    x[1] = -0.0
    x[2, :32] = tiny
    x[2, 32:] = -f.tiny
    x[3] = f.max
    x[4] = f.min
    x[5, 7] = float("nan")
    x[6, 40] = float("inf")
    x[7, 63] = -float("inf")
    x[8, :16] = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    x[9, :16] = x[8, :16] * 64
    x[10, :16] = torch.tensor([7.5, 6.5, 5.5, 5.01, 4.99, 2.51, 2.49, 0.26, 0.24, 0.1, -7.99, -7, 4, 3, 2, 1])
    x[11] = 1.0
    x[12, ::2] = f.max
    x[12, 1::2] = tiny
    x[13] = torch.linspace(-4, 4, 64).to(t)
    x[14] = f.tiny * 4
    x[15] = torch.linspace(-f.tiny * 6, f.tiny * 6, 64).to(t)
    x = x.cuda()
    q, s = run_quant(x)
    code, scale = P64.mx_quant(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), P64.pack(code))
    assert (s[5, 0], s[6, 1], s[7, 1]) == (255, 255, 255) and s[5, 1] != 255


@pytest.mark.parametrize("valid", [-3, 0, 1, 5, 8, 9, 1 << 30])
def test_rows_behind_are_left(valid):
    rows, cols = 8, 96
    x = mx_input(rows, cols, torch.bfloat16, 5)
    full_q, full_s = run_quant(x)
    n = max(0, min(rows, valid))
    q, s = run_quant(x, valid)
    assert torch.equal(q[:n], full_q[:n]) and torch.equal(s[:n], full_s[:n])
    assert (q[n:] == 0x5A).all() and (s[n:] == 0x5A).all()
    back = torch.full((rows, cols), -7.0, **CU)
    MM.megamoe_mxfp4_dequant(full_q, full_s, back, valid_rows=torch.tensor([valid], dtype=torch.int32, **CU))
    assert torch.equal(back[:n].double(), mx_values64(full_q, full_s)[:n])
    assert (back[n:] == -7).all()


@pytest.mark.parametrize("kind", sorted(TYPES))
def test_dequant_every_code_and_scale(kind):
    """All 16 codes under all 256 scale bytes, each rounded once to the output type."""
    q = torch.arange(256, dtype=torch.int32, **CU).view(1, 256).repeat(256, 1).to(torch.uint8)
    s = torch.arange(256, dtype=torch.int32, **CU).view(256, 1).repeat(1, 16).to(torch.uint8)
    out = torch.empty((256, 512), dtype=TYPES[kind], **CU)
    MM.megamoe_mxfp4_dequant(q, s, out)
    want = torch.from_numpy(P64.mx_values(q.cpu().numpy(), s.cpu().numpy())).to(TYPES[kind])
    assert torch.equal(torch.nan_to_num(out.cpu().double(), nan=-1.0), torch.nan_to_num(want.double(), nan=-1.0))


# ---------------------------------------------------------------------------------------------
# MXFP4 products


def mx_random(shape_rows, cols, std, seed):
    """Packed MXFP4 of normal values, quantised by the kernel that the tests above check."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = int(np.prod(shape_rows))
    q, s = run_quant(torch.randn((rows, cols), generator=g, **CU) * std)
    return q.view(*shape_rows, -1), s.view(*shape_rows, -1)


def groups(counts, M, top_k, seed):
    """sorted_route and expert_cumsum for given rows per expert; unused rows at the end hold -1."""
    R, n = M * top_k, sum(counts)
    assert n <= R
    r = torch.randperm(R, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    route = torch.full((R,), -1, dtype=torch.int32)
    route[:n] = r
    return route.cuda(), torch.cumsum(torch.tensor(counts), 0).to(torch.int32).cuda()


def gmm_reference(first, a, asc, route, cumsum, w, wsc, top_k):
    """Values in float64 and how far the kernel may be off, row by row."""
    av = mx_values64(a, asc)
    end = cumsum.tolist()
    rows_total = route.shape[0]
    N = w.shape[1] // (2 if first else 1)
    ref = torch.zeros((rows_total, N), dtype=torch.float64, **CU)
    tol = torch.zeros_like(ref)
    for e, (b, n) in enumerate(zip([0] + end[:-1], end)):
        if n == b:
            continue
        x = av[(route[b:n].long() // top_k)] if first else av[b:n]
        wt = mx_values64(w[e], wsc[e]).t().contiguous()
        p, ab = x @ wt, x.abs() @ wt.abs()
        # the products are exact; an fp32 sum of k terms is off by at most k 2^-24 sum|terms|, and
        # the matrix core may add a block's terms truncated rather than rounded: twice that
        dp = x.shape[1] * 2 * U24 * ab
        if first:
            u, gate = p[:, :N], p[:, N:]
            du, dg = dp[:, :N], dp[:, N:]
            sl = torch.sigmoid(u) * u
            y = sl * gate
            # |silu'| <= 1.1; silu itself: (3 |u| + 8) roundings of 2^-24; the product one more; bf16 a half step
            ref[b:n] = y
            tol[b:n] = (1.1 * du * gate.abs() + sl.abs() * dg + 1.1 * du * dg
                        + (3 * u.abs().clamp_max(104) + 9) * U24 * y.abs()) * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
        else:
            ref[b:n] = p
            tol[b:n] = dp * (1 + 2.0 ** -11) + 2.0 ** -11 * p.abs() + 2.0 ** -25
    return ref, tol


def run_gmm(first, d, a, asc, route, cumsum, w, wsc):
    R = d.M * d.top_k
    if first:
        y = torch.full((R, d.I), -7.0, dtype=torch.bfloat16, **CU)
        MM.megamoe_mxfp4_gmm1(d, a, asc, route, cumsum, w, wsc, y)
    else:
        y = torch.full((R, d.K), -7.0, dtype=torch.float16, **CU)
        MM.megamoe_mxfp4_gmm2(d, a, asc, cumsum, w, wsc, y)
    return y


def gmm_inputs(first, counts, M, K, top_k, I, seed=0):
    E, R = len(counts), M * top_k
    d = MM.dims(M, K, E, top_k, I)
    route, cumsum = groups(counts, M, top_k, seed)
    if first:
        a = mx_random((M,), K, 1.0, seed + 1)
        w = mx_random((E, 2 * I), K, 1.5 / K ** 0.5, seed + 2)
    else:
        a = mx_random((R,), I, 1.0, seed + 1)
        w = mx_random((E, K), I, 1.0 / I ** 0.5, seed + 2)
    return d, a, route, cumsum, w


GMM = [
    # rows per expert, M, K, top_k, I
    ([1], 1, 128, 1, 128), ([0, 2, 0, 0], 1, 256, 2, 128), ([0, 0, 0], 2, 128, 2, 128),
    ([3, 0, 1, 2], 3, 384, 2, 256), ([15, 16, 17, 0, 1], 25, 256, 2, 384), ([1] * 40, 40, 128, 1, 128),
    ([33, 31, 64, 65], 100, 640, 2, 128), ([127, 0, 129], 128, 256, 2, 128),
    ([255, 256, 257], 384, 384, 2, 256), ([600, 3, 0, 90], 400, 256, 2, 128),
    ([0, 1000, 0, 24], 512, 512, 2, 384), ([700, 800], 800, 1152, 2, 640), ([513], 600, 128, 1, 128),
    ([300] * 5 + [0] * 3, 800, 256, 2, 256), ([1, 2] * 64, 100, 256, 2, 128),
    ([16, 0] * 100, 900, 128, 2, 128), ([40, 56, 8, 0, 100], 110, 2048, 2, 1408),
]


@pytest.mark.parametrize("first", [True, False], ids=["gmm1", "gmm2"])
@pytest.mark.parametrize("case", range(len(GMM)))
def test_gmm(first, case):
    counts, M, K, top_k, I = GMM[case]
    d, (a, asc), route, cumsum, (w, wsc) = gmm_inputs(first, counts, M, K, top_k, I, seed=case)
    y = run_gmm(first, d, a, asc, route, cumsum, w, wsc)
    ref, tol = gmm_reference(first, a, asc, route, cumsum, w, wsc, top_k)
    n = sum(counts)
    off = (y[:n].double() - ref[:n]).abs()
    assert torch.isfinite(y[:n].float()).all()
    assert (off <= tol[:n]).all(), float((off / tol[:n].clamp_min(1e-300)).max())
    assert (y[n:] == -7).all(), "rows behind the last group were written"
    assert same_bits(y, run_gmm(first, d, a, asc, route, cumsum, w, wsc)), "two calls differ"


def check_gmm(first, counts, M, K, top_k, I, seed):
    d, (a, asc), route, cumsum, (w, wsc) = gmm_inputs(first, counts, M, K, top_k, I, seed=seed)
    y = run_gmm(first, d, a, asc, route, cumsum, w, wsc)
    ref, tol = gmm_reference(first, a, asc, route, cumsum, w, wsc, top_k)
    n = sum(counts)
    ref.sub_(y.double()).abs_()
    assert (ref[:n] <= tol[:n]).all()
    assert (y[n:] == -7).all()


# A persistent workgroup's second tile and those after it: of every number of stages from one to
# six, whole and half ones, and of different heights.
@pytest.mark.parametrize("first", [True, False], ids=["gmm1", "gmm2"])
@pytest.mark.parametrize("reduction", [128, 256, 384, 512, 640, 768, 1024, 1152, 1536])
def test_gmm_several_tiles_a_workgroup(first, reduction):
    K, I = (reduction, 8192) if first else (16384, reduction)
    check_gmm(first, [300, 0, 520, 70, 0, 513, 900, 257], 1300, K, 2, I, seed=reduction)


@pytest.mark.parametrize("K", [128, 768])
def test_gmm_long_tile_lists(K):
    """More tiles to a workgroup than it looks up at once."""
    check_gmm(True, [65] * 72, 2400, K, 2, 16384, seed=K)


@pytest.mark.parametrize("first", [True, False], ids=["gmm1", "gmm2"])
@pytest.mark.parametrize("counts,M", [([2, 0, 3], 4), ([40, 0, 30], 40), ([300, 0, 200], 300)])
def test_gmm_nan_stays_where_it_is(first, counts, M):
    """A NaN scale spoils its own row or column and nothing else; experts without rows and rows
    that no group holds are not read for their values."""
    K, I, top_k = 512, 256, 2
    d, (a, asc), route, cumsum, (w, wsc) = gmm_inputs(first, counts, M, K, top_k, I, seed=3)
    clean = run_gmm(first, d, a, asc, route, cumsum, w, wsc).float()
    n = sum(counts)
    wsc = wsc.clone()
    wsc[1] = 255                       # an expert without rows
    wsc[2, 5, 1] = 255                 # column 5 of expert 2
    asc = asc.clone()
    if first:
        used = torch.zeros(M, dtype=torch.bool, **CU)
        used[route[:n].long() // top_k] = True
        asc[~used] = 255
        tok = int(route[1]) // top_k
        asc[tok] = 255
        nan_rows = (route.long() // top_k == tok) & (torch.arange(M * top_k, **CU) < n)
    else:
        asc[n:] = 255
        asc[1, 0] = 255
        nan_rows = torch.arange(M * top_k, **CU) == 1
    y = run_gmm(first, d, a, asc, route, cumsum, w, wsc).float()
    want = clean.clone()
    b = int(cumsum[1])
    want[b:n, 5] = float("nan")
    want[nan_rows] = float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, nan=0.0), torch.nan_to_num(want, nan=0.0))


def test_gmm_large_values():
    """Scales at both ends of their range: sums pass fp16's and bf16's range to infinity, none turns NaN."""
    d, (a, asc), route, cumsum, (w, wsc) = gmm_inputs(False, [20, 50], 40, 256, 2, 128, seed=9)
    big = run_gmm(False, d, a, torch.full_like(asc, 190), route, cumsum, w, torch.full_like(wsc, 127)).float()
    assert not torch.isnan(big[:70]).any() and torch.isinf(big[:70]).any()
    small = run_gmm(False, d, a, torch.full_like(asc, 10), route, cumsum, w, torch.full_like(wsc, 20)).float()
    assert (small[:70] == 0).all()


# ---------------------------------------------------------------------------------------------
# together, in graphs, on streams


def mx_layer(M, K, E, top_k, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = MM.dims(M, K, E, top_k, I)
    x = torch.randn((M, K), generator=g, **CU).half()
    logits = torch.randn((M, E), generator=g, **CU)
    w1 = mx_random((E, 2 * I), K, 1.5 / K ** 0.5, seed + 1)
    w2 = mx_random((E, K), I, 1.0 / I ** 0.5, seed + 2)
    return d, x, logits, w1, w2


def mx_forward(d, x, ids, probs, w1, w2, fill=0xA5):
    ws = torch.full((MM.megamoe_mxfp4_workspace_bytes(d),), fill, dtype=torch.uint8, **CU)
    out = torch.full((d.M, d.K), float("nan"), dtype=torch.bfloat16, **CU)
    MM.megamoe_forward_mxfp4(d, x, ids, probs, *w1, *w2, out, ws)
    return out, MM.megamoe_last_error(ws)


@pytest.mark.parametrize("M,K,E,top_k,I", [(1, 256, 8, 2, 128), (5, 512, 16, 4, 256), (100, 384, 8, 3, 256),
                                           (700, 256, 4, 2, 384), (1300, 256, 6, 3, 128)])
def test_mxfp4_layer_from_router(M, K, E, top_k, I):
    """Router, then the MXFP4 layer: equal to its stages called one by one, and near the 64-bit
    layer on the same 4-bit weights and rows."""
    d, x, logits, w1, w2 = mx_layer(M, K, E, top_k, I, seed=M)
    logits[M // 2:, E // 2] = -float("inf")
    ids, probs = run_route(logits, top_k)
    out, dropped = mx_forward(d, x, ids, probs, w1, w2)
    assert dropped == int((ids < 0).sum())
    R = M * top_k
    qx = torch.empty((M, K), dtype=torch.int8, **CU)
    pts1 = torch.empty(R, **CU)
    eri, srt = torch.empty(R, dtype=torch.int32, **CU), torch.empty(R, dtype=torch.int32, **CU)
    cnt, cum = torch.empty(E, dtype=torch.int32, **CU), torch.empty(E, dtype=torch.int32, **CU)
    ws = torch.empty(MM.megamoe_permute_workspace_bytes(d), dtype=torch.uint8, **CU)
    MM.megamoe_permute_tokens(d, x, ids, qx, pts1, eri, srt, cnt, cum, ws)
    xq, xs = run_quant(x)
    y = run_gmm(True, d, xq, xs, srt, cum, *w1)
    n = int(cum[-1])
    yq, ys = run_quant(y, n)
    g2 = run_gmm(False, d, yq, ys, srt, cum, *w2)
    byhand = torch.empty((M, K), dtype=torch.bfloat16, **CU)
    MM.megamoe_unpermute(d, g2, torch.ones(R, **CU), eri, probs, byhand)
    assert same_bits(out, byhand)
    # the combine of the stages' rows in 64 bits: a bf16 rounding of each row (2^-8), one at the end
    # (2^-8), and top_k fp32 additions and products
    rows = torch.cat((g2[:n].double(), torch.zeros((1, K), dtype=torch.float64, **CU)))
    slot = torch.where(eri >= 0, eri.long(), n).view(M, top_k)
    p = torch.where(ids >= 0, probs, 0.0).double().unsqueeze(2)
    ref, mag = (rows[slot] * p).sum(1), (rows[slot].abs() * p).sum(1)
    assert ((out.double() - ref).abs() <= (2.0 ** -8 + (2 * top_k) * U24) * mag * 1.01 + 2.0 ** -8 * ref.abs()).all()


def test_router_into_few():
    """Router, then the int8 layer of a few tokens: equal to the staged forward on the same routes."""
    w, inp, dev, d, w1p, w2p = few_case(6, 512, 24, 4, 256, seed=2)
    logits = torch.randn((6, 24), generator=torch.Generator().manual_seed(3)).bfloat16()
    logits[2] = -float("inf")          # a padded token
    logits[:, 20:] = -float("inf")     # experts out of service
    dev["expert_idx"], dev["probs"] = run_route(logits.cuda(), 4)
    assert (dev["expert_idx"][2] == -1).all() and dev["expert_idx"].max() < 20
    ref, dropped = H.run_forward(w, dev, w1p, w2p)
    out, bad = run_few(d, dev, w1p, w2p)
    assert same_bits(out, ref) and bad == dropped == 4
    assert (out[2] == 0).all()


def test_graph_replays():
    """Router + few-token layer and router + MXFP4 layer captured in one graph, replayed with new
    contents and eager work in between, every replay equal to the eager result."""
    w, inp, dev, d, w1p, w2p = few_case(4, 512, 8, 3, 256, seed=5)
    dm, x, logits, w1, w2 = mx_layer(150, 256, 8, 2, 128, seed=6)
    few_logits = torch.randn((4, 8), generator=torch.Generator().manual_seed(1)).cuda()
    ids_f, pr_f = torch.zeros((4, 3), dtype=torch.int32, **CU), torch.zeros((4, 3), **CU)
    ids_m, pr_m = torch.zeros((150, 2), dtype=torch.int32, **CU), torch.zeros((150, 2), **CU)
    ws_f = torch.empty(MM.megamoe_few_workspace_bytes(d), dtype=torch.uint8, **CU)
    ws_m = torch.empty(MM.megamoe_mxfp4_workspace_bytes(dm), dtype=torch.uint8, **CU)
    out_f = torch.empty((4, 512), dtype=torch.bfloat16, **CU)
    out_m = torch.empty((150, 256), dtype=torch.bfloat16, **CU)

    def step():
        MM.megamoe_route(route_dims(4, 8, 3), few_logits, ids_f, pr_f)
        MM.megamoe_forward_few(d, dev["x"], ids_f, pr_f, w1p, dev["scale1"], w2p, dev["scale2"], out_f, ws_f)
        MM.megamoe_route(route_dims(150, 8, 2), logits, ids_m, pr_m, renormalize=False)
        MM.megamoe_forward_mxfp4(dm, x, ids_m, pr_m, *w1, *w2, out_m, ws_m)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for rep in range(4):
        g = torch.Generator(device="cuda").manual_seed(rep)
        few_logits.copy_(torch.randn((4, 8), generator=g, **CU))
        logits.copy_(torch.randn((150, 8), generator=g, **CU))
        dev["x"].copy_(torch.randn((4, 512), generator=g, **CU))
        step()
        torch.cuda.synchronize()
        want = out_f.clone(), out_m.clone()
        for t in (out_f, out_m):
            t.fill_(float("nan"))
        for t in (ws_f, ws_m):
            t.fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out_f, want[0]) and same_bits(out_m, want[1]), rep


def test_two_streams():
    """Calls with their own workspaces on two streams at once do not disturb each other."""
    cases = []
    for i in range(2):
        w, inp, dev, d, w1p, w2p = few_case(3 + i, 1024, 8, 3, 256, seed=20 + i)
        dm, x, logits, w1, w2 = mx_layer(200 + 100 * i, 256, 8, 2, 256, seed=30 + i)
        ids, probs = run_route(logits, 2)
        want = run_few(d, dev, w1p, w2p)[0], mx_forward(dm, x, ids, probs, w1, w2)[0]
        cases.append((dev, d, w1p, w2p, dm, x, ids, probs, w1, w2, want,
                      torch.empty(MM.megamoe_few_workspace_bytes(d), dtype=torch.uint8, **CU),
                      torch.empty(MM.megamoe_mxfp4_workspace_bytes(dm), dtype=torch.uint8, **CU),
                      torch.empty((d.M, d.K), dtype=torch.bfloat16, **CU),
                      torch.empty((dm.M, dm.K), dtype=torch.bfloat16, **CU), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for rep in range(5):
        for dev, d, w1p, w2p, dm, x, ids, probs, w1, w2, want, wf, wm, of, om, st in cases:
            MM.megamoe_forward_few(d, dev["x"], dev["expert_idx"], dev["probs"], w1p, dev["scale1"],
                                   w2p, dev["scale2"], of, wf, stream=st)
            MM.megamoe_forward_mxfp4(dm, x, ids, probs, *w1, *w2, om, wm, stream=st)
    torch.cuda.synchronize()
    for c in cases:
        assert same_bits(c[13], c[10][0]) and same_bits(c[14], c[10][1])


def test_holders():
    """The holder classes: router into the int8 layer, whole and of few tokens, and into the MXFP4 layer."""
    M, K, E, top_k, I = 5, 512, 8, 3, 256
    w, inp, dev, d, w1p, w2p = few_case(M, K, E, top_k, I, seed=11)
    logits = torch.randn((M, E), generator=torch.Generator().manual_seed(4)).half().cuda()
    logits[1] = float("nan")
    moe = MM.MegaMoE(M, K, E, top_k, I)
    moe.load_weights(dev["w1"], dev["scale1"], dev["w2"], dev["scale2"])
    ids, probs = moe.route(logits)
    whole = moe.forward(dev["x"], ids, probs)
    assert moe.last_error() == top_k
    few = moe.forward_few(dev["x"], ids, probs)
    assert moe.last_error() == top_k and same_bits(whole, few) and (whole[1] == 0).all()
    with pytest.raises(MM.MegaMoEError):
        MM.MegaMoE(17, K, E, top_k, I).forward_few(dev["x"], ids, probs)

    g = torch.Generator(device="cuda").manual_seed(12)
    w1 = (torch.randn((E, 2 * I, K), generator=g, **CU) / K ** 0.5).bfloat16()
    w2 = (torch.randn((E, K, I), generator=g, **CU) / I ** 0.5).bfloat16()
    mx = MM.MegaMoEMXFP4(M, K, E, top_k, I)
    mx.load_weights(w1, w2)
    ids, probs = mx.route(logits, bias=torch.ones(E, **CU), renormalize=False)
    out = mx.forward(dev["x"], ids, probs)
    assert mx.last_error() == top_k
    q1, s1 = run_quant(w1.view(-1, K))
    q2, s2 = run_quant(w2.view(-1, I))
    want, _ = mx_forward(mx.d, dev["x"], ids, probs, (q1.view(E, 2 * I, -1), s1.view(E, 2 * I, -1)),
                         (q2.view(E, K, -1), s2.view(E, K, -1)))
    assert same_bits(out, want) and (out[1] == 0).all()


def test_few_refuses_wrong_sizes():
    w, inp, dev, d, w1p, w2p = few_case(2, 256, 4, 2, 128, seed=1)
    out = torch.empty((2, 256), dtype=torch.bfloat16, **CU)
    ws = torch.empty(MM.megamoe_few_workspace_bytes(d), dtype=torch.uint8, **CU)
    good = dict(x=dev["x"], expert_idx=dev["expert_idx"], probs=dev["probs"], w1p=w1p, scale1=dev["scale1"],
                w2p=w2p, scale2=dev["scale2"], out=out, workspace=ws)
    for name, bad in (("w1p", w1p[:-16]), ("w2p", w2p[:-16]), ("scale1", dev["scale1"][:, :-4].contiguous()),
                      ("scale2", dev["scale2"][:-1]), ("x", dev["x"][:1]), ("out", out[:, :128].contiguous())):
        with pytest.raises(ValueError):
            MM.megamoe_forward_few(d, **{**good, name: bad})
    with pytest.raises(MM.MegaMoEError):
        MM.megamoe_forward_few(d, **{**good, "workspace": ws[:-256]})


# ---------------------------------------------------------------------------------------------
# offsets past 32 bits


def test_quant_past_32_bits():
    rows, cols = 600_000, 8192  # 4.9e9 elements, 9.8 GB
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, **CU)
    tail = torch.randn((77, cols), generator=torch.Generator(device="cuda").manual_seed(0), **CU).bfloat16()
    x[-77:] = tail
    q, s = run_quant(x)
    qt, st = run_quant(tail)
    assert torch.equal(q[-77:], qt) and torch.equal(s[-77:], st)
    back = torch.full_like(x, 7.0)
    MM.megamoe_mxfp4_dequant(q, s, back)
    assert same_bits(back[-77:], mx_values64(qt, st).bfloat16()) and bool((back[:-77].amax() == 0).item())


@pytest.mark.parametrize("rows", [3, 300])
def test_gmm_past_32_bits(rows):
    """Weights of 8.6 and 4.3 GB, used at their far end, with narrow and wide tiles."""
    M, K, E, top_k, I = rows * 256 // 64, 8192, 256, 64, 4096
    if rows == 3:
        M, top_k = 6, 1
    counts = [0] * E
    counts[1], counts[E - 3], counts[E - 1] = 1, rows // 2, rows
    for first in (True, False):
        N, red = (2 * I, K) if first else (K, I)
        d = MM.dims(M, K, E, top_k, I)
        route, cumsum = groups(counts, M, top_k, 5)
        a = mx_random((M,), K, 1.0, 1) if first else mx_random((M * top_k,), I, 1.0, 1)
        wq = torch.zeros((E, N, red // 2), dtype=torch.uint8, **CU)
        ws = torch.full((E, N, red // 32), 127, dtype=torch.uint8, **CU)
        for e in (1, E - 3, E - 1):
            wq[e], ws[e] = mx_random((N,), red, 1.0 / red ** 0.5, 7 + e)
        y = run_gmm(first, d, *a, route, cumsum, wq, ws)
        ref, tol = gmm_reference(first, *a, route, cumsum, wq, ws, top_k)
        n = sum(counts)
        assert ((y[:n].double() - ref[:n]).abs() <= tol[:n]).all()
        del wq, ws, ref, tol


def test_few_past_32_bits():
    M, K, E, top_k, I = 3, 8192, 256, 6, 4096
    moe = MM.MegaMoE(M, K, E, top_k, I)  # packed weights of 17 and 8.6 GB
    g = torch.Generator(device="cuda").manual_seed(3)
    moe.w1p.random_(-127, 128, generator=g)
    moe.w2p.random_(-127, 128, generator=g)
    moe.scale1 = torch.rand((E, 2 * I), generator=g, **CU) * 1e-3
    moe.scale2 = torch.rand((E, K), generator=g, **CU) * 1e-3
    logits = torch.randn((M, E), generator=g, **CU)
    logits[:, E - 2:] += 9
    ids, probs = moe.route(logits)
    x = torch.randn((M, K), generator=g, **CU).half()
    assert same_bits(moe.forward_few(x, ids, probs), moe.forward(x, ids, probs))


@pytest.mark.parametrize("M", [1, 3, 260])
def test_mxfp4_layer_edge_routes(M):
    """Every route dropped; one expert twice in a token; one expert alone; rows of a token behind it left out."""
    K, E, I = 256, 3, 128
    d, x, _, w1, w2 = mx_layer(M, K, E, 2, I, seed=40 + M)
    probs = torch.full((M, 2), 0.25, **CU)
    ids = torch.full((M, 2), -1, dtype=torch.int32, **CU)
    ids[:, 1] = E
    out, dropped = mx_forward(d, x, ids, probs, w1, w2)
    assert dropped == 2 * M and (out == 0).all()
    ids[:] = 2
    twice, dropped = mx_forward(d, x, ids, probs, w1, w2)
    assert dropped == 0
    d1 = MM.dims(M, K, 1, 1, I)
    one = torch.zeros((M, 1), dtype=torch.int32, **CU)
    alone, dropped = mx_forward(d1, x, one, torch.full((M, 1), 0.5, **CU), [t[2:].contiguous() for t in w1],
                                [t[2:].contiguous() for t in w2])
    # a quarter of a value and a quarter more are half of it, exactly
    assert dropped == 0 and same_bits(twice, alone) and torch.isfinite(alone.float()).all() and (alone != 0).any()
    ids[::2] = -1
    half, dropped = mx_forward(d, x, ids, probs, w1, w2)
    assert (half[::2] == 0).all() and same_bits(half[1::2], twice[1::2])


def test_valid_rows_from_a_view():
    """The row count read from the last element of a cumulative sum, at an address aligned to 4 bytes."""
    x = torch.randn((9, 64), generator=torch.Generator(device="cuda").manual_seed(0), **CU)
    cum = torch.tensor([1, 2, 5], dtype=torch.int32, **CU)
    q, s = torch.full((9, 32), 9, dtype=torch.uint8, **CU), torch.full((9, 2), 9, dtype=torch.uint8, **CU)
    MM.megamoe_mxfp4_quant(x, q, s, valid_rows=cum[-1:])
    qa, sa = run_quant(x)
    assert torch.equal(q[:5], qa[:5]) and torch.equal(s[:5], sa[:5]) and (q[5:] == 9).all() and (s[5:] == 9).all()


@pytest.mark.parametrize("M,I", [(5, 128), (60, 384), (130, 192 * 2), (900, 128)])
def test_mxfp4_layer_special_values(M, I):
    """Rows that are zero, tiny, huge, infinite or NaN: the layer, which quantises between its products in
    registers, equals its stages, which do so in memory."""
    K, E, top_k = 512, 4, 2
    d, x, logits, w1, w2 = mx_layer(M, K, E, top_k, I, seed=60 + M)
    x[0] = 0
    x[1] *= 2.0 ** -14
    x[2] *= 30000
    x[3, 7] = float("inf")
    x[4, 100] = float("nan")
    w1[1][:, ::5] -= 60      # silu columns, and gate columns, of quite different sizes
    w1[1][:, 1::7] += 50
    ids, probs = run_route(logits, top_k)
    out, _ = mx_forward(d, x, ids, probs, w1, w2)
    R = M * top_k
    qx, pts1 = torch.empty((M, K), dtype=torch.int8, **CU), torch.empty(R, **CU)
    eri, srt = torch.empty(R, dtype=torch.int32, **CU), torch.empty(R, dtype=torch.int32, **CU)
    cnt, cum = torch.empty(E, dtype=torch.int32, **CU), torch.empty(E, dtype=torch.int32, **CU)
    ws = torch.empty(MM.megamoe_permute_workspace_bytes(d), dtype=torch.uint8, **CU)
    MM.megamoe_permute_tokens(d, x, ids, qx, pts1, eri, srt, cnt, cum, ws)
    y = run_gmm(True, d, *run_quant(x), srt, cum, *w1)
    yq, ys = run_quant(y)
    assert (ys == 255).any() and (ys < 255).any() and (ys == 0).any()
    g2 = run_gmm(False, d, yq, ys, srt, cum, *w2)
    byhand = torch.empty((M, K), dtype=torch.bfloat16, **CU)
    MM.megamoe_unpermute(d, g2, torch.ones(R, **CU), eri, probs, byhand)
    assert torch.equal(torch.isnan(out), torch.isnan(byhand)) and torch.isnan(out[4]).all()
    assert same_bits(torch.nan_to_num(out), torch.nan_to_num(byhand))
