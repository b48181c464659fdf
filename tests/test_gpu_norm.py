"""The norms around the layer and the router, and their gradients, on the GPU against plain 64-bit forms."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests import half64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
CU = dict(device="cuda")
T = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


def near(name, got, want, bound, t):
    got = got.double()
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), name
    off = (got - want).abs()
    worst = (off / (bound + P.half_step(want.abs() + bound, t))).max().item()
    assert worst <= 1, f"{name}: {worst:.3g} times its bound, off by {off.max().item():.3g}"


def routes(M, k, seed=0, gone=0.2):
    """row_of [M k]: a permutation of the rows, some routes without one."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.randperm(M * k, generator=g).int()
    idx[torch.rand(M * k, generator=g) < gone] = -1
    return idx.cuda()


def gate_of(kind, M, K, g, t):
    shape = {None: None, "one": (1, 1), "token": (M, 1), "channel": (1, K), "element": (M, K)}[kind]
    return None if shape is None else torch.sigmoid(torch.randn(shape, generator=g, **CU)).to(t)


def depth(K):
    """Additions one after the other in a sum over K columns: in a thread (at most 32), across 64 lanes, across waves."""
    return 32 + 6 + 16


def forward_bounds(K, sv, sa, x, n, r, h, wa):
    """Errors of fp32 arithmetic.  The rows' sum is a few additions deep (their count, 256 at most, times u of the
    magnitudes).  A root mean square is off by depth(K) / 2 + 4 steps; n takes four products more."""
    bs = sa * 9 * P.U
    if n is None:
        br = torch.zeros_like(r)
    else:
        rel = (depth(K) + 12) * P.U
        grow = bs / sv.abs().clamp_min(1e-300)
        br = n.abs() * rel + (x.abs() if x is not None else 0) * P.U + r.abs() * P.U
        # an error of s moves n by as much relatively, and all of its row through the norm
        scale = n.abs() / sv.abs().clamp_min(1e-300)
        br = br + torch.minimum(grow * n.abs(), bs * scale)
        if wa is not None:
            br = br + n.abs() * (bs.norm(dim=1, keepdim=True) / sv.norm(dim=1, keepdim=True).clamp_min(1e-300))
    if h is None:
        return bs, br, None
    rel = (depth(K) + 12) * P.U
    per = h.abs() / r.abs().clamp_min(1e-300)
    bh = h.abs() * rel + br * per + h.abs() * (br.norm(dim=1, keepdim=True) / r.norm(dim=1, keepdim=True).clamp_min(1e-300))
    return bs, br, bh


FORWARD = [  # M, K, x, rows, top_k (0: dense), h, after, gate, before
    (1, 128, "fp32", "fp32", 0, "fp32", True, None, True), (1, 7168, "bf16", None, 0, "fp16", False, None, True),
    (3, 384, "fp16", "bf16", 3, "bf16", True, "token", True), (7, 4096, "fp32", "bf16", 8, "bf16", True, "channel", True),
    (2, 8192, "bf16", "bf16", 2, "fp32", False, "element", True), (2, 8320, "bf16", "fp16", 1, "bf16", True, "one", True),
    (2, 32768, "fp32", "fp32", 9, "fp16", True, "element", True), (5, 16512, "bf16", "bf16", 2, "bf16", True, "token", False),
    (129, 256, None, "bf16", 4, "bf16", False, None, False), (4, 512, None, "fp16", 17, "fp32", True, "one", True),
    (600, 128, "fp16", "fp32", 0, "fp16", True, "token", True), (9, 1408, "bf16", None, 0, "bf16", False, None, True),
    (33, 4224, "fp32", "fp16", 6, "fp32", False, "channel", False),
]


@pytest.mark.parametrize("M,K,x,rows,k,h,after,gate,before", FORWARD)
def test_norm(M, K, x, rows, k, h, after, gate, before):
    g = torch.Generator(device="cuda").manual_seed(K + M)
    d = MM.dims(M, K, 256, max(k, 1), 128)
    tx = T[x] if x else T[rows]
    X = torch.randn((M, K), generator=g, **CU).to(tx) if x else None
    idx = routes(M, k, M) if rows and k else None
    Y = (torch.randn((M * k if idx is not None else M, K), generator=g, **CU) * 3).to(T[rows]) if rows else None
    G = gate_of(gate, M, K, g, T[rows] if rows else None)
    wa = 1 + 0.2 * torch.randn(K, generator=g, **CU) if after else None
    wb = 1 + 0.2 * torch.randn(K, generator=g, **CU) if before else None
    full = lambda t: torch.full((M, K), math.nan, dtype=t, **CU)
    S, R, O = full(T[rows]) if rows else None, full(tx), full(T[h]) if before else None
    H.megamoe_norm(d, x=X, rows=Y, expanded_row_idx=idx, w_after=wa, gate=G, alpha=0.75, w_before=wb, eps=EPS, s=S, r=R, h=O)
    wide = lambda t: None if t is None else t.double()
    sv, sa = P.rows_sum(Y, idx, M) if rows else (None, torch.zeros((M, K), **CU))
    r, hh = P.norm(wide(X), sv, wide(wa), wide(G), 0.75, wide(wb), EPS)
    n = None if sv is None else (r if X is None else r - X.double())
    bs, br, bh = forward_bounds(K, sv, sa, wide(X), n, r, hh, wa)
    if rows:
        near("s", S, sv, bs, T[rows])
    near("r", R, r, br, tx)
    if before:
        near("h", O, hh, bh, T[h])
    # each output by itself is the same
    for key in ("s", "r", "h"):
        ref = dict(s=S, r=R, h=O)[key]
        if ref is None:
            continue
        one = torch.full_like(ref, math.nan)
        H.megamoe_norm(d, x=X, rows=Y, expanded_row_idx=idx, w_after=wa, gate=G, alpha=0.75, eps=EPS,
                        w_before=wb if key == "h" else None, **{key: one})
        assert torch.equal(one, ref), key


def test_norm_in_place_and_views():
    """r in x's own memory; rows of a larger tensor; a gate that is a row of one."""
    M, K = 6, 512
    g = torch.Generator(device="cuda").manual_seed(4)
    d = MM.dims(M, K, 4, 1, 128)
    X, Y = torch.randn((M + 2, K), generator=g, **CU).bfloat16(), torch.randn((M + 2, K), generator=g, **CU).bfloat16()
    G = torch.rand((5, K), generator=g, **CU)
    x, y = X[1:-1], Y[1:-1]
    want = torch.empty_like(x)
    H.megamoe_norm(d, x=x, rows=y, gate=G[2:3], r=want)
    before = X.clone()
    H.megamoe_norm(d, x=x, rows=y, gate=G[2:3], r=x)
    assert torch.equal(X[1:-1], want) and torch.equal(X[0], before[0]) and torch.equal(X[-1], before[-1])


def test_norm_rows_of_zeros_and_extremes():
    """A token without a row, a row of zeros, large and tiny values, infinities in rows that nobody names."""
    M, K, k = 4, 256, 2
    d = MM.dims(M, K, 4, k, 128)
    rows = torch.zeros((M * k, K), **CU)
    rows[0], rows[1], rows[2] = math.inf, 1e15, 1e-30
    idx = torch.tensor([-1, -1, 1, -1, 2, 3, 5, 1 << 30], dtype=torch.int32, **CU)
    w = torch.ones(K, **CU)
    s, r, h = (torch.full((M, K), math.nan, **CU) for _ in range(3))
    H.megamoe_norm(d, x=torch.zeros((M, K), **CU), rows=rows, expanded_row_idx=idx, w_after=w, w_before=w, s=s, r=r, h=h, eps=1e-6)
    assert (s[0] == 0).all() and (r[0] == 0).all() and (h[0] == 0).all()
    assert torch.allclose(r[1], torch.ones(K, **CU)) and (s[1] == 1e15).all()
    assert torch.allclose(r[2], torch.full((K,), 1e-27, **CU), rtol=1e-5) and (r[3] == 0).all()
    assert torch.isfinite(h).all()


GRAD = [  # M, K, x, rows, dh's type, top_k of dh (0: dense), after, gate, dr, before
    (1, 128, "fp32", "fp32", "fp32", 0, True, "one", True, True), (1, 7168, "bf16", "bf16", "bf16", 8, True, "channel", True, True),
    (3, 384, "fp16", "bf16", "bf16", 3, True, "token", True, True), (700, 256, "fp32", "bf16", "fp16", 2, True, "channel", True, True),
    (5, 4096, "bf16", "fp16", "bf16", 0, False, "element", True, True), (2, 8320, "bf16", "bf16", "fp32", 1, True, "one", False, True),
    (2, 32768, "fp32", "fp32", "fp16", 9, True, "element", True, True), (1030, 128, "bf16", "bf16", "bf16", 4, True, "one", True, True),
    (4, 16512, "bf16", "bf16", "bf16", 2, True, "token", True, True), (20, 640, "bf16", None, "bf16", 6, False, None, True, True),
    (33, 1408, "fp32", None, "fp32", 0, False, None, False, True), (9, 512, "bf16", "bf16", None, 0, True, "channel", True, False),
    (513, 384, "bf16", "bf16", None, 0, False, None, True, False), (40, 1024, "fp16", "fp16", "fp16", 2, False, "channel", True, True),
]


@pytest.mark.parametrize("M,K,x,rows,h,k,after,gate,with_dr,before", GRAD)
def test_norm_gradients(M, K, x, rows, h, k, after, gate, with_dr, before):
    """Against autograd of the plain form in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    rnd = lambda *s: torch.randn(s, generator=g, **CU)
    d = MM.dims(M, K, 256, max(k, 1), 128)
    tx = T[x]
    R = rnd(M, K).to(tx) if before else None
    S = (rnd(M, K) * 2).to(T[rows]) if rows else None
    DR = rnd(M, K).to(tx) if with_dr else None
    idx = routes(M, k, M) if k else None
    DH = rnd(M * k if k else M, K).to(T[h]) if before else None
    G = gate_of(gate, M, K, g, torch.float32 if gate != "element" else T[rows])
    wa = 1 + 0.2 * rnd(K) if after else None
    wb = 1 + 0.2 * rnd(K) if before else None
    nan = lambda t, *s: torch.full(s, math.nan, dtype=t, **CU)
    o = dict(dx=nan(tx, M, K), ds=nan(T[rows], M, K) if rows else None, dw_after=nan(torch.float32, K) if after else None,
             dw_before=nan(torch.float32, K) if before else None, dgate=None if G is None else nan(G.dtype, *G.shape))
    ws = torch.full((H.megamoe_norm_grad_workspace_bytes(d),), 0xFF, dtype=torch.uint8, **CU)
    call = lambda o: H.megamoe_norm_grad(d, R, ws, dr=DR, dh=DH, expanded_row_idx=idx, s=S, w_after=wa, gate=G, alpha=0.75,
                                          w_before=wb, eps=EPS, **o)
    call(o)

    leaf = lambda t: None if t is None else t.double().requires_grad_()
    s, a, b, q = leaf(S), leaf(wa), leaf(wb), leaf(G)
    with torch.no_grad():
        block = None if S is None else P.norm(None, S.double(), None if wa is None else wa.double(),
                                              None if G is None else G.double(), 0.75, None, EPS)[0]
        base = R.double() if before else torch.zeros((M, K), dtype=torch.float64, **CU) + (0 if block is None else block)
        xx = base if block is None else base - block
    xx.requires_grad_()
    r, hh = P.norm(xx, s, a, q, 0.75, b, EPS)
    outs, grads = [r], [DR.double() if with_dr else torch.zeros_like(r)]
    mag = grads[0].abs()
    if before:
        dh, dha = P.rows_sum(DH, idx, M)
        outs, grads = outs + [hh], grads + [dh]
    leaves = {"dx": xx, "ds": s, "dw_after": a, "dw_before": b, "dgate": q}
    want = dict(zip([n for n in leaves if leaves[n] is not None],
                    torch.autograd.grad(outs, [v for v in leaves.values() if v is not None], grads)))
    # bounds: every term of a formula is off by a few roundings of its own magnitude, and a mean by those of its row's
    rel = (depth(K) + 24) * P.U
    with torch.no_grad():
        if before:
            rs = 1 / torch.sqrt(R.double().square().mean(1, keepdim=True) + EPS)
            e = dha * wb.double().abs() * rs
            rh = R.double().abs() * rs
            mag = mag + e + rh * (e * rh).mean(1, keepdim=True)
        bound = {"dx": mag * rel}
        if before:
            # tokens in a row: at most M / 256 + 1 in a workgroup, and 1024 / 16 + 16 parts; M <= 2200 here
            bound["dw_before"] = (dha * rh).sum(0) * (rel + (M / 512 + 140) * P.U)
        if rows:
            ss = 1 / torch.sqrt(S.double().square().mean(1, keepdim=True) + EPS) if after else 1.0
            sh = S.double().abs() * ss
            wj = wa.double().abs() if after else 1.0
            gg = 0.75 * (G.double().abs() if G is not None else 1.0) * mag
            f = gg * wj * ss
            bound["ds"] = (f + sh * (f * sh).mean(1, keepdim=True) if after else f) * 3 * rel
            if after:
                bound["dw_after"] = (gg * sh).sum(0) * (3 * rel + (M / 512 + 140) * P.U)
            if G is not None:
                n = (0.75 * mag * sh * wj) * (3 * rel + (M / 512 + 140) * P.U)
                for i in range(2):
                    if G.shape[i] == 1:
                        n = n.sum(i, keepdim=True)
                bound["dgate"] = n
    for key, v in want.items():
        near(key, o[key], v, bound[key], o[key].dtype)
    again = {key: None if v is None else torch.full_like(v, math.nan) for key, v in o.items()}
    call(again)
    assert all(v is None or torch.equal(v, again[key]) for key, v in o.items())


def test_norm_gradient_formula_against_differences():
    """The plain form's gradient, which the kernels are held against, against central differences."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    M, K, step = 3, 8, 1e-6
    args = [rnd(M, K), rnd(M, K), rnd(K), torch.rand((M, 1), generator=g, dtype=torch.float64), rnd(K)]
    dr, dh = rnd(M, K), rnd(M, K)

    def f(v):
        r, h = P.norm(v[0], v[1], v[2], v[3], 0.75, v[4], EPS)
        return (r * dr).sum() + (h * dh).sum()
    leaves = [a.clone().requires_grad_() for a in args]
    grads = torch.autograd.grad(f(leaves), leaves)
    for i, a in enumerate(args):
        num = torch.zeros_like(a)
        for j in range(a.numel()):
            v = [b.clone() for b in args]
            v[i].view(-1)[j] += step
            up = f(v)
            v[i].view(-1)[j] -= 2 * step
            num.view(-1)[j] = (up - f(v)) / (2 * step)
        assert torch.allclose(grads[i], num, atol=1e-7)


# ---------------------------------------------------------------------------------------------
# the router's gradient


def route_grad64(x, bias, ids, dp, renormalize):
    """Autograd of the weights that the router gives these experts, in 64 bits."""
    M, E = x.shape
    out = torch.zeros((M, E), dtype=torch.float64)
    x, ids, dp = x.double().cpu(), ids.cpu(), dp.double().cpu()
    score = x if bias is None else x + bias.double().cpu()
    for t in range(M):
        chosen = [(s, e) for s, e in enumerate(ids[t].tolist()) if 0 <= e < E]
        part = sorted({e for _, e in chosen}) if renormalize else [e for e in range(E) if score[t, e] > -math.inf]
        if not chosen:
            continue
        leaf = x[t, part].clone().requires_grad_()
        w = torch.softmax(leaf, 0)
        loss = sum(w[part.index(e)] * dp[t, s] for s, e in chosen)
        out[t, part] = torch.autograd.grad(loss, leaf)[0]
    return out.cuda()


@pytest.mark.parametrize("kind", sorted(T))
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (1, 32, 8), (3, 7, 7), (17, 33, 4), (5, 64, 64), (130, 65, 6), (4, 129, 3),
                                   (70, 256, 8), (2, 256, 256), (31, 251, 1), (257, 8, 2)])
def test_route_gradient(kind, M, E, k):
    g = torch.Generator(device="cuda").manual_seed(M * 1000 + E)
    x = (torch.randn((M, E), generator=g, **CU) * 3).to(T[kind])
    if M > 2 and E > 2:
        x[1, ::2] = -math.inf
        x[2] = math.nan if E % 2 else -math.inf  # nothing takes part
    bias = torch.randn(E, generator=g, **CU) * 0.5
    if E > 8:
        bias[3] = -math.inf
    d = MM.dims(M, 128, E, k, 128)
    for b in (None, bias):
        for renorm in (True, False):
            ids, probs = torch.empty((M, k), dtype=torch.int32, **CU), torch.empty((M, k), **CU)
            MM.megamoe_route(d, x, ids, probs, bias=b, renormalize=renorm)
            dp = torch.randn((M, k), generator=g, **CU)
            out = torch.full((M, E), math.nan, **CU).to(T[kind])
            H.megamoe_route_grad(d, x, ids, probs, dp, out, bias=b, renormalize=renorm)
            want = route_grad64(x, b, ids, dp, renorm)
            # a weight is off by the exponent's argument (3 steps of the spread), the sum and the quotient, twice: probs' own
            # and the kernel's; dot by as much of its magnitude
            f = x.double()
            f = torch.where(torch.isfinite(f), f, 0)
            rel = 2 * (3 * min(float(f.max() - f.min()), 104.0) + 40) * P.U
            size = dp.abs().double().max() * 2
            near("dlogits", out, want, size * rel * 2, T[kind])
            assert (out[2] == 0).all() if M > 2 and E > 2 else True


def test_route_gradient_extremes():
    """+inf logits share, slots outside the experts are skipped, an expert named twice counts twice."""
    d = MM.dims(3, 128, 8, 3, 128)
    x = torch.zeros((3, 8), **CU)
    x[0, [2, 5]] = math.inf
    ids = torch.tensor([[2, 5, -1], [1, 8, 1 << 30], [4, 4, 6]], dtype=torch.int32, **CU)
    probs = torch.tensor([[.5, .5, 0], [1, 9, 9], [.25, .25, .5]], **CU)
    dp = torch.tensor([[1., 3, 7], [2, 5, 5], [1, 1, 2]], **CU)
    out = torch.full((3, 8), math.nan, **CU)
    H.megamoe_route_grad(d, x, ids, probs, dp, out)
    want = torch.zeros((3, 8), **CU)
    want[0, 2], want[0, 5] = 0.5 * (1 - 2), 0.5 * (3 - 2)
    want[2, 4], want[2, 6] = 0.5 * (1 - 1.5), 0.5 * (2 - 1.5)
    assert torch.equal(out, want)
