"""Products of 16-bit experts, their gradients and SwiGLU on the GPU, against plain 64-bit forms (tests/half64.py)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests import half64 as P  # noqa: E402

pytestmark = pytest.mark.gpu
CU = dict(device="cuda")
T = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


def same_bits(a, b):
    v = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(v), b.contiguous().view(v))


def near(name, got, want, bound, t):
    got = got.double()
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), name
    off = (got - want).abs()
    tol = bound + P.half_step(want.abs() + bound, t)
    worst = (off / tol).max().item()
    assert worst <= 1, f"{name}: {worst:.3g} times its bound, off by {off.max().item():.3g}"


def ids_uniform(g, M, E, k):
    return torch.rand((M, E), generator=g).argsort(1)[:, :k].int()


def make_ids(M, E, k, how, seed=0):
    g = torch.Generator().manual_seed(seed)
    if how == "one":  # every route of one expert, the rest dropped
        ids = torch.full((M, k), -1, dtype=torch.int32)
        ids[:, 0] = E // 2
    elif how == "none":
        ids = torch.full((M, k), E, dtype=torch.int32)
    elif how == "zipf":
        w = (torch.arange(E) + 1.0) ** -1.2
        ids = torch.multinomial(w.expand(M, E), k, generator=g).int()
    elif how == "twice":  # a token names an expert in every slot
        ids = ids_uniform(g, M, E, 1).expand(M, k).contiguous()
    else:
        ids = ids_uniform(g, M, E, k)
        if how == "drop":
            ids[torch.rand(ids.shape, generator=g) < 0.3] = -1
    return ids.cuda()


def counted(counts, k=1):
    """ids [M, 1] with so many rows per expert."""
    ids = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(counts)])
    g = torch.Generator().manual_seed(1)
    return ids[torch.randperm(len(ids), generator=g)].view(-1, 1).cuda()


class Case:
    """Routes, rows and weights of one problem; buffers start as a pattern that results must not leave behind."""

    def __init__(self, M, K, E, k, I, ids, t, seed=0):
        self.d, self.t, self.ids = MM.dims(M, K, E, k, I), t, ids
        self.M, self.K, self.E, self.k, self.I, self.R = M, K, E, k, I, M * k
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        self.g = g
        R = self.R

        def rnd(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, **CU) * scale).to(t)
        self.x, self.w1 = rnd(M, K), rnd(E, 2 * I, K, scale=K ** -0.5)
        self.y, self.w2 = rnd(R, I), rnd(E, K, I, scale=I ** -0.5)
        self.dc, self.dout = rnd(R, 2 * I, scale=0.25), rnd(M, K, scale=0.25)
        self.probs = torch.softmax(torch.randn((M, k), generator=g, **CU), 1)
        self.row_of, self.route, self.end = P.sort(ids, E)
        self.n = int(self.end[-1])
        self.token = (self.route.long().clamp_min(0) // k)
        self.p = self.probs.flatten().double()[self.route.long().clamp_min(0)].unsqueeze(1)

    def out(self, cols):
        return torch.full((self.R, cols), -7.5, dtype=self.t, **CU)

    def rest(self, y):
        assert (y[self.n:] == -7.5).all(), "rows behind the last group were written"


SHAPES = [
    # M, K, E, top_k, I, routing
    (1, 128, 1, 1, 128, "uniform"), (1, 256, 4, 2, 128, "uniform"), (1, 7168, 32, 8, 256, "uniform"),
    (2, 384, 16, 4, 256, "drop"), (5, 1408, 64, 6, 384, "zipf"), (16, 128, 4, 4, 128, "twice"),
    (33, 640, 7, 7, 640, "uniform"), (64, 256, 3, 1, 896, "zipf"), (130, 512, 8, 2, 256, "drop"),
    (300, 384, 2, 2, 128, "uniform"), (700, 256, 40, 8, 384, "zipf"), (257, 128, 256, 3, 128, "uniform"),
    (40, 256, 5, 3, 128, "none"), (513, 256, 9, 2, 256, "one"), (1100, 1152, 4, 2, 640, "uniform"),
]
EDGES = [[31, 32, 33, 0, 1], [63, 64, 65], [0, 0, 127, 128, 129, 0], [191, 192, 193], [255, 256, 257], [511, 512, 513, 0]]


def cases(t):
    for M, K, E, k, I, how in SHAPES:
        yield pytest.param(lambda M=M, K=K, E=E, k=k, I=I, how=how: Case(M, K, E, k, I, make_ids(M, E, k, how, M), T[t]),
                           id=f"{t}-M{M}-K{K}-E{E}-k{k}-I{I}-{how}")
    for i, c in enumerate(EDGES):
        yield pytest.param(lambda c=c, i=i: Case(sum(c), 256 + 128 * i, len(c), 1, 128 + 128 * (i % 4), counted(c), T[t]),
                           id=f"{t}-rows-" + "-".join(map(str, c)))


ALL = [c for t in ("bf16", "fp16") for c in cases(t)]


@pytest.mark.parametrize("case", ALL)
def test_products(case):
    c = case()
    v1, b1 = P.product(c.x, c.token, c.w1, c.end, c.R)
    out = c.out(2 * c.I)
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, out)
    near("gmm1", out[:c.n], v1[:c.n], b1[:c.n], c.t)
    c.rest(out)
    for probs, p in ((c.probs, c.p), (None, torch.ones_like(c.p))):
        y, b = P.swiglu(v1, p, b1)
        out = c.out(c.I)
        H.megamoe_half_gmm1_swiglu(c.d, c.x, c.route, c.end, c.w1, out, probs=probs)
        near("gmm1_swiglu", out[:c.n], y[:c.n], b[:c.n], c.t)
        c.rest(out)
    v2, b2 = P.product(c.y, None, c.w2, c.end, c.R)
    out = c.out(c.K)
    H.megamoe_half_gmm2(c.d, c.y, c.end, c.w2, out)
    near("gmm2", out[:c.n], v2[:c.n], b2[:c.n], c.t)
    c.rest(out)


@pytest.mark.parametrize("case", ALL)
def test_row_gradients(case):
    c = case()
    v, b = P.product(c.dc, None, c.w1, c.end, c.R, transposed=True)
    out = c.out(c.K)
    H.megamoe_half_gmm1_dgrad(c.d, c.dc, c.end, c.w1, out)
    near("gmm1_dgrad", out[:c.n], v[:c.n], b[:c.n], c.t)
    c.rest(out)
    v, b = P.product(c.dout, c.token, c.w2, c.end, c.R, transposed=True)
    out = c.out(c.I)
    H.megamoe_half_gmm2_dgrad(c.d, c.dout, c.route, c.end, c.w2, out)
    near("gmm2_dgrad", out[:c.n], v[:c.n], b[:c.n], c.t)
    c.rest(out)


@pytest.mark.parametrize("case", ALL)
def test_weight_gradients(case):
    c = case()
    c.dc[c.n:] = math.nan  # what lies behind the last group is nobody's
    c.y[c.n:] = math.nan
    for first in (True, False):
        if first:
            want, bound = P.weights(c.dc, None, c.x, c.token, c.end, c.E)
            call = lambda dw, **k: H.megamoe_half_gmm1_wgrad(c.d, c.dc, c.x, c.route, c.end, dw, **k)
        else:
            want, bound = P.weights(c.dout, c.token, c.y, None, c.end, c.E)
            call = lambda dw, **k: H.megamoe_half_gmm2_wgrad(c.d, c.dout, c.y, c.route, c.end, dw, **k)
        for t in (c.t, torch.float32):
            dw = torch.full(want.shape, math.nan, dtype=t, **CU)
            call(dw)
            near("wgrad", dw, want, bound, t)
            old = torch.randn(want.shape, generator=c.g, **CU).to(t)
            dw = old.clone()
            call(dw, accumulate=True)
            # one more fp32 addition
            near("wgrad accumulated", dw, want + old.double(), bound + (want + old.double()).abs() * P.U * 2, t)
            empty = torch.ones(c.E, dtype=torch.bool)
            for e, _, _ in P.groups(c.end):
                empty[e] = False
            assert same_bits(dw[empty.cuda()], old[empty.cuda()])


@pytest.mark.parametrize("t", sorted(T))
def test_nothing_leaks_between_groups(t):
    """A row of infinities and NaN spoils its own outputs and its own expert's gradients alone."""
    c = Case(200, 256, 6, 2, 256, make_ids(200, 6, 2, "uniform", 3), T[t])
    bad = 2
    lo, hi = (0 if bad == 0 else int(c.end[bad - 1])), int(c.end[bad])
    clean = torch.ones(c.R, dtype=torch.bool, **CU)
    clean[lo:hi] = False
    others = torch.tensor([e for e in range(6) if e != bad], **CU)
    for v in (math.inf, -math.inf, math.nan):
        y, dc, w1, w2 = c.y.clone(), c.dc.clone(), c.w1.clone(), c.w2.clone()
        y[lo:hi], dc[lo:hi], w1[bad], w2[bad] = v, v, v, v
        outs = []
        for a, b, x, z in ((c.y, c.dc, c.w1, c.w2), (y, dc, w1, w2)):
            o = [c.out(2 * c.I), c.out(c.I), c.out(c.K), c.out(c.K), c.out(c.I)]
            H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, x, o[0])
            H.megamoe_half_gmm1_swiglu(c.d, c.x, c.route, c.end, x, o[1])
            H.megamoe_half_gmm2(c.d, a, c.end, z, o[2])
            H.megamoe_half_gmm1_dgrad(c.d, b, c.end, x, o[3])
            H.megamoe_half_gmm2_dgrad(c.d, c.dout, c.route, c.end, z, o[4])
            dw1, dw2 = torch.zeros_like(c.w1), torch.zeros_like(c.w2)
            H.megamoe_half_gmm1_wgrad(c.d, b, c.x, c.route, c.end, dw1)
            H.megamoe_half_gmm2_wgrad(c.d, c.dout, a, c.route, c.end, dw2)
            outs.append([q[clean] for q in o] + [dw1[others], dw2[others]])
        for p, q in zip(*outs):
            assert torch.isfinite(q).all() and same_bits(p, q)


@pytest.mark.parametrize("t", sorted(T))
def test_one_row_spoils_itself_alone(t):
    c = Case(90, 256, 2, 1, 128, counted([50, 40]), T[t])
    x = c.x.clone()
    token = int(c.token[7])
    x[token, 3] = math.nan
    a, b = c.out(2 * c.I), c.out(2 * c.I)
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, a)
    H.megamoe_half_gmm1(c.d, x, c.route, c.end, c.w1, b)
    assert b[7].isnan().all()
    keep = torch.arange(c.R, **CU) != 7
    assert same_bits(a[keep], b[keep])


@pytest.mark.parametrize("t", sorted(T))
def test_large_values(t):
    """Sums past fp16's range are infinite, in bf16 finite; fp16's subnormals count."""
    c = Case(40, 256, 3, 2, 128, make_ids(40, 3, 2, "uniform", 5), T[t])
    c.x.fill_(100.0)
    c.w1.fill_(100.0)
    out = c.out(2 * c.I)
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, out)
    assert (out == (math.inf if t == "fp16" else 2.56e6)).all()
    tiny = 2.0 ** -20 if t == "fp16" else 2.0 ** -100
    c.x.fill_(tiny)
    c.w1.fill_(1.0 / 256)
    H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, out)
    assert (out == tiny).all()


def test_extreme_preactivations():
    """silu of far negative and positive values, in the fused product and from memory, and its gradient."""
    for t in T.values():
        c = Case(4, 128, 1, 1, 128, counted([4]), t)
        big = 6e4 if t == torch.float16 else 1e30
        pre = torch.zeros((4, 256), dtype=t, **CU)
        pre[:, :128] = torch.linspace(-300, 300, 128, **CU)
        pre[0, :4] = torch.tensor([-big, big, -0.0, 0.0], **CU)
        pre[:, 128:] = 0.5
        dy = torch.ones((4, 128), dtype=t, **CU)
        y, dc, dp = c.out(128), c.out(256), torch.full((4, 1), -7.5, **CU)
        H.megamoe_half_swiglu(c.d, pre, c.route, c.end, y, probs=c.probs)
        H.megamoe_half_swiglu_grad(c.d, pre, dy, c.route, c.row_of, c.end, dc, probs=c.probs, dprobs=dp)
        assert torch.isfinite(y).all() and torch.isfinite(dc).all() and torch.isfinite(dp).all()
        assert y[0, 0] == 0 and (y[0, 1].item() == pre[0, 1].item() * 0.5) and dc[0, 0] == 0 and dc[0, 1] == 0.5


@pytest.mark.parametrize("t", sorted(T))
@pytest.mark.parametrize("M,E,k,I,how", [(1, 1, 1, 128, "uniform"), (1, 32, 8, 2048, "uniform"), (5, 64, 6, 1408, "zipf"),
                                         (37, 9, 3, 384, "drop"), (300, 16, 4, 640, "drop"), (3, 4, 2, 16384, "uniform"),
                                         (8, 4, 2, 128, "none"), (1200, 8, 8, 256, "uniform")])
def test_swiglu(t, M, E, k, I, how):
    c = Case(M, 128, E, k, I, make_ids(M, E, k, how, I), T[t])
    pre = (torch.randn((c.R, 2 * I), generator=c.g, **CU) * 2).to(c.t)
    pre[c.n:] = math.nan
    dy = (torch.randn((c.R, I), generator=c.g, **CU) * 0.3).to(c.t)
    for probs, p in ((c.probs, c.p), (None, torch.ones_like(c.p))):
        y = c.out(I)
        H.megamoe_half_swiglu(c.d, pre, c.route, c.end, y, probs=probs)
        want, bound = P.swiglu(pre[:c.n], p[:c.n])
        near("swiglu", y[:c.n], want, bound, c.t)
        c.rest(y)
        dc, dp = c.out(2 * I), torch.full((M, k), math.nan, **CU)
        H.megamoe_half_swiglu_grad(c.d, pre, dy, c.route, c.row_of, c.end, dc, probs=probs, dprobs=dp)
        want, bound, wp, bp = P.swiglu_grad(pre[:c.n], dy[:c.n], p[:c.n])
        near("dc", dc[:c.n], want, bound, c.t)
        c.rest(dc)
        full, fb = torch.zeros(c.R, dtype=torch.float64, **CU), torch.zeros(c.R, dtype=torch.float64, **CU)
        full[c.route[:c.n].long()], fb[c.route[:c.n].long()] = wp, bp
        near("dprobs", dp.flatten(), full, fb, torch.float32)
        again = c.out(2 * I)
        H.megamoe_half_swiglu_grad(c.d, pre, dy, c.route, c.row_of, c.end, again, probs=probs)
        assert same_bits(again, dc)


def test_swiglu_gradient_against_differences():
    """The gradient's formula against central differences of the forward's, in 64 bits, and the kernel against it."""
    g = torch.Generator().manual_seed(2)
    u, v, d = (torch.randn(64, generator=g, dtype=torch.float64) * 2 for _ in range(3))
    f = lambda u, v: torch.sigmoid(u) * u * v
    h = 1e-6
    c = torch.cat((u, v)).unsqueeze(0)
    want, _, dp, _ = P.swiglu_grad(c, d.unsqueeze(0), torch.tensor([[0.3]], dtype=torch.float64))
    num = torch.cat((f(u + h, v) - f(u - h, v), f(u, v + h) - f(u, v - h))) / (2 * h) * torch.cat((d, d)) * 0.3
    assert torch.allclose(want[0], num, atol=1e-8) and torch.allclose(dp, (d * f(u, v)).sum())


@pytest.mark.parametrize("t", sorted(T))
def test_same_bits_every_time(t):
    c = Case(600, 512, 12, 3, 384, make_ids(600, 12, 3, "zipf", 9), T[t])
    dw1, dw2 = torch.empty_like(c.w1), torch.empty_like(c.w2)
    first = None
    for _ in range(3):
        o = [c.out(2 * c.I), c.out(c.I), c.out(c.K), c.out(c.K), c.out(c.I)]
        H.megamoe_half_gmm1(c.d, c.x, c.route, c.end, c.w1, o[0])
        H.megamoe_half_gmm1_swiglu(c.d, c.x, c.route, c.end, c.w1, o[1], probs=c.probs)
        H.megamoe_half_gmm2(c.d, c.y, c.end, c.w2, o[2])
        H.megamoe_half_gmm1_dgrad(c.d, c.dc, c.end, c.w1, o[3])
        H.megamoe_half_gmm2_dgrad(c.d, c.dout, c.route, c.end, c.w2, o[4])
        H.megamoe_half_gmm1_wgrad(c.d, c.dc, c.x, c.route, c.end, dw1)
        H.megamoe_half_gmm2_wgrad(c.d, c.dout, c.y, c.route, c.end, dw2)
        o += [dw1.clone(), dw2.clone()]
        first = first or o
        assert all(same_bits(a, b) for a, b in zip(first, o))


def test_sort_routes_equals_permute():
    for M, E, k, how in ((1, 4, 2, "uniform"), (77, 9, 3, "drop"), (3000, 64, 6, "zipf"), (5, 3, 2, "none")):
        d = MM.dims(M, 128, E, k, 128)
        ids = make_ids(M, E, k, how, M)
        i32 = dict(dtype=torch.int32, **CU)
        o = [torch.full((M * k,), -9, **i32), torch.full((M * k,), -9, **i32), torch.full((E,), -9, **i32), torch.full((E,), -9, **i32)]
        ws = torch.empty(MM.megamoe_permute_workspace_bytes(d), dtype=torch.uint8, **CU)
        H.megamoe_sort_routes(d, ids, *o, ws)
        dropped = MM.megamoe_last_error(ws)
        row_of, route, end = P.sort(ids, E)
        assert torch.equal(o[0], row_of) and torch.equal(o[1], route) and torch.equal(o[3], end)
        assert torch.equal(torch.cumsum(o[2], 0).int(), end) and dropped == M * k - int(end[-1])
