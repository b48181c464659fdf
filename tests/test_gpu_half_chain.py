"""16-bit experts as they are used together: the layer in one call, a training step of a block with its norms and its
router, graphs, streams, and offsets past 32 bits."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

from moe_expert_ffn_amd import half as H  # noqa: E402
from moe_expert_ffn_amd import megamoe as MM  # noqa: E402
from tests import half64 as P  # noqa: E402
from tests.test_gpu_half import Case, make_ids, near, same_bits  # noqa: E402

pytestmark = pytest.mark.gpu
CU = dict(device="cuda")
T = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    MM.load()


def holder(c):
    moe = H.MegaMoEHalf(c.M, c.K, c.E, c.k, c.I, dtype=c.t)
    moe.load_weights(c.w1, c.w2)
    return moe


@pytest.mark.parametrize("t", sorted(T))
@pytest.mark.parametrize("M,K,E,k,I,how", [(1, 256, 8, 2, 128, "uniform"), (5, 512, 64, 6, 384, "drop"), (1, 128, 4, 4, 256, "none"),
                                           (700, 384, 9, 3, 256, "zipf"), (1200, 256, 16, 8, 128, "drop"), (64, 2048, 4, 2, 512, "twice")])
def test_forward_equals_its_stages(t, M, K, E, k, I, how):
    c = Case(M, K, E, k, I, make_ids(M, E, k, how, M), T[t])
    moe = holder(c)
    moe.workspace.fill_(0xFF)
    out = moe.forward(c.x, c.ids, c.probs, out=torch.full((M, K), math.nan, dtype=c.t, **CU))
    assert moe.last_error() == c.R - c.n
    y, rows = c.out(I), c.out(K)
    H.megamoe_half_gmm1_swiglu(c.d, c.x, c.route, c.end, c.w1, y, probs=c.probs)
    H.megamoe_half_gmm2(c.d, y, c.end, c.w2, rows)
    want = torch.full((M, K), math.nan, dtype=c.t, **CU)
    H.megamoe_norm(c.d, rows=rows, expanded_row_idx=c.row_of, r=want)
    assert same_bits(out, want)
    # the rows through 64 bits from the y that the first product wrote; then at most 8 additions in fp32
    v, b = P.product(y, None, c.w2, c.end, c.R)
    near("rows", rows[:c.n], v[:c.n], b[:c.n], c.t)
    s, a = P.rows_sum(rows, c.row_of, M)
    near("out", out, s, a * 9 * P.U, c.t)


@pytest.mark.parametrize("t", sorted(T))
def test_forward_rows_and_combine(t):
    """The training forward rounds c to 16 bits on its way, which the serving one does not."""
    c = Case(300, 256, 8, 3, 256, make_ids(300, 8, 3, "drop", 4), T[t])
    moe = holder(c)
    p = moe.forward_rows(c.x, c.ids, c.probs)
    v, b = P.product(c.x, c.token, c.w1, c.end, c.R)
    near("c", p.c[:c.n], v[:c.n], b[:c.n], c.t)
    y, b = P.swiglu(p.c[:c.n], c.p[:c.n])
    near("y", p.y[:c.n], y, b, c.t)
    out = moe.combine(p)
    s, a = P.rows_sum(p.rows, c.row_of, c.M)
    near("out", out, s, a * 9 * P.U, c.t)


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("t", sorted(T))
@pytest.mark.parametrize("renormalize", [True, False])
def test_training_step_of_a_block(t, renormalize):
    """h = norm(x); routes and the layer of h; r = x + alpha gate norm(layer), h2 = norm(r): every gradient against
    autograd of the same in 64 bits, with the experts that the router chose."""
    M, K, E, k, I, eps, alpha = 150, 256, 10, 3, 384, 1e-5, 0.8
    c = Case(M, K, E, k, I, make_ids(M, E, k, "uniform"), T[t])
    g, d, moe = c.g, c.d, holder(c)
    rnd = lambda *s: torch.randn(s, generator=g, **CU)
    x, wr = rnd(M, K).to(c.t), rnd(K, E) * K ** -0.5
    wb1, wa, wb2 = (1 + 0.2 * rnd(K) for _ in range(3))
    gate = torch.sigmoid(rnd(M, 1))
    dr, dh2 = rnd(M, K).to(c.t), rnd(M, K).to(c.t)
    empty = lambda *s, t=c.t: torch.empty(s, dtype=t, **CU)

    h, logits = empty(M, K), None
    H.megamoe_norm(d, x=x, w_before=wb1, eps=eps, h=h)
    logits = h.float() @ wr
    ids, probs = moe.route(logits, renormalize=renormalize)
    p = moe.forward_rows(h, ids, probs)
    s, r, h2 = empty(M, K), empty(M, K), empty(M, K)
    H.megamoe_norm(d, x=x, rows=p.rows, expanded_row_idx=p.expanded_row_idx, w_after=wa, gate=gate, alpha=alpha, w_before=wb2,
                   eps=eps, s=s, r=r, h=h2)
    ws = torch.empty(H.megamoe_norm_grad_workspace_bytes(d), dtype=torch.uint8, **CU)
    f32 = torch.float32
    dx1, ds, dwa, dwb2, dgate = empty(M, K), empty(M, K), empty(K, t=f32), empty(K, t=f32), torch.empty_like(gate)
    H.megamoe_norm_grad(d, r, ws, dr=dr, dh=dh2, s=s, w_after=wa, gate=gate, alpha=alpha, w_before=wb2, eps=eps, dx=dx1, ds=ds,
                        dw_after=dwa, dw_before=dwb2, dgate=dgate)
    dx_rows, dprobs, dw1, dw2 = moe.backward(p, ds)
    dlogits = torch.empty_like(logits)
    H.megamoe_route_grad(d, logits, ids, probs, dprobs, dlogits, renormalize=renormalize)
    dh = (moe.combine(p, dx_rows).float() + dlogits @ wr.t()).to(c.t)
    dx, dwb1 = empty(M, K), empty(K, t=f32)
    H.megamoe_norm_grad(d, x, ws, dr=dx1, dh=dh, w_before=wb1, eps=eps, dx=dx, dw_before=dwb1)

    leaf = lambda v: v.double().requires_grad_()
    X, WR, WB1, WA, WB2, G, W1, W2 = map(leaf, (x, wr, wb1, wa, wb2, gate, c.w1, c.w2))
    hh = P.norm(X, None, None, None, 1, WB1, eps)[1]
    L = hh @ WR
    L.retain_grad()
    w = torch.softmax(L.gather(1, ids.long()), 1) if renormalize else torch.softmax(L, 1).gather(1, ids.long())
    out = torch.zeros((M, K), dtype=torch.float64, **CU)
    for e in range(E):
        for j in range(k):
            tok = torch.nonzero(ids[:, j] == e).flatten()
            pre = hh[tok] @ W1[e].t()
            y = w[tok, j:j + 1] * torch.sigmoid(pre[:, :I]) * pre[:, :I] * pre[:, I:]
            out = out.index_add(0, tok, y @ W2[e].t())
    R2, H2 = P.norm(X, out, WA, G, alpha, WB2, eps)
    torch.autograd.backward([R2, H2], [dr.double(), dh2.double()])
    # 16-bit tensors on the way forwards: h, c, y, rows, s, r (6); and back: dx1, ds, dy, dc, dx_rows, its sum, dh (7).  Each
    # is off by at most half a step, relatively; what a factor inherits from its inputs is at most doubled by a square or
    # a quotient of it (silu's slope, the norms).  Norms of the whole gradient, in which errors add up at most.
    tol = 2 * 13 * torch.finfo(c.t).eps / 2
    for name, got, want in (("r", r, R2.detach()), ("h2", h2, H2.detach()), ("dx", dx, X.grad), ("dw1", dw1, W1.grad),
                            ("dw2", dw2, W2.grad), ("dw_after", dwa, WA.grad), ("dw_before2", dwb2, WB2.grad),
                            ("dw_before1", dwb1, WB1.grad), ("dgate", dgate, G.grad), ("dlogits", dlogits, L.grad)):
        assert relative(got, want) <= tol, (name, relative(got, want), tol)


def test_accumulated_gradients():
    c = Case(60, 256, 6, 2, 128, make_ids(60, 6, 2, "zipf", 8), torch.bfloat16)
    moe = holder(c)
    p = moe.forward_rows(c.x, c.ids, c.probs)
    once = moe.backward(p, c.dout, torch.empty(c.w1.shape, **CU), torch.empty(c.w2.shape, **CU))
    sums = [torch.zeros(c.w1.shape, **CU), torch.zeros(c.w2.shape, **CU)]
    for _ in range(2):
        moe.backward(p, c.dout, *sums, accumulate=True)
    assert torch.equal(sums[0], 2 * once[2]) and torch.equal(sums[1], 2 * once[3])
    with pytest.raises(ValueError):
        moe.backward(p, c.dout, accumulate=True)


@pytest.mark.parametrize("M", [3, 200])
def test_graph(M):
    """The serving layer and a training pass captured, replayed on new inputs with eager work between the replays."""
    c = Case(M, 256, 8, 2, 128, make_ids(M, 8, 2, "drop", 2), torch.bfloat16)
    moe = holder(c)
    ids, x, probs, out = c.ids.clone(), c.x.clone(), c.probs.clone(), c.x.clone()
    dout, dw1, dw2 = c.dout.clone(), torch.empty_like(c.w1), torch.empty_like(c.w2)
    ws = torch.empty(H.megamoe_norm_grad_workspace_bytes(c.d), dtype=torch.uint8, **CU)
    w, dw, h, dx = torch.ones(c.K, **CU), torch.empty(c.K, **CU), torch.empty_like(x), torch.empty_like(x)
    logits, dlogits = torch.randn((M, 8), **CU), torch.empty((M, 8), **CU)

    def step():
        moe.forward(x, ids, probs, out=out)
        p = moe.forward_rows(x, ids, probs)
        g = moe.backward(p, dout, dw1, dw2)
        H.megamoe_norm(c.d, x=x, rows=p.rows, expanded_row_idx=p.expanded_row_idx, w_before=w, h=h)
        H.megamoe_norm_grad(c.d, x, ws, dr=dout, dh=g[0], expanded_row_idx=p.expanded_row_idx, w_before=w, dx=dx, dw_before=dw)
        H.megamoe_route_grad(c.d, logits, ids, probs, g[1], dlogits)
        return out, g[1], dw1, dw2, h, dx, dw, dlogits, moe.combine(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(4):
        n = Case(M, 256, 8, 2, 128, make_ids(M, 8, 2, "zipf" if seed % 2 else "drop", seed + 10), torch.bfloat16, seed=seed)
        for a, b in ((ids, n.ids), (x, n.x), (probs, n.probs), (dout, n.dout)):
            a.copy_(b)
        graph.replay()
        got = [v.clone() for v in held]
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, step())), seed


def test_two_streams():
    """Two layers at once, each on a stream and in a workspace of its own."""
    cs = [Case(300, 256, 8, 2, 256, make_ids(300, 8, 2, "zipf", s), torch.bfloat16, seed=s) for s in range(2)]
    moes = [holder(c) for c in cs]
    want = [m.forward(c.x, c.ids, c.probs) for m, c in zip(moes, cs)]
    back = [m.backward(m.forward_rows(c.x, c.ids, c.probs), c.dout) for m, c in zip(moes, cs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        got = []
        for m, c, s in zip(moes, cs, streams):
            with torch.cuda.stream(s):
                got.append((m.forward(c.x, c.ids, c.probs), m.backward(m.forward_rows(c.x, c.ids, c.probs), c.dout)))
        torch.cuda.synchronize()
        for (o, g), w, b in zip(got, want, back):
            assert same_bits(o, w) and same_bits(g[1], b[1]) and same_bits(g[2], b[2]) and same_bits(g[3], b[3])


def test_offsets_past_32_bits():
    """Weights and their gradients of more than 2^32 elements: the last expert's are found and written."""
    M, K, E, k, I = 40, 8192, 34, 2, 8192
    t = torch.bfloat16
    d = MM.dims(M, K, E, k, I)
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.full((M, k), E - 1, dtype=torch.int32)
    ids[::3, 0], ids[1::3, 1] = 0, 17
    row_of, route, end = P.sort(ids, E)
    token = route.long().clamp_min(0) // k
    used = [0, 17, E - 1]
    rnd = lambda *s: (torch.randn(s, generator=g, **CU) * 0.3).to(t)
    R = M * k
    x, dc, y, dout = rnd(M, K), rnd(R, 2 * I), rnd(R, I), rnd(M, K)
    w = torch.zeros((E, 2 * I, K), dtype=t, **CU)
    for e in used:
        w[e] = rnd(2 * I, K)
    out, dx = torch.empty((R, 2 * I), dtype=t, **CU), torch.empty((R, K), dtype=t, **CU)
    H.megamoe_half_gmm1(d, x, route, end, w, out)
    H.megamoe_half_gmm1_dgrad(d, dc, end, w, dx)
    v, b = P.product(x, token, w, end, R)
    near("gmm1", out, v, b, t)
    v, b = P.product(dc, None, w, end, R, transposed=True)
    near("gmm1_dgrad", dx, v, b, t)
    del v, b
    w.fill_(math.nan)
    H.megamoe_half_gmm1_wgrad(d, dc, x, route, end, w)
    for e, i, n in P.groups(end):
        one = torch.tensor([n - i], dtype=torch.int32, **CU)
        v, b = P.weights(dc[i:n], None, x[token[i:n]], None, one, 1)
        near("gmm1_wgrad", w[e], v[0], b[0], t)
        w[e] = 0
    assert not w.any()
