"""Calls of the 16-bit experts' products and their gradients, of SwiGLU with its gradient, of the norms around the
layer and of the router's gradient, as programs that serve or train a mixture-of-experts model make them.

Each case is one call, at sizes from a single decoded token to a training batch.  With `own` false the same
mathematics runs as elementary torch operations in fp32; with `own` true it runs through the framework's entry points.

The formulas (fp16 or bf16 in and out, sums in fp32; row d of the expert-major order belongs to expert e, to route
sorted_route[d] and to token sorted_route[d] // top_k; rows past the last group are left as they were):

gmm1          c[d, n] = sum_k x[token, k] w1[e, n, k]; with act: y[d, i] = p[route] silu(c[d, i]) c[d, I + i]
gmm2          z[d, k] = sum_i y[d, i] w2[e, k, i]
gmm1_dgrad    dx[d, k] = sum_n dc[d, n] w1[e, n, k]
gmm2_dgrad    dy[d, i] = sum_k dout[token, k] w2[e, k, i]
gmm1_wgrad    dw1[e, n, k] = sum_d dc[d, n] x[token, k]
gmm2_wgrad    dw2[e, k, i] = sum_d dout[token, k] y[d, i]
swiglu        y[d, i] = p[route] silu(c[d, i]) c[d, I + i]
swiglu_grad   dc of it, and dp[route] = sum_i dy[d, i] silu(c[d, i]) c[d, I + i], 0 for a route without a row
norm          s[t] = the rows of token t's routes, summed (or row t); n = s / rms(s) * w_after (or s);
              r = x + alpha gate n (or x); h = r / rms(r) * w_before; rms(v) = sqrt(mean v^2 + eps)
norm_grad     from dr and dh (dense, or rows of the routes to be summed): dx, ds, dw_after, dw_before, dgate
route_grad    dlogits of the router's weights: softmax over the chosen experts (renormalize) or over all that take part
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
GMM = ("gmm1", "gmm2", "gmm1_dgrad", "gmm2_dgrad", "gmm1_wgrad", "gmm2_wgrad")


def listed():
    return [
        # single-stream decoding with unquantised experts: eight experts' weights are streamed for a row each
        dict(name="gmm1 one token", op="gmm1", act=True, M=1, K=7168, E=32, top_k=8, I=2048, routing="uniform",
             dropped=0.0, type="bf16"),
        # second product of a decode batch: every expert has some 32 rows
        dict(name="gmm2 decode batch", op="gmm2", M=128, K=7168, E=32, top_k=8, I=2048, routing="uniform",
             dropped=0.0, type="bf16"),
        # first product of a training batch: matrix-core bound
        dict(name="gmm1 batch", op="gmm1", act=False, M=2048, K=7168, E=32, top_k=8, I=2048, routing="uniform",
             dropped=0.0, type="bf16"),
        # gradient of the second product's rows, skewed routing, experts without rows, dropped routes
        dict(name="gmm2 rows' gradient skewed", op="gmm2_dgrad", M=4096, K=4096, E=64, top_k=6, I=1408,
             routing="zipf_empty", dropped=0.02, type="fp16"),
        # gradient of the second product's weights, groups from a few rows to thousands
        dict(name="gmm2 weights' gradient skewed", op="gmm2_wgrad", M=4096, K=4096, E=64, top_k=6, I=1408,
             routing="zipf", dropped=0.0, type="bf16", out="bf16"),
        # a few streams' activations
        dict(name="swiglu five tokens", op="swiglu", M=5, E=64, top_k=6, I=1408, routing="zipf", dropped=0.03,
             type="fp16", weighted=True),
        # a training batch's activations, backwards
        dict(name="swiglu gradient batch", op="swiglu_grad", M=2048, E=32, top_k=8, I=2048, routing="uniform",
             dropped=0.01, type="bf16", weighted=True),
        # the norm before the layer for one decoded token
        dict(name="norm one token", op="norm", M=1, K=7168, x="bf16", rows=None, h="fp16", after=False, gate=None,
             before=True, E=32, top_k=8, dropped=0.0),
        # a prompt's layer output, eight rows a token: combine, norm, gate, residual and the next block's norm
        dict(name="norm after and before prompt", op="norm", M=2048, K=7168, x="fp32", rows="bf16", routed=True,
             h="bf16", after=True, gate="token", before=True, E=32, top_k=8, dropped=0.01),
        # the same backwards, a learned scale per channel, rows of the first product's gradient to be summed
        dict(name="norm gradient batch", op="norm_grad", M=4096, K=4096, x="bf16", rows="bf16", routed=True, h="bf16",
             after=True, gate="channel", before=True, E=64, top_k=6, dropped=0.02),
        # the router of a small training batch
        dict(name="route gradient small", op="route_grad", M=128, E=32, top_k=8, type="fp32", renormalize=True,
             masked=0.0),
        # a long batch over many experts, some switched off, padded tokens at its end
        dict(name="route gradient long", op="route_grad", M=32768, E=256, top_k=8, type="bf16", renormalize=False,
             masked=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(GMM + ("gmm1", "swiglu", "swiglu_grad", "norm", "norm_grad", "route_grad"))
    E = _log_int(rng, 4, 128)
    top_k = rng.randint(1, min(E, 8))
    if op == "route_grad":
        E = _log_int(rng, 4, 256)
        return dict(op=op, M=_log_int(rng, 1, 32768), E=E, top_k=rng.randint(1, min(E, 10)), type=rng.choice(sorted(TYPES)),
                    renormalize=rng.random() < 0.5, masked=rng.choice([0.0, 0.05, 0.3]))
    if op in ("norm", "norm_grad"):
        K, M = 128 * _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
        block = rng.random() < 0.75  # else the norm before alone
        kinds = sorted(TYPES)
        routed = rng.random() < 0.5
        while M * K * (top_k if routed else 1) > 4096 * 6 * 4096:
            M //= 2
        return dict(op=op, M=M, K=K, x=rng.choice(kinds), rows=rng.choice(kinds) if block else None, routed=routed,
                    h=rng.choice(kinds), after=block and rng.random() < 0.7,
                    gate=rng.choice([None, "one", "token", "channel", "element"]) if block else None,
                    before=not block or op == "norm_grad" or rng.random() < 0.7, E=E, top_k=top_k,
                    dropped=rng.choice([0.0, 0.02, 0.2]))
    K, I = 128 * _log_int(rng, 2, 64), 128 * _log_int(rng, 1, 20)
    most = 64 * 4096 * 1408 if op.endswith("wgrad") else 32 * 7168 * 2048
    while E * K * I * (2 if op == "gmm1_wgrad" else 1) > most:
        K, I = max(256, K // 256 * 128), max(128, I // 256 * 128)
        if K == 256 and I == 128:
            break
    M = _log_int(rng, 1, 4096)
    routing = rng.choice(["uniform", "zipf", "zipf_empty"])
    while routing != "uniform" and E * min(M, 2 * M * top_k) * K > 64 * 4096 * 4096:
        M //= 2
    while M * top_k * K * I > 16384 * 7168 * 2048:
        M //= 2
    if routing == "zipf_empty":
        top_k = max(1, min(top_k, 3 * E // 4))
    dropped = rng.choice([0.0, 0.02, 0.2]) if M * top_k >= 8 else 0.0
    c = dict(op=op, M=M, E=E, top_k=top_k, I=I, routing=routing, dropped=dropped, type=rng.choice(["fp16", "bf16"]))
    if op in GMM:
        c["K"] = K
    else:
        c["weighted"] = rng.random() < 0.7
    if op == "gmm1":
        c["act"] = rng.random() < 0.5
    if op.endswith("wgrad"):
        c["out"] = rng.choice([c["type"], "fp32"])
    return c


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _popularity(c):
    """How often each expert is picked first: equal, or falling as rank^-1.2, the last quarter never."""
    p = torch.ones(c["E"], dtype=torch.float64)
    routing = c.get("routing", "uniform")
    if routing != "uniform":
        p = (torch.arange(c["E"], dtype=torch.float64) + 1) ** -1.2
    if routing == "zipf_empty":
        p[3 * c["E"] // 4:] = 0
    return p / p.sum()


def _routes(c, g):
    """Expert ids [M, top_k], distinct within a token, -1 where the route was dropped, and softmax weights."""
    logp = torch.log(_popularity(c)).to(DEV)
    u = torch.rand((c["M"], c["E"]), generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-12)
    ids = torch.topk(logp - torch.log(-torch.log(u)), c["top_k"], dim=1).indices.to(torch.int32)
    gone = torch.rand(ids.shape, generator=g, device=DEV) < c["dropped"]
    return torch.where(gone, -1, ids), torch.softmax(_randn(g, c["M"], c["top_k"]), dim=1)


def _sort(s, ids, E):
    """The expert-major order of the routes, as the framework's sort writes it."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    s["expert_cumsum"] = torch.cumsum(counts, 0).to(torch.int32)
    valid = int(s["expert_cumsum"][-1])
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device=DEV)
    s["expanded_row_idx"] = torch.where(place < valid, place, -1).to(torch.int32)
    s["sorted_route"] = torch.where(torch.arange(len(order), device=DEV) < valid, order, -1).to(torch.int32)
    s["most"] = int(counts.max())


def _weights(g, E, rows, cols, t):
    w = torch.empty((E, rows, cols), dtype=t, device=DEV)
    for e in range(E):
        w[e] = _randn(g, rows, cols) / math.sqrt(cols)
    return w


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    op = c["op"]
    if op in ("norm", "norm_grad"):
        return _prepare_norm(c, g, s)
    if op == "route_grad":
        logits = _randn(g, c["M"], c["E"]) * 2
        if c["masked"]:
            off = torch.rand(c["E"], generator=g, device=DEV) < c["masked"]  # experts out of service
            logits = torch.where(off, -math.inf, logits)
            logits[int(c["M"] * 0.98):][1:] = -math.inf  # padded tokens
        s["logits"] = logits.to(TYPES[c["type"]])
        s["expert_idx"], s["probs"] = _route(s["logits"].float(), c["top_k"], c["renormalize"])
        s["dprobs"] = _randn(g, c["M"], c["top_k"])
        s["dlogits"] = torch.zeros((c["M"], c["E"]), dtype=TYPES[c["type"]], device=DEV)
        return s
    t, M, E, I, R = TYPES[c["type"]], c["M"], c["E"], c["I"], c["M"] * c["top_k"]
    ids, probs = _routes(c, g)
    _sort(s, ids, E)

    def zeros(*shape, dtype=t):
        return torch.zeros(shape, dtype=dtype, device=DEV)

    if op in ("swiglu", "swiglu_grad"):
        s["probs"] = probs if c["weighted"] else None
        s["c"] = (_randn(g, R, 2 * I) * 1.5).to(t)
        if op == "swiglu":
            s["y"] = zeros(R, I)
        else:
            s["dy"] = (_randn(g, R, I) * 0.1).to(t)
            s["dc"] = zeros(R, 2 * I)
            s["dprobs"] = zeros(M, c["top_k"], dtype=torch.float32) if c["weighted"] else None
        return s
    K = c["K"]
    rows_x = lambda: _randn(g, M, K).to(t)                       # normed hidden states
    rows_y = lambda: (torch.nn.functional.silu(_randn(g, R, I) * 1.5) * _randn(g, R, I)).to(t)  # activations
    grad = lambda n, cols: (_randn(g, n, cols) * 0.1).to(t)
    if op == "gmm1":
        s.update(a=rows_x(), w=_weights(g, E, 2 * I, K, t), y=zeros(R, I if c["act"] else 2 * I), probs=probs)
    elif op == "gmm2":
        s.update(a=rows_y(), w=_weights(g, E, K, I, t), y=zeros(R, K))
    elif op == "gmm1_dgrad":
        s.update(a=grad(R, 2 * I), w=_weights(g, E, 2 * I, K, t), y=zeros(R, K))
    elif op == "gmm2_dgrad":
        s.update(a=grad(M, K), w=_weights(g, E, K, I, t), y=zeros(R, I))
    elif op == "gmm1_wgrad":
        s.update(a=grad(R, 2 * I), b=rows_x(), dw=zeros(E, 2 * I, K, dtype=TYPES[c["out"]]))
    else:
        s.update(a=grad(M, K), b=rows_y(), dw=zeros(E, K, I, dtype=TYPES[c["out"]]))
    return s


def _prepare_norm(c, g, s):
    M, K = c["M"], c["K"]
    tx, th = TYPES[c["x"]], TYPES[c["h"]]
    tr = TYPES[c["rows"]] if c["rows"] else None
    s["alpha"] = 0.7
    routed = c.get("routed", False)
    if routed:
        _sort(s, _routes(c, g)[0], c["E"])
    idx = s.pop("expanded_row_idx", None)

    def wide(*shape):  # hidden states: rows of different size, some channels that stand out
        x = _randn(g, *shape) * torch.exp(0.5 * _randn(g, shape[0], 1))
        x[:, :: max(1, shape[1] // 5)] *= 8
        return x

    shape = {None: None, "one": (1, 1), "token": (M, 1), "channel": (1, K), "element": (M, K)}[c["gate"]]
    s["gate"] = torch.sigmoid(_randn(g, *shape)) if shape else None
    if c["gate"] == "element":
        s["gate"] = s["gate"].to(tr)
    s["w_after"] = 1 + 0.1 * _randn(g, K) if c["after"] else None
    s["w_before"] = 1 + 0.1 * _randn(g, K) if c["before"] else None
    empty = lambda t, *shape: torch.zeros(shape, dtype=t, device=DEV)
    if c["op"] == "norm":
        s["x"] = wide(M, K).to(tx)
        s["rows"] = None if tr is None else wide(M * c["top_k"] if routed else M, K).to(tr)
        s["idx"] = idx if tr is not None else None
        s["r"] = empty(tx, M, K) if tr is not None else None
        s["h"] = empty(th, M, K) if c["before"] else None
        s["s"] = empty(tr, M, K) if s["idx"] is not None else None
        return s
    s["r"] = wide(M, K).to(tx)
    s["s"] = wide(M, K).to(tr) if tr is not None else None
    s["dr"] = (_randn(g, M, K) * 0.1).to(tx)
    s["dh"] = (_randn(g, M * c["top_k"] if routed else M, K) * 0.1).to(th)
    s["idx"] = idx
    s["dx"] = empty(tx, M, K)
    s["ds"] = empty(tr, M, K) if tr is not None else None
    s["dw_after"] = empty(torch.float32, K) if c["after"] else None
    s["dw_before"] = empty(torch.float32, K)
    s["dgate"] = None if s["gate"] is None else empty(s["gate"].dtype, *shape)
    if own:  # the workspace that a training program keeps
        from moe_expert_ffn_amd import half as H
        s["workspace"] = torch.empty(H.megamoe_norm_grad_workspace_bytes(_dims(c)), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass


def _dims(c):
    from moe_expert_ffn_amd import megamoe as MM
    return MM.dims(c["M"], c.get("K", 128), c["E"], c["top_k"], c.get("I", 128))


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"swiglu": _swiglu, "swiglu_grad": _swiglu_grad, "norm": _norm, "norm_grad": _norm_grad,
                "route_grad": _route_grad}.get(op, _wgrad if op.endswith("wgrad") else _gmm)(s, c)
    from moe_expert_ffn_amd import half as H
    d = _dims(c)
    if op == "route_grad":
        H.megamoe_route_grad(d, s["logits"], s["expert_idx"], s["probs"], s["dprobs"], s["dlogits"],
                             renormalize=c["renormalize"])
        return s["dlogits"]
    if op == "norm":
        H.megamoe_norm(d, x=s["x"], rows=s["rows"], expanded_row_idx=s["idx"], w_after=s["w_after"], gate=s["gate"],
                       alpha=s["alpha"], w_before=s["w_before"], eps=EPS, s=s["s"], r=s["r"], h=s["h"])
        return [s[k] for k in ("s", "r", "h") if s[k] is not None]
    if op == "norm_grad":
        H.megamoe_norm_grad(d, s["r"], s["workspace"], dr=s["dr"], dh=s["dh"], expanded_row_idx=s["idx"], s=s["s"],
                            w_after=s["w_after"], gate=s["gate"], alpha=s["alpha"], w_before=s["w_before"], eps=EPS,
                            dx=s["dx"], ds=s["ds"], dw_after=s["dw_after"], dw_before=s["dw_before"],
                            dgate=s["dgate"])
        return [s[k] for k in ("dx", "ds", "dw_after", "dw_before", "dgate") if s[k] is not None]
    route, end = s["sorted_route"], s["expert_cumsum"]
    if op == "swiglu":
        H.megamoe_half_swiglu(d, s["c"], route, end, s["y"], probs=s["probs"])
        return s["y"]
    if op == "swiglu_grad":
        H.megamoe_half_swiglu_grad(d, s["c"], s["dy"], route, s["expanded_row_idx"], end, s["dc"], probs=s["probs"],
                                   dprobs=s["dprobs"])
        return [s["dc"]] + ([s["dprobs"]] if c["weighted"] else [])
    if op == "gmm1":
        if c["act"]:
            H.megamoe_half_gmm1_swiglu(d, s["a"], route, end, s["w"], s["y"], probs=s["probs"])
        else:
            H.megamoe_half_gmm1(d, s["a"], route, end, s["w"], s["y"])
    elif op == "gmm2":
        H.megamoe_half_gmm2(d, s["a"], end, s["w"], s["y"])
    elif op == "gmm1_dgrad":
        H.megamoe_half_gmm1_dgrad(d, s["a"], end, s["w"], s["y"])
    elif op == "gmm2_dgrad":
        H.megamoe_half_gmm2_dgrad(d, s["a"], route, end, s["w"], s["y"])
    elif op == "gmm1_wgrad":
        H.megamoe_half_gmm1_wgrad(d, s["a"], s["b"], route, end, s["dw"])
    else:
        H.megamoe_half_gmm2_wgrad(d, s["a"], s["b"], route, end, s["dw"])
    return s["dw"] if op.endswith("wgrad") else s["y"]


def _silu(u):
    return u / (1 + torch.exp(-u))


def _groups(s, R):
    """Rows of every expert's group, padded to the largest one: indices [E, most] and which of them are rows."""
    end = s["expert_cumsum"].long()
    begin = torch.cat((torch.zeros_like(end[:1]), end[:-1]))
    row = begin.unsqueeze(1) + torch.arange(s["most"], device=DEV)
    return begin, end, row.clamp_max(R - 1), row < end.unsqueeze(1)


def _gmm(s, c):
    """The grouped products: every group gathered into a batch entry; without many rows, a batch entry a row."""
    op, k, I = c["op"], c["top_k"], c["I"]
    R = c["M"] * k
    route = s["sorted_route"].clamp_min(0).long()
    gathered = op in ("gmm1", "gmm2_dgrad")
    r = torch.arange(R, device=DEV)
    end = s["expert_cumsum"].long()
    e = torch.searchsorted(end, r, right=True).clamp_max(c["E"] - 1)
    if R < c["E"]:
        a, w = s["a"][route // k if gathered else r].float().unsqueeze(1), s["w"][e].float()
        at = (r, 0)
    else:
        begin, _, row, _ = _groups(s, R)
        a, w = s["a"][(route[row] // k) if gathered else row].float(), s["w"].float()
        at = (e, (r - begin[e]).clamp(0, max(0, s["most"] - 1)))
    y = torch.matmul(a, w if op.endswith("dgrad") else w.transpose(1, 2))[at]
    if c.get("act"):
        y = s["probs"].reshape(-1)[route].unsqueeze(1) * (_silu(y[:, :I]) * y[:, I:])
    return torch.where((r < end[-1]).unsqueeze(1), y, 0.0).to(s["y"].dtype)


def _wgrad(s, c):
    R = c["M"] * c["top_k"]
    _, _, row, there = _groups(s, R)
    token = s["sorted_route"][row].clamp_min(0).long() // c["top_k"]
    first = c["op"] == "gmm1_wgrad"
    a = torch.where(there.unsqueeze(2), s["a"][row if first else token].float(), 0.0)
    b = torch.where(there.unsqueeze(2), s["b"][token if first else row].float(), 0.0)
    return torch.matmul(a.transpose(1, 2), b).to(s["dw"].dtype)


def _row_weights(s):
    route = s["sorted_route"].long()
    p = torch.ones(len(route), device=DEV) if s["probs"] is None else s["probs"].reshape(-1)[route.clamp_min(0)]
    return p.unsqueeze(1), (route >= 0).unsqueeze(1)


def _swiglu(s, c):
    p, there = _row_weights(s)
    u, g = s["c"].float().chunk(2, dim=1)
    return torch.where(there, p * (_silu(u) * g), 0.0).to(s["y"].dtype)


def _swiglu_grad(s, c):
    p, there = _row_weights(s)
    u, g = s["c"].float().chunk(2, dim=1)
    dy = s["dy"].float()
    sig = 1 / (1 + torch.exp(-u))
    q = p * dy
    dc = torch.cat((q * g * sig * (1 + u * (1 - sig)), q * (u * sig)), dim=1)
    dc = torch.where(there, dc, 0.0).to(s["dc"].dtype)
    if not c["weighted"]:
        return [dc]
    dp = (dy * (u * sig) * g).sum(1)
    row = s["expanded_row_idx"].long()
    return [dc, torch.where(row >= 0, dp[row.clamp_min(0)], 0.0).view(c["M"], c["top_k"])]


def _tokens(rows, idx, M):
    """Row t, or the sum of the rows of token t's routes."""
    if idx is None:
        return rows.float()
    idx = idx.view(M, -1).long()
    y = torch.zeros((M, rows.shape[1]), device=DEV)
    for j in range(idx.shape[1]):
        y = y + torch.where((idx[:, j] >= 0).unsqueeze(1), rows[idx[:, j].clamp_min(0)].float(), 0.0)
    return y


def _norm(s, c):
    res = []
    r = s["x"].float()
    if s["rows"] is not None:
        n = _tokens(s["rows"], s["idx"], c["M"])
        if s["s"] is not None:
            res.append(n.to(s["s"].dtype))
        if s["w_after"] is not None:
            n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + EPS) * s["w_after"]
        if s["gate"] is not None:
            n = n * s["gate"].float()
        r = r + s["alpha"] * n
        res.append(r.to(s["r"].dtype))
    if s["h"] is not None:
        res.append((r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w_before"]).to(s["h"].dtype))
    return res


def _norm_grad(s, c):
    r = s["r"].float()
    dh = _tokens(s["dh"], s["idx"], c["M"])
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    rh = r * rstd
    gb = dh * s["w_before"]
    dx = s["dr"].float() + rstd * (gb - rh * (gb * rh).mean(1, keepdim=True))
    dw_before = (dh * rh).sum(0)
    res = [dx.to(s["dx"].dtype)]
    dw_after = dgate = None
    if s["s"] is not None:
        v = s["s"].float()
        rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
        vh = v * rstd
        n = v if s["w_after"] is None else vh * s["w_after"]
        dn = s["alpha"] * dx
        if s["gate"] is not None:
            dgate = dn * n
            for i in range(2):
                if s["gate"].shape[i] == 1:
                    dgate = dgate.sum(i, keepdim=True)
            dgate = dgate.to(s["dgate"].dtype)
            dn = dn * s["gate"].float()
        if s["w_after"] is None:
            ds = dn
        else:
            dw_after = (dn * vh).sum(0)
            ga = dn * s["w_after"]
            ds = rstd * (ga - vh * (ga * vh).mean(1, keepdim=True))
        res.append(ds.to(s["ds"].dtype))
    return res + [v for v in (dw_after, dw_before, dgate) if v is not None]


def _route(x, top_k, renormalize):
    """Softmax top-k of fp32 logits: ids and weights."""
    out = torch.isnan(x) | (x == -math.inf)
    x = torch.where(out, -math.inf, x)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids, chosen = ids[:, :top_k], top[:, :top_k] > -math.inf
    over = torch.where(chosen, top[:, :top_k], -math.inf) if renormalize else x
    most = over.amax(1, keepdim=True)
    z = torch.where(over > -math.inf, torch.exp(over - torch.where(most > -math.inf, most, 0.0)), 0.0)
    w = z if renormalize else z.gather(1, ids)
    w = torch.where(chosen, w / z.sum(1, keepdim=True), 0.0)
    return torch.where(chosen, ids, -1).to(torch.int32), w


def _route_grad(s, c):
    ids, dp = s["expert_idx"].long(), s["dprobs"]
    there = ids >= 0
    p = torch.where(there, s["probs"], 0.0)
    dp = torch.where(there, dp, 0.0)
    dot = (p * dp).sum(1, keepdim=True)
    x = s["logits"].float()
    if c["renormalize"]:
        d = torch.zeros_like(x).scatter_add_(1, ids.clamp_min(0), torch.where(there, p * (dp - dot), 0.0))
    else:
        part = x > -math.inf
        most = x.amax(1, keepdim=True)
        z = torch.where(part, torch.exp(x - torch.where(most > -math.inf, most, 0.0)), 0.0)
        w = z / z.sum(1, keepdim=True).clamp_min(1e-30)
        d = torch.zeros_like(x).scatter_add_(1, ids.clamp_min(0), dp) - dot
        d = torch.where(part, w * d, 0.0)
    return d.to(s["dlogits"].dtype)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def _active(c):
    """Expected number of experts with a row."""
    uniform = c["routing"] == "uniform"
    once = torch.full((c["E"],), c["top_k"] / c["E"]) if uniform else 1 - (1 - _popularity(c)) ** c["top_k"]
    return float((1 - (1 - once.double() * (1 - c["dropped"])) ** c["M"]).sum())


def work(case):
    c, op = case, case["op"]
    M = c["M"]
    if op == "route_grad":
        n = M * c["E"] * SIZE[c["type"]]
        return {"bytes": n * (1 if c["renormalize"] else 2) + 12 * M * c["top_k"],
                "flops": (1 if c["renormalize"] else 6) * M * c["E"]}
    if op in ("norm", "norm_grad"):
        n = M * c["K"]
        x, h = SIZE[c["x"]], SIZE[c["h"]]
        b = SIZE[c["rows"]] if c["rows"] else 0
        live = c["top_k"] * (1 - c["dropped"]) if c.get("routed") else 1
        gate = {None: 0, "one": 1, "token": M, "channel": c["K"], "element": n}[c["gate"]]
        gate *= b if c["gate"] == "element" else 4
        if op == "norm":
            total = n * (x + b * live + (x if b else 0) + h * c["before"]) + gate
            total += n * b if c.get("routed") and b else 0
            return {"bytes": total, "flops": n * (10 + live)}
        return {"bytes": n * (3 * x + 2 * b + h * live) + 2 * gate, "flops": n * (20 + live)}
    I, size, R = c["I"], SIZE[c["type"]], M * c["top_k"] * (1 - c["dropped"])
    if op in ("swiglu", "swiglu_grad"):
        n = (3 if op == "swiglu" else 5) * R * I * size
        return {"bytes": n + (8 if op == "swiglu" else 16) * R, "flops": (5 if op == "swiglu" else 15) * R * I}
    K = c["K"]
    wide = 2 * I if op.startswith("gmm1") else I  # of the inner side
    inner = R * (I if c.get("act") else wide)
    outer = (min(M, R) if op in ("gmm1", "gmm1_wgrad", "gmm2_dgrad", "gmm2_wgrad") else R) * K
    weights = c["E"] * SIZE[c["out"]] if op.endswith("wgrad") else _active(c) * size
    return {"bytes": weights * wide * K + (inner + outer) * size, "flops": 2 * R * wide * K}


# ---------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, c)
    if op == "route_grad":
        return _exact_route_grad(s, c)
    k, I = c["top_k"], c["I"]
    route = s["sorted_route"].long()
    valid = int(s["expert_cumsum"][-1])
    if op in ("swiglu", "swiglu_grad"):
        p = torch.ones(c["M"] * k, dtype=torch.float64, device=DEV) if s["probs"] is None else s["probs"].double().flatten()
        u, v = s["c"][:valid, :I].double(), s["c"][:valid, I:].double()
        p = p[route[:valid]].unsqueeze(1)
        sig = torch.sigmoid(u)
        if op == "swiglu":
            y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
            y[:valid] = p * sig * u * v
            return y
        dy = s["dy"][:valid].double()
        dc = torch.zeros(s["dc"].shape, dtype=torch.float64, device=DEV)
        dc[:valid, :I] = p * dy * v * (sig + u * sig * (1 - sig))
        dc[:valid, I:] = p * dy * u * sig
        if not c["weighted"]:
            return [dc]
        dp = torch.zeros(c["M"] * k, dtype=torch.float64, device=DEV)
        dp[route[:valid]] = (dy * sig * u * v).sum(1)
        return [dc, dp.view(c["M"], k)]
    end = s["expert_cumsum"].tolist()
    out = torch.zeros((s["dw"] if "dw" in s else s["y"]).shape, dtype=torch.float64, device=DEV)
    for e, (b, n) in enumerate(zip([0] + end[:-1], end)):
        if n == b:
            continue
        token = route[b:n] // k
        a = s["a"][token if op in ("gmm1", "gmm2_dgrad", "gmm2_wgrad") else slice(b, n)].double()
        if op.endswith("wgrad"):
            out[e] = a.t() @ s["b"][token if op == "gmm1_wgrad" else slice(b, n)].double()
            continue
        w = s["w"][e].double()
        y = a @ w if op.endswith("dgrad") else a @ w.t()
        if c.get("act"):
            y = torch.sigmoid(y[:, :I]) * y[:, :I] * y[:, I:] * s["probs"].double().flatten()[route[b:n]].unsqueeze(1)
        out[b:n] = y
    return out


def _exact_sum(rows, idx, M):
    if idx is None:
        return rows.double()
    idx = idx.view(M, -1).long()
    total = torch.zeros((M, rows.shape[1]), dtype=torch.float64, device=DEV)
    for j in range(idx.shape[1]):
        t = torch.nonzero(idx[:, j] >= 0).flatten()
        total[t] += rows[idx[t, j]].double()
    return total


def _exact_norm(s, c):
    """The gradients in 64 bits are autograd's of the forward formulas."""
    def forward(x, v, wa, wb, gate):
        n = v
        if v is not None:
            if wa is not None:
                n = v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * wa
            if gate is not None:
                n = n * gate
            x = x + s["alpha"] * n
        return x, None if wb is None else x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * wb

    wide = lambda t: None if t is None else t.double()
    if c["op"] == "norm":
        v = None if s["rows"] is None else _exact_sum(s["rows"], s["idx"], c["M"])
        r, h = forward(s["x"].double(), v, wide(s["w_after"]), wide(s["w_before"]), wide(s["gate"]))
        return [t for t, o in ((v, s["s"]), (r, s["r"]), (h, s["h"])) if o is not None]
    leaf = lambda t: None if t is None else t.double().requires_grad_()
    v, wa, wb, gate = leaf(s["s"]), leaf(s["w_after"]), leaf(s["w_before"]), leaf(s["gate"])
    # r is what the forward wrote; the residual that gives exactly it is r - alpha gate n
    with torch.no_grad():
        zero = torch.zeros_like(s["r"], dtype=torch.float64)
        x = s["r"].double() - forward(zero, v, wa, None, gate)[0]
    x.requires_grad_()
    r, h = forward(x, v, wa, wb, gate)
    leaves = [t for t in (x, v, wa, wb, gate) if t is not None]
    return list(torch.autograd.grad([r, h], leaves, [s["dr"].double(), _exact_sum(s["dh"], s["idx"], c["M"])]))


def _exact_route_grad(s, c):
    x = s["logits"].double()
    ids = s["expert_idx"].long()
    there = ids >= 0
    part = x > -math.inf
    if c["renormalize"]:
        part = torch.zeros_like(part)
        part[torch.nonzero(there)[:, 0], ids[there]] = True
    x = torch.where(part, x, -math.inf)
    some = part.any(1)
    w = torch.where(some.unsqueeze(1), torch.softmax(torch.where(some.unsqueeze(1), x, 0.0), dim=1), 0.0)
    g = torch.zeros_like(x)
    g[torch.nonzero(there)[:, 0], ids[there]] = s["dprobs"].double()[there]
    return torch.where(part, w * (g - (w * g).sum(1, keepdim=True)), 0.0)
