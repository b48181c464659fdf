"""Calls of the router, the few-token expert layer and the MXFP4 expert products, as a serving program makes them.

Each case is one call (the quantiser's is a call and the read-back of what it wrote) at sizes that a
mixture-of-experts layer meets: a single decoded token, a decode batch, a prompt.  With `own` false the same
mathematics runs as elementary torch operations in fp32; with `own` true it runs through the framework's entry
points.

The formulas:

route       score[t, e] = logit[t, e] + bias[e] in fp32.  An expert whose score is NaN or -inf takes no part.  The
            top_k others with the largest scores, largest first, ties to the lowest index, are the token's experts;
            slots left over hold -1 with weight 0.  Their weights are softmax(logits), over the chosen experts
            (renormalize) or over every expert that takes part.
few         out = the whole int8 expert layer: x to int8 by token (scale max|x| / 127, halves away from zero), GMM1
            in integers, fp16 of its dequantised output, silu times gate, int8 by row (halves to even), GMM2 in
            integers, fp16, then the bf16 rows of a token weighted by probs.
quant       blocks of 32 along a row share the scale 2^(floor(log2 max|x|) - 2); the elements x / scale are rounded
            to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code) and saturate at 6.
gmm1        y = silu(x w1[u]) * (x w1[gate]) for the rows of every expert's group, x and w1 in MXFP4, y in bf16.
gmm2        out = y w2 for the rows of every expert's group, y and w2 in MXFP4, out in fp16.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token's router row
        dict(name="route one token", op="route", M=1, E=32, top_k=8, type="fp32", bias=False, renormalize=True, masked=0.0),
        # a long prompt over many experts, some switched off, padded tokens at its end
        dict(name="route long prompt", op="route", M=32768, E=256, top_k=8, type="bf16", bias=True, renormalize=False, masked=0.05),
        # single-stream decoding: one token through the whole int8 layer
        dict(name="few one token", op="few", M=1, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # a handful of streams, skewed routing, a route that the router dropped now and then
        dict(name="few five skewed", op="few", M=5, K=4096, E=64, top_k=6, I=1408, routing="zipf", dropped=0.03),
        # the largest batch that the few-token layer takes: nearly every expert has a row
        dict(name="few sixteen tokens", op="few", M=16, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # a decode batch's tokens on their way into the products
        dict(name="quant decode tokens", op="quant", rows=128, cols=7168, type="fp16", valid=128),
        # a prompt's activated rows, the last ones unused because their routes were dropped
        dict(name="quant prompt rows", op="quant", rows=16384, cols=2048, type="bf16", valid=16211),
        # first product of one decoded token: weight streaming and latency
        dict(name="gmm1 one token", op="gmm1", M=1, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # first product of a decode batch
        dict(name="gmm1 decode batch", op="gmm1", M=128, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # first product of a prompt: matrix-core bound
        dict(name="gmm1 prompt", op="gmm1", M=2048, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # second product of a mid-size batch
        dict(name="gmm2 mid batch", op="gmm2", M=512, K=7168, E=32, top_k=8, I=2048, routing="uniform", dropped=0.0),
        # second product of a prompt with skewed routing, experts without rows and dropped routes
        dict(name="gmm2 prompt skewed", op="gmm2", M=4096, K=4096, E=64, top_k=6, I=1408, routing="zipf_empty", dropped=0.02),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "few", "quant", "gmm1", "gmm2"])
    if op == "route":
        E = _log_int(rng, 4, 256)
        return dict(op=op, M=_log_int(rng, 1, 32768), E=E, top_k=rng.randint(1, min(E, 10)), type=rng.choice(sorted(TYPES)),
                    bias=rng.random() < 0.5, renormalize=rng.random() < 0.5, masked=rng.choice([0.0, 0.05, 0.3]))
    if op == "quant":
        rows, cols = _log_int(rng, 1, 16384), 128 * _log_int(rng, 1, 56)
        while rows * cols > 16384 * 2048:
            rows //= 2
        return dict(op=op, rows=rows, cols=cols, type=rng.choice(sorted(TYPES)), valid=rng.choice([rows, rng.randint(1, rows)]))
    E = _log_int(rng, 4, 128)
    top_k = rng.randint(1, min(E, 8))
    K, I = 128 * _log_int(rng, 2, 64), 128 * _log_int(rng, 1, 20)
    while E * K * I > 32 * 7168 * 2048:
        K, I = max(256, K // 256 * 128), max(128, I // 256 * 128)
    M = _log_int(rng, 1, 16 if op == "few" else 4096)
    routing = rng.choice(["uniform", "zipf", "zipf_empty"])
    while routing != "uniform" and E * min(M, 2 * M * top_k) * K > 64 * 4096 * 4096:
        M //= 2
    while M * top_k * K * I > 16384 * 7168 * 2048:
        M //= 2
    if routing == "zipf_empty":
        top_k = max(1, min(top_k, 3 * E // 4))
    dropped = rng.choice([0.0, 0.02, 0.2]) if M * top_k >= 8 else 0.0
    return dict(op=op, M=M, K=K, E=E, top_k=top_k, I=I, routing=routing, dropped=dropped)


# ---------------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _popularity(c):
    """How often each expert is picked first: equal, or falling as rank^-1.2, the last quarter never."""
    p = torch.ones(c["E"], dtype=torch.float64)
    if c["routing"] != "uniform":
        p = (torch.arange(c["E"], dtype=torch.float64) + 1) ** -1.2
    if c["routing"] == "zipf_empty":
        p[3 * c["E"] // 4:] = 0
    return p / p.sum()


def _routes(c, g):
    """Expert ids [M, top_k] int32, distinct within a token, -1 where the route was dropped, and softmax weights."""
    logp = torch.log(_popularity(c)).to(DEV)
    u = torch.rand((c["M"], c["E"]), generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-12)
    ids = torch.topk(logp - torch.log(-torch.log(u)), c["top_k"], dim=1).indices.to(torch.int32)
    gone = torch.rand(ids.shape, generator=g, device=DEV) < c["dropped"]
    probs = torch.softmax(torch.randn(ids.shape, generator=g, device=DEV), dim=1)
    return torch.where(gone, -1, ids), probs


def _sorted(ids, E):
    """The expert-major order of the routes: sorted_route [R] (-1 past the valid rows) and expert_cumsum [E]."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.argsort(key, stable=True).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    cumsum = torch.cumsum(counts, 0).to(torch.int32)
    valid = int(cumsum[-1])
    order[valid:] = -1
    return order, cumsum, int(counts.max())


def _mx_weights(g, E, N, K, std):
    """Normal weights in MXFP4, quantised expert by expert: codes [E, N, K / 2], scales [E, N, K / 32]."""
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((E, N, K // 32), dtype=torch.uint8, device=DEV)
    for e in range(E):
        q[e], s[e] = _mx_quantise(torch.randn((N, K), generator=g, device=DEV) * std)
    return q, s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c=c)
    if c["op"] == "route":
        logits = torch.randn((c["M"], c["E"]), generator=g, device=DEV) * 2
        if c["masked"]:
            off = torch.rand(c["E"], generator=g, device=DEV) < c["masked"]  # experts out of service
            logits = torch.where(off, -math.inf, logits)
            logits[int(c["M"] * 0.98):][1:] = -math.inf  # padded tokens
        s["logits"] = logits.to(TYPES[c["type"]])
        s["bias"] = torch.randn(c["E"], generator=g, device=DEV) * 0.1 if c["bias"] else None
        s["expert_idx"] = torch.zeros((c["M"], c["top_k"]), dtype=torch.int32, device=DEV)
        s["probs"] = torch.zeros((c["M"], c["top_k"]), device=DEV)
    elif c["op"] == "quant":
        x = torch.randn((c["rows"], c["cols"]), generator=g, device=DEV)
        x *= torch.exp(torch.randn((c["rows"], 1), generator=g, device=DEV))  # rows of different size
        x[:, :: max(1, c["cols"] // 5)] *= 12  # channels that stand out
        s["x"] = x.to(TYPES[c["type"]])
        s["valid"] = torch.tensor([c["valid"]], dtype=torch.int32, device=DEV)
        s["q"] = torch.zeros((c["rows"], c["cols"] // 2), dtype=torch.uint8, device=DEV)
        s["scale"] = torch.zeros((c["rows"], c["cols"] // 32), dtype=torch.uint8, device=DEV)
        s["values"] = torch.zeros((c["rows"], c["cols"]), dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "few":
        M, K, E, I = c["M"], c["K"], c["E"], c["I"]
        s["x"] = torch.randn((M, K), generator=g, device=DEV).half()
        s["expert_idx"], s["probs"] = _routes(c, g)
        s["w1"] = torch.randint(-127, 128, (E, K, 2 * I), generator=g, device=DEV, dtype=torch.int8)
        s["w2"] = torch.randint(-127, 128, (E, I, K), generator=g, device=DEV, dtype=torch.int8)
        s["scale1"] = (torch.rand((E, 2 * I), generator=g, device=DEV) + 0.2) * (0.02 / math.sqrt(K))
        s["scale2"] = (torch.rand((E, K), generator=g, device=DEV) + 0.2) * (0.02 / math.sqrt(I))
        if own:  # the packed weights and the workspace that a serving program keeps
            from moe_expert_ffn_amd import megamoe as MM
            d = MM.dims(M, K, E, c["top_k"], I)
            n1, n2 = MM.megamoe_packed_weight_bytes(d)
            s["w1p"] = torch.empty(n1, dtype=torch.int8, device=DEV)
            s["w2p"] = torch.empty(n2, dtype=torch.int8, device=DEV)
            MM.megamoe_prepack_w1(d, s["w1"], s["w1p"])
            MM.megamoe_prepack_w2(d, s["w2"], s["w2p"])
            del s["w1"], s["w2"]
            s["workspace"] = torch.empty(MM.megamoe_few_workspace_bytes(d), dtype=torch.uint8, device=DEV)
        s["out"] = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    else:
        M, K, E, I = c["M"], c["K"], c["E"], c["I"]
        ids, _ = _routes(c, g)
        s["sorted_route"], s["cumsum"], s["most"] = _sorted(ids, E)
        R = M * c["top_k"]
        if c["op"] == "gmm1":
            s["a"], s["a_scale"] = _mx_quantise(torch.randn((M, K), generator=g, device=DEV))
            s["w"], s["w_scale"] = _mx_weights(g, E, 2 * I, K, 1.5 / math.sqrt(K))
            s["y"] = torch.zeros((R, I), dtype=torch.bfloat16, device=DEV)
        else:
            u, v = (torch.randn((R, I), generator=g, device=DEV) * 1.5 for _ in range(2))
            s["a"], s["a_scale"] = _mx_quantise(u * torch.sigmoid(u) * v)
            s["w"], s["w_scale"] = _mx_weights(g, E, K, I, 1 / math.sqrt(I))
            s["y"] = torch.zeros((R, K), dtype=torch.float16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass


def run(s):
    c = s["c"]
    if not own:
        return {"route": _route, "quant": _quant, "few": _few, "gmm1": _gmm, "gmm2": _gmm}[c["op"]](s)
    from moe_expert_ffn_amd import megamoe as MM
    if c["op"] == "route":
        d = MM.dims(c["M"], 128, c["E"], c["top_k"], 128)
        MM.megamoe_route(d, s["logits"], s["expert_idx"], s["probs"], bias=s["bias"], renormalize=c["renormalize"])
        return s["expert_idx"], s["probs"]
    if c["op"] == "quant":
        MM.megamoe_mxfp4_quant(s["x"], s["q"], s["scale"], valid_rows=s["valid"])
        MM.megamoe_mxfp4_dequant(s["q"], s["scale"], s["values"], valid_rows=s["valid"])
        return s["values"]
    d = MM.dims(c["M"], c["K"], c["E"], c["top_k"], c["I"])
    if c["op"] == "few":
        MM.megamoe_forward_few(d, s["x"], s["expert_idx"], s["probs"], s["w1p"], s["scale1"], s["w2p"], s["scale2"],
                               s["out"], s["workspace"])
        return s["out"]
    if c["op"] == "gmm1":
        MM.megamoe_mxfp4_gmm1(d, s["a"], s["a_scale"], s["sorted_route"], s["cumsum"], s["w"], s["w_scale"], s["y"])
    else:
        MM.megamoe_mxfp4_gmm2(d, s["a"], s["a_scale"], s["cumsum"], s["w"], s["w_scale"], s["y"])
    return s["y"]


def _route(s):
    c = s["c"]
    x = s["logits"].float()
    score = x + 0.0 if s["bias"] is None else x + s["bias"]
    out = torch.isnan(score) | (score == -math.inf)
    score = torch.where(out, -math.inf, score + 0.0)  # -0 ties with 0
    top, ids = torch.sort(score, dim=1, descending=True, stable=True)
    ids, chosen = ids[:, : c["top_k"]], top[:, : c["top_k"]] > -math.inf
    x = torch.where(out, -math.inf, x)
    over = torch.where(chosen, x.gather(1, ids), -math.inf) if c["renormalize"] else x
    most = over.amax(1, keepdim=True)
    z = torch.where(over == most, 1.0, torch.exp(over - most))
    z = torch.where(over > -math.inf, z, 0.0)
    w = z if c["renormalize"] else z.gather(1, ids)
    w = torch.where(chosen, w / z.sum(1, keepdim=True), 0.0)
    return torch.where(chosen, ids, -1).to(torch.int32), w


def _mx_quantise(x):
    """MXFP4 codes (two a byte, the even element low) and scale bytes of x along its last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    e = torch.where(most > 0, torch.frexp(most).exponent - 3, -127).clamp(-127, 127)
    a = torch.ldexp(b, -e)
    m = a.abs()
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte()
            + (m >= 3.5).byte() + (m > 5.0).byte() + torch.signbit(a).byte() * 8).flatten(-2)
    return code[..., ::2] + code[..., 1::2] * 16, (e + 127).squeeze(-1).byte()


def _mx_values(q, scale, dtype=torch.float32):
    """What MXFP4 codes and scale bytes stand for."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=q.device)
    v = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), dim=-1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scale.to(dtype) - 127).unsqueeze(-1)).flatten(-2)


def _quant(s):
    v = _mx_values(*_mx_quantise(s["x"])).to(torch.bfloat16)
    row = torch.arange(v.shape[0], device=DEV).unsqueeze(1)
    return torch.where(row < s["valid"], v, 0)


def _few(s):
    """The int8 layer: the products as [experts] batches, over the chosen experts alone where they are fewer."""
    c = s["c"]
    M, k, E, I, t = c["M"], c["top_k"], c["E"], c["I"], torch.float32
    x = s["x"].float()
    pts1 = x.abs().amax(1, keepdim=True) / 127
    v = torch.where(pts1 > 0, x / pts1, 0.0).double()
    q = torch.trunc(v + torch.copysign(torch.full_like(v, 0.5), v)).to(t)
    ids = s["expert_idx"].long()
    use = ids.clamp_min(0).reshape(-1)
    if M * k < E:  # a batch entry for each route
        pick, q, p1 = use, q.repeat_interleave(k, 0).unsqueeze(1), pts1.repeat_interleave(k, 0).unsqueeze(1)
        at = (torch.arange(M * k, device=DEV), 0)
    else:          # every token with every expert
        pick, p1 = slice(None), pts1
        at = (use, torch.arange(M, device=DEV).repeat_interleave(k))
    acc = torch.matmul(q, s["w1"][pick].to(t))
    gmC = (acc.float() * s["scale1"][pick].unsqueeze(1)).half().float() * p1
    u, gate = gmC[..., :I], gmC[..., I:]
    y = u / (1 + torch.exp(-u)) * gate
    most = y.abs().amax(-1, keepdim=True)
    q2 = torch.round(y * torch.where(most > 0, 127 / most, 0.0)).to(t)
    acc = torch.matmul(q2, s["w2"][pick].to(t))
    rows = (acc.float() * s["scale2"][pick].unsqueeze(1)).half().float() * (most / 127)
    rows = rows[at].bfloat16().float().view(M, k, -1)
    return (rows * torch.where(ids >= 0, s["probs"], 0.0).unsqueeze(2)).sum(1).bfloat16()


def _gmm(s):
    """The grouped products: every expert's rows gathered into a batch entry, padded to the largest group."""
    c = s["c"]
    R, I = s["sorted_route"].shape[0], c["I"]
    a = _mx_values(s["a"], s["a_scale"])
    end = s["cumsum"].long()
    begin = torch.cat((torch.zeros_like(end[:1]), end[:-1]))
    row = (begin.unsqueeze(1) + torch.arange(s["most"], device=DEV)).clamp_max(R - 1)
    if c["op"] == "gmm1":
        row = (s["sorted_route"][row].clamp_min(0) // c["top_k"]).long()
    p = torch.matmul(a[row], _mx_values(s["w"], s["w_scale"]).transpose(1, 2))
    if c["op"] == "gmm1":
        u, gate = p[..., :I], p[..., I:]
        p = u / (1 + torch.exp(-u)) * gate
    r = torch.arange(R, device=DEV)
    e = torch.searchsorted(end, r, right=True).clamp_max(c["E"] - 1)
    y = p[e, (r - begin[e]).clamp(0, max(0, s["most"] - 1))]
    return torch.where((r < end[-1]).unsqueeze(1), y, 0.0).to(s["y"].dtype)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without


def _active(c):
    """Expected number of experts with a row."""
    once = 1 - (1 - _popularity(c)) ** c["top_k"] if c["routing"] != "uniform" else torch.full((c["E"],), c["top_k"] / c["E"])
    return float((1 - (1 - once.double() * (1 - c["dropped"])) ** c["M"]).sum())


def work(case):
    c = case
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if c["op"] == "route":
        return {"bytes": c["M"] * (c["E"] * size[c["type"]] + 8 * c["top_k"]) + 4 * c["E"] * c["bias"], "flops": 4 * c["M"] * c["E"]}
    if c["op"] == "quant":  # written once and read back once in 4 bits, and the values
        n = c["valid"] * c["cols"]
        return {"bytes": max(1, n * (size[c["type"]] + 2) + 2 * n * 17 / 32), "flops": 4 * n}
    M, K, I, R = c["M"], c["K"], c["I"], c["M"] * c["top_k"] * (1 - c["dropped"])
    if c["op"] == "few":
        return {"bytes": _active(c) * (3 * I * K + 8 * I + 4 * K) + 4 * M * K + 8 * M * c["top_k"], "flops": 6 * R * I * K}
    if c["op"] == "gmm1":
        return {"bytes": (_active(c) * 2 * I + min(M, R)) * K * 17 / 32 + 2 * R * I, "flops": 4 * R * I * K}
    return {"bytes": (_active(c) * K + R) * I * 17 / 32 + 2 * R * K, "flops": 2 * R * I * K}


# ---------------------------------------------------------------------------------------------------------------
# the same in 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "route":
        x, bias = s["logits"].float().cpu().numpy(), s["bias"]
        score = x if bias is None else x + bias.cpu().numpy()  # the sum is defined in fp32
        out = np.isnan(score) | (score == -np.inf)
        x, score = np.where(out, -np.inf, x.astype(np.float64)), np.where(out, -np.inf, score)
        ids = np.argsort(-score, axis=1, kind="stable")[:, : c["top_k"]]
        chosen = np.take_along_axis(score, ids, 1) > -np.inf
        lx = np.where(chosen, np.take_along_axis(x, ids, 1), -np.inf)
        over = lx if c["renormalize"] else x
        most = over.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            total = np.where(over == most, 1.0, np.exp(over - most))
            total = np.where(over > -np.inf, total, 0.0).sum(1, keepdims=True)
            w = np.where(lx == most, 1.0, np.exp(lx - most)) / np.where(total > 0, total, 1.0)
        return np.where(chosen, ids, -1).astype(np.int32), np.where(chosen, w, 0.0)
    if c["op"] == "quant":
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        res = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        for r in range(0, c["valid"], 1024):
            b = s["x"][r: min(r + 1024, c["valid"])].double().view(-1, c["cols"] // 32, 32)
            most = b.abs().amax(2, keepdim=True).clamp_min(2.0 ** -149)
            scale = torch.exp2((torch.floor(torch.log2(most)) - 2).clamp_min(-127))
            m = (b / scale).abs().clamp_max(6.0)
            hi = torch.searchsorted(grid, m.contiguous()).clamp_max(7)
            lo = (hi - 1).clamp_min(0)
            up, down = grid[hi] - m, m - grid[lo]
            code = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
            res[r: r + b.shape[0]] = (grid[code] * scale * torch.sign(b)).flatten(1)
        return res
    if c["op"] == "few":
        return _exact_few(s)
    a = _mx_values(s["a"], s["a_scale"], torch.float64)
    end = s["cumsum"].tolist()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    for e, (b, n) in enumerate(zip([0] + end[:-1], end)):
        if n > b:
            w = _mx_values(s["w"][e], s["w_scale"][e], torch.float64)
            rows = s["sorted_route"][b:n].long() // c["top_k"] if c["op"] == "gmm1" else slice(b, n)
            p = a[rows] @ w.t()
            y[b:n] = torch.sigmoid(p[:, : c["I"]]) * p[:, : c["I"]] * p[:, c["I"]:] if c["op"] == "gmm1" else p
    return y


def _exact_few(s):
    """Token by token and slot by slot; the codes and the fp16 and bf16 roundings are part of the definition."""
    c = s["c"]
    M, I = c["M"], c["I"]
    out = torch.zeros((M, c["K"]), dtype=torch.float64, device=DEV)
    ids = s["expert_idx"].tolist()
    for e in sorted({i for row in ids for i in row if i >= 0}):
        tok = [t for t in range(M) if e in ids[t]]
        x = s["x"][tok].double()
        # the scale and the quotient are fp32 by definition: x = max|x| / 2 lies on a border, 63.5 steps
        scale = x.abs().amax(1, keepdim=True).float() / 127
        pts1 = scale.double()
        q = torch.sign(x) * torch.floor((x.abs().float() / scale.clamp_min(1e-30)).double() + 0.5)
        h = (q @ s["w1"][e].double() * s["scale1"][e].double()).half().double() * pts1
        y = torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:]
        pts2 = y.abs().amax(1, keepdim=True) / 127
        q2 = torch.round(y / pts2.clamp_min(1e-300))
        rows = ((q2 @ s["w2"][e].double() * s["scale2"][e].double()).half().double() * pts2).bfloat16().double()
        for j, t in enumerate(tok):
            p = sum(float(s["probs"][t, k]) for k in range(c["top_k"]) if ids[t][k] == e)
            out[t] += rows[j] * p
    return out
