"""Plain 64-bit forms of the 16-bit products, SwiGLU, the norms and the router's gradient, for the tests, with the
bounds that the kernels' fp32 arithmetic keeps.  torch in float64, one formula at a time; nothing is shared with the kernels.

Bounds.  u = 2^-24 is half an fp32 step.  A matrix instruction multiplies exactly and adds 16 products to a sum; its
additions may round by a whole step, 2 u of the magnitude of what is added.  A sum of n products is at most n / 16 + 1
such steps deep outside and 16 inside, and nothing on the way exceeds S = sum |a| |b|:
    |error| <= (n / 16 + 17) 2 u S
and the result is rounded once to its type, by at most half a step, eps / 2 of its value (2^-25 near 0 in fp16)."""
from __future__ import annotations

import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def half_step(v, t):
    """What rounding v to t may move it by."""
    return v.abs() * (torch.finfo(t).eps / 2) + TINY[t] / 2


def sort(ids, E):
    """Expert-major order of ids [M, top_k]: row_of [R], sorted_route [R], cumsum [E] (int32, on the GPU)."""
    flat = ids.reshape(-1).long().cpu()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.argsort(key, stable=True)
    end = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0)
    n = int(end[-1])
    row_of = torch.full_like(order, -1)
    row_of[order[:n]] = torch.arange(n)
    order[n:] = -1
    return row_of.int().cuda(), order.int().cuda(), end.int().cuda()


def groups(cumsum):
    b = 0
    for e, n in enumerate(cumsum.tolist()):
        if n > b:
            yield e, b, n
        b = n


def product(a, token, w, cumsum, R, transposed=False):
    """Rows times weights [E, N, K] (transposed: [E, K, N]) -> value [R, N], bound; token (nullable): gathered rows."""
    N = w.shape[2] if transposed else w.shape[1]
    v = torch.zeros((R, N), dtype=torch.float64, device=a.device)
    s = torch.zeros_like(v)
    for e, b, n in groups(cumsum):
        x = a[b:n] if token is None else a[token[b:n]]
        x, m = x.double(), w[e].double() if transposed else w[e].double().t()
        v[b:n] = x @ m
        s[b:n] = x.abs() @ m.abs()
    k = a.shape[1]
    return v, s * ((k / 16 + 17) * 2 * U)


def weights(a, ta, b, tb, cumsum, E):
    """Gradient of the weights: value [E, M, N] and bound; ta, tb (nullable): gathered rows."""
    v = torch.zeros((E, a.shape[1], b.shape[1]), dtype=torch.float64, device=a.device)
    s = torch.zeros_like(v)
    for e, i, n in groups(cumsum):
        x = (a[i:n] if ta is None else a[ta[i:n]]).double().t()
        y = (b[i:n] if tb is None else b[tb[i:n]]).double()
        v[e] = x @ y
        s[e] = (x.abs() @ y.abs()) * (((n - i) / 16 + 17) * 2 * U)
    return v, s


def swiglu(c, p, bound=None):
    """p silu(u) g of c [., 2 I] and the bound of its fp32 arithmetic.

    The exponent's argument is off by 2 u |u| and the exponential by a few steps, which move silu by as much relatively;
    the quotient, the two products and the sigmoid's sum round: (2 |u| + 16) u of the value.  bound: that of c itself;
    |silu'| <= 1.1."""
    I = c.shape[1] // 2
    u, g = c[:, :I].double(), c[:, I:].double()
    sig = torch.sigmoid(u)
    y = p * (u * sig) * g
    err = y.abs() * (2 * u.abs().clamp_max(104) + 16) * U
    if bound is not None:
        bu, bg = bound[:, :I], bound[:, I:]
        err = err + p.abs() * (1.1 * bu * g.abs() + (u * sig).abs() * bg + 1.1 * bu * bg)
    return y, err


def swiglu_grad(c, dy, p):
    """dc, its bound, dp (a row each), its bound."""
    I = c.shape[1] // 2
    u, g, d = c[:, :I].double(), c[:, I:].double(), dy.double()
    s = torch.sigmoid(u)
    rel = (2 * u.abs().clamp_max(104) + 24) * U
    # s + u s (1 - s): the two terms may cancel, so the bound takes their magnitudes; 1 - s is off by a step of 1
    du = p * d * g * (s + u * s * (1 - s))
    bu = (p * d * g).abs() * (s + (u * s).abs() * (1 - s + U)) * rel + (p * d * g * u * s).abs() * 8 * U
    dg = p * d * u * s
    dp = d * u * s * g
    # a sum of I terms, 16 to a lane and chunk at most I / 64 deep with the lanes' tree
    bp = dp.abs().mul(rel).sum(1) + dp.abs().sum(1) * (I / 64 + 16) * U
    return torch.cat((du, dg), 1), torch.cat((bu, dg.abs() * rel), 1), dp.sum(1), bp


def rows_sum(rows, row_of, M):
    """Rows of each token's slots, summed, and the sum of their magnitudes."""
    if row_of is None:
        return rows.double(), rows.double().abs()
    idx = row_of.view(M, -1).long()
    v = torch.zeros((M, rows.shape[1]), dtype=torch.float64, device=rows.device)
    s = torch.zeros_like(v)
    for j in range(idx.shape[1]):
        t = torch.nonzero(idx[:, j] >= 0).flatten()
        x = rows[idx[t, j]].double()
        v[t] += x
        s[t] += x.abs()
    return v, s


def norm(x, s, w_after, gate, alpha, w_before, eps):
    """r and h from the rows' sum s (64 bits; None: no block), differentiable."""
    n = s
    if s is not None:
        if w_after is not None:
            n = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * w_after
        if gate is not None:
            n = n * gate
        n = alpha * n
    r = n if x is None else x if n is None else x + n
    h = None if w_before is None else r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * w_before
    return r, h
