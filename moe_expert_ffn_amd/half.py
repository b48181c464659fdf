"""Thin ctypes binding of include/megamoe/half.h: 16-bit experts, and what training takes.

Argument marshalling and checks only, as in megamoe.py, whose dims, errors and conventions hold here:
the functions keep the C names, tensors are contiguous GPU tensors of the shapes and types the header
states, and a call runs on its tensors' device and that device's current stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .megamoe import (_at, _check, _device, _launch, _route, _type, _workspace, dims, load, megamoe_check_dims,
                      megamoe_dims, megamoe_last_error)

EXPORTED = [
    "megamoe_sort_routes", "megamoe_half_gmm1", "megamoe_half_gmm1_swiglu", "megamoe_half_gmm2",
    "megamoe_half_gmm1_dgrad", "megamoe_half_gmm2_dgrad", "megamoe_half_gmm1_wgrad",
    "megamoe_half_gmm2_wgrad", "megamoe_half_swiglu", "megamoe_half_swiglu_grad", "megamoe_norm",
    "megamoe_norm_grad_workspace_bytes", "megamoe_norm_grad", "megamoe_route_grad",
    "megamoe_half_workspace_bytes", "megamoe_forward_half",
]


def megamoe_sort_routes(d, expert_idx, expanded_row_idx, sorted_route, tokens_per_expert,
                        expert_cumsum, workspace, stream=None):
    R, E, dev, i32 = d.M * d.top_k, d.E, _device(expert_idx), torch.int32
    _launch("megamoe_sort_routes", dev, stream, ctypes.byref(d),
            _at("expert_idx", expert_idx, i32, (d.M, d.top_k), dev),
            _at("expanded_row_idx", expanded_row_idx, i32, (R,), dev),
            _at("sorted_route", sorted_route, i32, (R,), dev),
            _at("tokens_per_expert", tokens_per_expert, i32, (E,), dev),
            _at("expert_cumsum", expert_cumsum, i32, (E,), dev),
            _at("workspace", workspace, None, None, dev),
            workspace.numel() * workspace.element_size())


def _half(t: torch.Tensor | None) -> tuple[int, torch.dtype]:
    """megamoe_type and dtype of a 16-bit tensor."""
    if t is None or t.dtype == torch.bfloat16:  # None: a null pointer, which the library refuses
        return 2, torch.bfloat16
    if t.dtype != torch.float16:
        raise TypeError(f"expected torch.float16 or torch.bfloat16, got {t.dtype}")
    return 1, torch.float16


def megamoe_half_gmm1(d, x, sorted_route, expert_cumsum, w1, c, stream=None):
    """x [M, K] -> c [R, 2I], fp16 or bf16; w1 [E, 2I, K]."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(x), _half(x)
    _launch("megamoe_half_gmm1", dev, stream, ctypes.byref(d), _at("x", x, t, (d.M, K), dev), kind,
            _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("w1", w1, t, (E, 2 * I, K), dev), _at("c", c, t, (R, 2 * I), dev))


def megamoe_half_gmm1_swiglu(d, x, sorted_route, expert_cumsum, w1, y, probs=None, stream=None):
    """x [M, K] -> y [R, I], weighted by probs fp32 [M, top_k] where they are given."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(x), _half(x)
    _launch("megamoe_half_gmm1_swiglu", dev, stream, ctypes.byref(d), _at("x", x, t, (d.M, K), dev),
            kind, _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("probs", probs, torch.float32, (d.M, d.top_k), dev),
            _at("w1", w1, t, (E, 2 * I, K), dev), _at("y", y, t, (R, I), dev))


def megamoe_half_gmm2(d, y, expert_cumsum, w2, gmm2_out, stream=None):
    """y [R, I] -> gmm2_out [R, K]; w2 [E, K, I]."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(y), _half(y)
    _launch("megamoe_half_gmm2", dev, stream, ctypes.byref(d), _at("y", y, t, (R, I), dev), kind,
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("w2", w2, t, (E, K, I), dev), _at("gmm2_out", gmm2_out, t, (R, K), dev))


def megamoe_half_gmm1_dgrad(d, dc, expert_cumsum, w1, dx_rows, stream=None):
    """dc [R, 2I] -> dx_rows [R, K]."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(dc), _half(dc)
    _launch("megamoe_half_gmm1_dgrad", dev, stream, ctypes.byref(d),
            _at("dc", dc, t, (R, 2 * I), dev), kind,
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("w1", w1, t, (E, 2 * I, K), dev), _at("dx_rows", dx_rows, t, (R, K), dev))


def megamoe_half_gmm2_dgrad(d, dout, sorted_route, expert_cumsum, w2, dy, stream=None):
    """dout [M, K] -> dy [R, I]."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(dout), _half(dout)
    _launch("megamoe_half_gmm2_dgrad", dev, stream, ctypes.byref(d),
            _at("dout", dout, t, (d.M, K), dev), kind,
            _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("w2", w2, t, (E, K, I), dev), _at("dy", dy, t, (R, I), dev))


def _dw_type(dw: torch.Tensor | None, kind: int, t: torch.dtype) -> tuple[int, torch.dtype]:
    return (0, torch.float32) if dw is not None and dw.dtype == torch.float32 else (kind, t)


def megamoe_half_gmm1_wgrad(d, dc, x, sorted_route, expert_cumsum, dw1, accumulate=False,
                            stream=None):
    """dc [R, 2I], x [M, K] -> dw1 [E, 2I, K] of their type or fp32."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(dc), _half(dc)
    dk, dt = _dw_type(dw1, kind, t)
    _launch("megamoe_half_gmm1_wgrad", dev, stream, ctypes.byref(d),
            _at("dc", dc, t, (R, 2 * I), dev), _at("x", x, t, (d.M, K), dev), kind,
            _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("dw1", dw1, dt, (E, 2 * I, K), dev), dk, 1 if accumulate else 0)


def megamoe_half_gmm2_wgrad(d, dout, y, sorted_route, expert_cumsum, dw2, accumulate=False,
                            stream=None):
    """dout [M, K], y [R, I] -> dw2 [E, K, I] of their type or fp32."""
    K, E, I, R, dev, (kind, t) = d.K, d.E, d.I, d.M * d.top_k, _device(dout), _half(dout)
    dk, dt = _dw_type(dw2, kind, t)
    _launch("megamoe_half_gmm2_wgrad", dev, stream, ctypes.byref(d),
            _at("dout", dout, t, (d.M, K), dev), _at("y", y, t, (R, I), dev), kind,
            _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("dw2", dw2, dt, (E, K, I), dev), dk, 1 if accumulate else 0)


def megamoe_half_swiglu(d, c, sorted_route, expert_cumsum, y, probs=None, stream=None):
    """c [R, 2I] -> y [R, I], weighted by probs fp32 [M, top_k] where they are given."""
    I, R, dev, (kind, t) = d.I, d.M * d.top_k, _device(c), _half(c)
    _launch("megamoe_half_swiglu", dev, stream, ctypes.byref(d), _at("c", c, t, (R, 2 * I), dev),
            kind, _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (d.E,), dev),
            _at("probs", probs, torch.float32, (d.M, d.top_k), dev), _at("y", y, t, (R, I), dev))


def megamoe_half_swiglu_grad(d, c, dy, sorted_route, expanded_row_idx, expert_cumsum, dc,
                             probs=None, dprobs=None, stream=None):
    """dy [R, I] -> dc [R, 2I] and, where wanted, dprobs fp32 [M, top_k]."""
    I, R, dev, (kind, t) = d.I, d.M * d.top_k, _device(c), _half(c)
    _launch("megamoe_half_swiglu_grad", dev, stream, ctypes.byref(d),
            _at("c", c, t, (R, 2 * I), dev), _at("dy", dy, t, (R, I), dev), kind,
            _at("sorted_route", sorted_route, torch.int32, (R,), dev),
            _at("expanded_row_idx", expanded_row_idx, torch.int32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (d.E,), dev),
            _at("probs", probs, torch.float32, (d.M, d.top_k), dev),
            _at("dc", dc, t, (R, 2 * I), dev),
            _at("dprobs", dprobs, torch.float32, (d.M, d.top_k), dev))


def _gate(gate: torch.Tensor | None, M: int, K: int, dev: int):
    """Address, type, rows and columns of a gate [1 or M, 1 or K]."""
    if gate is None:
        return None, 0, 1, 1
    if gate.dim() != 2 or gate.shape[0] not in (1, M) or gate.shape[1] not in (1, K):
        raise ValueError(f"gate: expected [1 or {M}, 1 or {K}], got {tuple(gate.shape)}")
    return _at("gate", gate, None, None, dev), _type(gate), gate.shape[0], gate.shape[1]


def megamoe_norm(d, x=None, rows=None, expanded_row_idx=None, w_after=None, gate=None, alpha=1.0,
                 w_before=None, eps=1e-6, s=None, r=None, h=None, stream=None):
    """s = rows[t], or summed over the token's routes; n = s / rms(s) * w_after, or s;
    r = x + alpha * gate * n; h = r / rms(r) * w_before.  s, r, h: outputs, those that are
    wanted.  x and r have one type, rows and s one, h its own."""
    # what is not there is passed by at once: at one token the call takes longer than the kernel
    M, K, f32 = d.M, d.K, torch.float32
    dev = _device(rows if x is None else x)
    stream_side, block_side = r if x is None else x, s if rows is None else rows
    xt = bt = None
    xk = bk = 0
    if stream_side is not None:
        xt, xk = stream_side.dtype, _type(stream_side)
    if block_side is not None:
        bt, bk = block_side.dtype, _type(block_side)
    ga, gk, g0, g1 = (None, 0, 1, 1) if gate is None else _gate(gate, M, K, dev)
    R = M if expanded_row_idx is None else M * d.top_k
    _launch("megamoe_norm", dev, stream, ctypes.byref(d),
            None if x is None else _at("x", x, xt, (M, K), dev), xk,
            None if rows is None else _at("rows", rows, bt, (R, K), dev), bk,
            None if expanded_row_idx is None
            else _at("expanded_row_idx", expanded_row_idx, torch.int32, (R,), dev),
            None if w_after is None else _at("w_after", w_after, f32, (K,), dev), ga, gk, g0, g1, alpha,
            None if w_before is None else _at("w_before", w_before, f32, (K,), dev), eps,
            None if s is None else _at("s", s, bt, (M, K), dev),
            None if r is None else _at("r", r, xt, (M, K), dev),
            None if h is None else _at("h", h, None, (M, K), dev), 0 if h is None else _type(h))


def megamoe_norm_grad_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_norm_grad_workspace_bytes",
           load().megamoe_norm_grad_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_norm_grad(d, r, workspace, dr=None, dh=None, expanded_row_idx=None, s=None,
                      w_after=None, gate=None, alpha=1.0, w_before=None, eps=1e-6, dx=None,
                      ds=None, dw_after=None, dw_before=None, dgate=None, stream=None):
    """The gradients of megamoe_norm from its s and r and the gradients dr [M, K] and dh
    ([M, K], or [R, K] with expanded_row_idx); r, dr and dx have one type, s and ds one."""
    M, K, f32, dev = d.M, d.K, torch.float32, _device(dx)
    xt = None if dx is None else dx.dtype
    bt = None if s is None else s.dtype
    R = M if expanded_row_idx is None else M * d.top_k
    ga, gk, g0, g1 = _gate(gate, M, K, dev)
    _launch("megamoe_norm_grad", dev, stream, ctypes.byref(d), _at("dr", dr, xt, (M, K), dev),
            _at("r", r, xt, (M, K), dev), 0 if dx is None else _type(dx),
            _at("dh", dh, None, (R, K), dev), 0 if dh is None else _type(dh),
            _at("expanded_row_idx", expanded_row_idx, torch.int32, (R,), dev),
            _at("s", s, bt, (M, K), dev), 0 if s is None else _type(s),
            _at("w_after", w_after, f32, (K,), dev), ga, gk, g0, g1, alpha,
            _at("w_before", w_before, f32, (K,), dev), eps, _at("dx", dx, xt, (M, K), dev),
            _at("ds", ds, bt, (M, K), dev), _at("dw_after", dw_after, f32, (K,), dev),
            _at("dw_before", dw_before, f32, (K,), dev),
            _at("dgate", dgate, None if gate is None else gate.dtype, (g0, g1), dev),
            _at("workspace", workspace, None, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_route_grad(d, logits, expert_idx, probs, dprobs, dlogits, bias=None, renormalize=True,
                       stream=None):
    """dprobs [M, top_k] -> dlogits [M, E] of the logits' type."""
    M, E, k, dev = d.M, d.E, d.top_k, _device(logits)
    _launch("megamoe_route_grad", dev, stream, ctypes.byref(d),
            _at("logits", logits, None, (M, E), dev), 0 if logits is None else _type(logits),
            None if bias is None else _at("bias", bias, torch.float32, (E,), dev),
            1 if renormalize else 0, _at("expert_idx", expert_idx, torch.int32, (M, k), dev),
            _at("probs", probs, torch.float32, (M, k), dev),
            _at("dprobs", dprobs, torch.float32, (M, k), dev),
            _at("dlogits", dlogits, None if logits is None else logits.dtype, (M, E), dev))


def megamoe_half_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_half_workspace_bytes",
           load().megamoe_half_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_forward_half(d, x, expert_idx, probs, w1, w2, out, workspace, stream=None):
    M, K, E, k, I, dev, (kind, t) = d.M, d.K, d.E, d.top_k, d.I, _device(x), _half(x)
    _launch("megamoe_forward_half", dev, stream, ctypes.byref(d), _at("x", x, t, (M, K), dev), kind,
            _at("expert_idx", expert_idx, torch.int32, (M, k), dev),
            _at("probs", probs, torch.float32, (M, k), dev),
            _at("w1", w1, t, (E, 2 * I, K), dev), _at("w2", w2, t, (E, K, I), dev),
            _at("out", out, t, (M, K), dev), _at("workspace", workspace, None, None, dev),
            workspace.numel() * workspace.element_size())


class HalfPass(NamedTuple):
    """What MegaMoEHalf.forward_rows leaves for backward, and its result: rows [R, K]."""
    x: torch.Tensor
    probs: torch.Tensor
    expanded_row_idx: torch.Tensor
    sorted_route: torch.Tensor
    expert_cumsum: torch.Tensor
    c: torch.Tensor
    y: torch.Tensor
    rows: torch.Tensor


class MegaMoEHalf:
    """Convenience holder: fp16 or bf16 weights + workspace for one set of dims.  The weights stay the
    caller's tensors: what an optimiser writes to them is what the next call multiplies with.

    forward serves.  forward_rows and backward train: a token's output is the sum of its rows, which
    combine gives, or megamoe_norm on its way through the norm after the layer.  forward and forward_rows
    share the workspace: calls of one holder belong in one order."""

    def __init__(self, M: int, K: int, E: int, top_k: int, I: int, dtype=torch.bfloat16, device="cuda"):
        self.d = dims(M, K, E, top_k, I)
        _check("megamoe_check_dims", megamoe_check_dims(self.d))
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"expected torch.float16 or torch.bfloat16, got {dtype}")
        self.dtype = dtype
        self.workspace = _workspace(megamoe_half_workspace_bytes(self.d), device)
        self.device = self.workspace.device  # with its index: "cuda" is another one when another is current
        self.w1 = self.w2 = None

    def _empty(self, *shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.dtype, device=self.device)

    def load_weights(self, w1, w2):
        """w1 [E, 2I, K], w2 [E, K, I]: rows over the reduction, contiguous, of the holder's type."""
        d, dev = self.d, self.workspace.get_device()
        _at("w1", w1, self.dtype, (d.E, 2 * d.I, d.K), dev)
        _at("w2", w2, self.dtype, (d.E, d.K, d.I), dev)
        self.w1, self.w2 = w1, w2

    def route(self, logits, bias=None, renormalize=True):
        """Router logits [M, E] -> expert_idx and probs for forward and forward_rows."""
        return _route(self.d, logits, bias, renormalize)

    def forward(self, x, expert_idx, probs, out=None):
        if out is None:
            out = self._empty(self.d.M, self.d.K)
        megamoe_forward_half(self.d, x, expert_idx, probs, self.w1, self.w2, out, self.workspace)
        return out

    def forward_rows(self, x, expert_idx, probs) -> HalfPass:
        """The layer up to the combine, keeping what backward needs: x and probs themselves, which have to
        hold the same values then.  Rows behind the last group are not written."""
        d, i32 = self.d, torch.int32
        R = d.M * d.top_k
        row_of, route = self._empty(R, dtype=i32), self._empty(R, dtype=i32)
        end = self._empty(d.E, dtype=i32)
        megamoe_sort_routes(d, expert_idx, row_of, route, self._empty(d.E, dtype=i32), end,
                            self.workspace)
        c, y, rows = self._empty(R, 2 * d.I), self._empty(R, d.I), self._empty(R, d.K)
        megamoe_half_gmm1(d, x, route, end, self.w1, c)
        megamoe_half_swiglu(d, c, route, end, y, probs=probs)
        megamoe_half_gmm2(d, y, end, self.w2, rows)
        return HalfPass(x, probs, row_of, route, end, c, y, rows)

    def combine(self, p: HalfPass, rows=None, out=None):
        """Token t's sum over its routes' rows: the layer's output, or that of other rows of its order."""
        if out is None:
            out = self._empty(self.d.M, self.d.K)
        megamoe_norm(self.d, rows=p.rows if rows is None else rows,
                     expanded_row_idx=p.expanded_row_idx, r=out)
        return out

    def backward(self, p: HalfPass, dout, dw1=None, dw2=None, accumulate=False):
        """dout [M, K], the gradient of the combined output -> dx_rows [R, K] (combine sums them to x's),
        dprobs [M, top_k], dw1, dw2.  dw1 and dw2: where the weights' gradients go, of the weights' type
        or fp32, to be added to with accumulate.  Rows of dx_rows behind the last group are not written."""
        if accumulate and (dw1 is None or dw2 is None):
            raise ValueError("accumulate adds to dw1 and dw2, which have to be given")
        d = self.d
        R = d.M * d.top_k
        dw1 = torch.empty_like(self.w1) if dw1 is None else dw1
        dw2 = torch.empty_like(self.w2) if dw2 is None else dw2
        dy, dc, dx_rows = self._empty(R, d.I), self._empty(R, 2 * d.I), self._empty(R, d.K)
        dprobs = self._empty(d.M, d.top_k, dtype=torch.float32)
        megamoe_half_gmm2_dgrad(d, dout, p.sorted_route, p.expert_cumsum, self.w2, dy)
        megamoe_half_gmm2_wgrad(d, dout, p.y, p.sorted_route, p.expert_cumsum, dw2, accumulate)
        megamoe_half_swiglu_grad(d, p.c, dy, p.sorted_route, p.expanded_row_idx, p.expert_cumsum, dc,
                                 probs=p.probs, dprobs=dprobs)
        megamoe_half_gmm1_dgrad(d, dc, p.expert_cumsum, self.w1, dx_rows)
        megamoe_half_gmm1_wgrad(d, dc, p.x, p.sorted_route, p.expert_cumsum, dw1, accumulate)
        return dx_rows, dprobs, dw1, dw2

    def last_error(self) -> int:
        """Routes that the last forward or forward_rows dropped, 0 before the first."""
        return megamoe_last_error(self.workspace)
