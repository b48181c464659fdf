"""Thin ctypes binding of the MegaMoE C ABI (include/megamoe.h).

Argument marshalling only: every step of the pipeline runs in the HIP kernels
of libmegamoe.so.  PyTorch provides device memory and the current stream.
The functions keep the C names; tensors must be contiguous CUDA (HIP) tensors
of the dtypes the header states.  fp16 tensors are torch.float16, bf16 tensors
torch.bfloat16.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmegamoe.so")

MEGAMOE_OK = 0
MEGAMOE_EUNSUPPORTED = 2  # dims outside the limits
MEGAMOE_EDEVICE = 5  # megamoe_last_error: routes were dropped


class MegaMoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({strerror(status)})")
        self.status = status


class megamoe_dims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("I", ctypes.c_int32)]

    def __repr__(self):
        return f"megamoe_dims(M={self.M}, K={self.K}, E={self.E}, top_k={self.top_k}, I={self.I})"


EXPORTED = [
    "megamoe_strerror", "megamoe_check_dims", "megamoe_workspace_bytes",
    "megamoe_permute_workspace_bytes", "megamoe_packed_weight_bytes", "megamoe_prepack_w1",
    "megamoe_prepack_w2", "megamoe_forward", "megamoe_permute", "megamoe_permute_tokens",
    "megamoe_permute_noalloc",
    "megamoe_gmm1", "megamoe_gmm1_gather", "megamoe_swiglu_quant", "megamoe_gmm2",
    "megamoe_unpermute", "megamoe_last_error", "megamoe_set_overlap",
    "megamoe_paired_q2_bytes", "megamoe_permute_tokens_paired", "megamoe_swiglu_quant_paired",
    "megamoe_gmm2_paired", "megamoe_gmm1_split_workspace_bytes", "megamoe_gmm1_gather_split",
    "megamoe_route", "megamoe_few_workspace_bytes", "megamoe_forward_few", "megamoe_mxfp4_quant",
    "megamoe_mxfp4_dequant", "megamoe_mxfp4_gmm1", "megamoe_mxfp4_gmm2",
    "megamoe_mxfp4_workspace_bytes", "megamoe_forward_mxfp4",
]

# megamoe_type: element types of the arguments that take more than one
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

_lib = None


def load() -> ctypes.CDLL:
    """Load libmegamoe.so.  There is no fallback: a missing library is an error."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                           "`python -m moe_expert_ffn_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, D, i32, sz = ctypes.c_void_p, ctypes.POINTER(megamoe_dims), ctypes.c_int, ctypes.c_size_t
    psz = ctypes.POINTER(ctypes.c_size_t)
    L.megamoe_strerror.argtypes, L.megamoe_strerror.restype = [i32], ctypes.c_char_p
    L.megamoe_check_dims.argtypes, L.megamoe_check_dims.restype = [D], i32
    L.megamoe_workspace_bytes.argtypes, L.megamoe_workspace_bytes.restype = [D, psz], i32
    L.megamoe_permute_workspace_bytes.argtypes = [D, psz]
    L.megamoe_permute_workspace_bytes.restype = i32
    L.megamoe_packed_weight_bytes.argtypes = [D, psz, psz]
    L.megamoe_packed_weight_bytes.restype = i32
    L.megamoe_prepack_w1.argtypes, L.megamoe_prepack_w1.restype = [D, P, P, P], i32
    L.megamoe_prepack_w2.argtypes, L.megamoe_prepack_w2.restype = [D, P, P, P], i32
    L.megamoe_forward.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_forward.restype = i32
    L.megamoe_permute.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_permute.restype = i32
    L.megamoe_permute_tokens.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_permute_tokens.restype = i32
    L.megamoe_permute_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P, P]
    L.megamoe_permute_noalloc.restype = i32
    L.megamoe_gmm1.argtypes, L.megamoe_gmm1.restype = [D, P, P, P, P, P, P, P], i32
    L.megamoe_gmm1_gather.argtypes = [D, P, P, P, P, P, P, P, P]
    L.megamoe_gmm1_gather.restype = i32
    L.megamoe_swiglu_quant.argtypes = [D, P, P, P, P, P, P]
    L.megamoe_swiglu_quant.restype = i32
    L.megamoe_gmm2.argtypes, L.megamoe_gmm2.restype = [D, P, P, P, P, P, P, P], i32
    L.megamoe_unpermute.argtypes, L.megamoe_unpermute.restype = [D, P, P, P, P, P, P], i32
    L.megamoe_last_error.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
    L.megamoe_last_error.restype = i32
    L.megamoe_set_overlap.argtypes, L.megamoe_set_overlap.restype = [i32], i32
    L.megamoe_paired_q2_bytes.argtypes, L.megamoe_paired_q2_bytes.restype = [D, psz], i32
    L.megamoe_gmm1_split_workspace_bytes.argtypes = [D, psz]
    L.megamoe_gmm1_split_workspace_bytes.restype = i32
    L.megamoe_gmm1_gather_split.argtypes = [D, P, P, P, P, P, P, P, sz, P]
    L.megamoe_gmm1_gather_split.restype = i32
    L.megamoe_permute_tokens_paired.argtypes = [D, P, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_permute_tokens_paired.restype = i32
    L.megamoe_swiglu_quant_paired.argtypes = [D, P, P, P, P, P, P, P]
    L.megamoe_swiglu_quant_paired.restype = i32
    L.megamoe_gmm2_paired.argtypes = [D, P, P, P, P, P, P, P]
    L.megamoe_gmm2_paired.restype = i32
    i64 = ctypes.c_int64
    L.megamoe_route.argtypes, L.megamoe_route.restype = [D, P, i32, P, i32, P, P, P], i32
    L.megamoe_few_workspace_bytes.argtypes, L.megamoe_few_workspace_bytes.restype = [D, psz], i32
    L.megamoe_forward_few.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_forward_few.restype = i32
    L.megamoe_mxfp4_quant.argtypes, L.megamoe_mxfp4_quant.restype = [P, i32, i64, i64, P, P, P, P], i32
    L.megamoe_mxfp4_dequant.argtypes = [P, P, i64, i64, P, P, i32, P]
    L.megamoe_mxfp4_dequant.restype = i32
    L.megamoe_mxfp4_gmm1.argtypes, L.megamoe_mxfp4_gmm1.restype = [D, P, P, P, P, P, P, P, P], i32
    L.megamoe_mxfp4_gmm2.argtypes, L.megamoe_mxfp4_gmm2.restype = [D, P, P, P, P, P, P, P], i32
    L.megamoe_mxfp4_workspace_bytes.argtypes = [D, psz]
    L.megamoe_mxfp4_workspace_bytes.restype = i32
    L.megamoe_forward_mxfp4.argtypes = [D, P, P, P, P, P, P, P, P, P, sz, P]
    L.megamoe_forward_mxfp4.restype = i32
    _lib = L
    return L


def strerror(status: int) -> str:
    try:
        return load().megamoe_strerror(status).decode()
    except Exception:  # noqa: BLE001 - message only
        return "unknown"


def dims(M: int, K: int, E: int, top_k: int, I: int) -> megamoe_dims:
    return megamoe_dims(M, K, E, top_k, I)


def _check(fn: str, rc: int) -> None:
    if rc != MEGAMOE_OK:
        raise MegaMoEError(fn, rc)


def _device(t: torch.Tensor | None) -> int:
    if t is None:  # a null pointer, which the library refuses
        return torch._C._cuda_getDevice()
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on the GPU")
    return dev


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None, dev: int) -> int | None:
    """The address of t, which has to be contiguous, of that type and on device dev."""
    if t is None:
        return None
    if t.get_device() != dev:
        _device(t)
        raise ValueError("tensors must be on one device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _handle(dev: int, stream) -> int:
    """The stream's handle; without one, that of the current stream of the tensors' device."""
    if stream is None:  # the same handle as torch.cuda.current_stream(dev).cuda_stream, sooner
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("the stream must be on the tensors' device")
    return stream.cuda_stream


def _launch(name: str, dev: int, stream, *args) -> None:
    """Calls the entry point `name` with args and the stream, on the tensors' device, whichever is
    current.  Without a stream, that device's current one."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _handle(dev, stream)
    fn = getattr(_lib or load(), name)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != MEGAMOE_OK:
        raise MegaMoEError(name, rc)


def megamoe_check_dims(d: megamoe_dims) -> int:
    return load().megamoe_check_dims(ctypes.byref(d))


def megamoe_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_workspace_bytes", load().megamoe_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_permute_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_permute_workspace_bytes",
           load().megamoe_permute_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_packed_weight_bytes(d: megamoe_dims) -> tuple[int, int]:
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("megamoe_packed_weight_bytes",
           load().megamoe_packed_weight_bytes(ctypes.byref(d), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def megamoe_prepack_w1(d, w1, w1p, stream=None):
    dev = _device(w1)
    _launch("megamoe_prepack_w1", dev, stream, ctypes.byref(d), _ptr(w1, torch.int8, dev),
            _ptr(w1p, torch.int8, dev))


def megamoe_prepack_w2(d, w2, w2p, stream=None):
    dev = _device(w2)
    _launch("megamoe_prepack_w2", dev, stream, ctypes.byref(d), _ptr(w2, torch.int8, dev),
            _ptr(w2p, torch.int8, dev))


def megamoe_forward(d, x, expert_idx, probs, w1p, scale1, w2p, scale2, out, workspace,
                    stream=None):
    dev = _device(x)
    _launch("megamoe_forward", dev, stream, ctypes.byref(d), _ptr(x, torch.float16, dev),
            _ptr(expert_idx, torch.int32, dev), _ptr(probs, torch.float32, dev),
            _ptr(w1p, torch.int8, dev), _ptr(scale1, torch.float32, dev),
            _ptr(w2p, torch.int8, dev), _ptr(scale2, torch.float32, dev),
            _ptr(out, torch.bfloat16, dev), _ptr(workspace, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_permute(d, x, expert_idx, gmA, pts1, expanded_row_idx, sorted_route,
                    tokens_per_expert, expert_cumsum, workspace, stream=None):
    dev = _device(x)
    _launch("megamoe_permute", dev, stream, ctypes.byref(d), _ptr(x, torch.float16, dev),
            _ptr(expert_idx, torch.int32, dev), _ptr(gmA, torch.int8, dev),
            _ptr(pts1, torch.float32, dev), _ptr(expanded_row_idx, torch.int32, dev),
            _ptr(sorted_route, torch.int32, dev), _ptr(tokens_per_expert, torch.int32, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(workspace, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_permute_tokens(d, x, expert_idx, qx, pts1, expanded_row_idx, sorted_route,
                           tokens_per_expert, expert_cumsum, workspace, stream=None):
    dev = _device(x)
    _launch("megamoe_permute_tokens", dev, stream, ctypes.byref(d), _ptr(x, torch.float16, dev),
            _ptr(expert_idx, torch.int32, dev), _ptr(qx, torch.int8, dev),
            _ptr(pts1, torch.float32, dev), _ptr(expanded_row_idx, torch.int32, dev),
            _ptr(sorted_route, torch.int32, dev), _ptr(tokens_per_expert, torch.int32, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(workspace, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_permute_noalloc(d, x, expert_idx, gmA, pts1, expanded_row_idx, sorted_route,
                            tokens_per_expert, expert_cumsum, dropped, stream=None):
    dev = _device(x)
    _launch("megamoe_permute_noalloc", dev, stream, ctypes.byref(d), _ptr(x, torch.float16, dev),
            _ptr(expert_idx, torch.int32, dev), _ptr(gmA, torch.int8, dev),
            _ptr(pts1, torch.float32, dev), _ptr(expanded_row_idx, torch.int32, dev),
            _ptr(sorted_route, torch.int32, dev), _ptr(tokens_per_expert, torch.int32, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(dropped, torch.int32, dev))


def megamoe_gmm1_gather(d, qx, sorted_route, expert_cumsum, w1p, scale1, gmC, acc_dbg=None,
                        stream=None):
    dev = _device(qx)
    _launch("megamoe_gmm1_gather", dev, stream, ctypes.byref(d), _ptr(qx, torch.int8, dev),
            _ptr(sorted_route, torch.int32, dev), _ptr(expert_cumsum, torch.int32, dev),
            _ptr(w1p, torch.int8, dev), _ptr(scale1, torch.float32, dev),
            _ptr(gmC, torch.float16, dev), _ptr(acc_dbg, torch.int32, dev))


def megamoe_gmm1(d, gmA, expert_cumsum, w1p, scale1, gmC, acc_dbg=None, stream=None):
    dev = _device(gmA)
    _launch("megamoe_gmm1", dev, stream, ctypes.byref(d), _ptr(gmA, torch.int8, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(w1p, torch.int8, dev),
            _ptr(scale1, torch.float32, dev), _ptr(gmC, torch.float16, dev),
            _ptr(acc_dbg, torch.int32, dev))


def megamoe_swiglu_quant(d, gmC, pts1, expert_cumsum, q2, pts2, stream=None):
    dev = _device(gmC)
    _launch("megamoe_swiglu_quant", dev, stream, ctypes.byref(d), _ptr(gmC, torch.float16, dev),
            _ptr(pts1, torch.float32, dev), _ptr(expert_cumsum, torch.int32, dev),
            _ptr(q2, torch.int8, dev), _ptr(pts2, torch.float32, dev))


def megamoe_gmm2(d, q2, expert_cumsum, w2p, scale2, gmm2_out, acc_dbg=None, stream=None):
    dev = _device(q2)
    _launch("megamoe_gmm2", dev, stream, ctypes.byref(d), _ptr(q2, torch.int8, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(w2p, torch.int8, dev),
            _ptr(scale2, torch.float32, dev), _ptr(gmm2_out, torch.float16, dev),
            _ptr(acc_dbg, torch.int32, dev))


def megamoe_gmm1_split_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_gmm1_split_workspace_bytes",
           load().megamoe_gmm1_split_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_gmm1_gather_split(d, qx, sorted_route, expert_cumsum, w1p, scale1, gmC, split_ws,
                              stream=None):
    dev = _device(qx)
    _launch("megamoe_gmm1_gather_split", dev, stream, ctypes.byref(d), _ptr(qx, torch.int8, dev),
            _ptr(sorted_route, torch.int32, dev), _ptr(expert_cumsum, torch.int32, dev),
            _ptr(w1p, torch.int8, dev), _ptr(scale1, torch.float32, dev),
            _ptr(gmC, torch.float16, dev), _ptr(split_ws, torch.uint8, dev), split_ws.numel())


def megamoe_paired_q2_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_paired_q2_bytes", load().megamoe_paired_q2_bytes(ctypes.byref(d),
                                                                     ctypes.byref(n)))
    return n.value


def megamoe_permute_tokens_paired(d, x, expert_idx, qx, pts1, expanded_row_idx, sorted_route,
                                  tokens_per_expert, expert_cumsum, prow, workspace,
                                  stream=None):
    dev = _device(x)
    _launch("megamoe_permute_tokens_paired", dev, stream, ctypes.byref(d),
            _ptr(x, torch.float16, dev), _ptr(expert_idx, torch.int32, dev),
            _ptr(qx, torch.int8, dev), _ptr(pts1, torch.float32, dev),
            _ptr(expanded_row_idx, torch.int32, dev), _ptr(sorted_route, torch.int32, dev),
            _ptr(tokens_per_expert, torch.int32, dev), _ptr(expert_cumsum, torch.int32, dev),
            _ptr(prow, torch.int32, dev), _ptr(workspace, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_swiglu_quant_paired(d, gmC, pts1, expert_cumsum, prow, q2p, pts2, stream=None):
    dev = _device(gmC)
    _launch("megamoe_swiglu_quant_paired", dev, stream, ctypes.byref(d),
            _ptr(gmC, torch.float16, dev), _ptr(pts1, torch.float32, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(prow, torch.int32, dev),
            _ptr(q2p, torch.int8, dev), _ptr(pts2, torch.float32, dev))


def megamoe_gmm2_paired(d, q2p, expert_cumsum, w2p, scale2, gmm2_out, acc_dbg=None,
                        stream=None):
    dev = _device(q2p)
    _launch("megamoe_gmm2_paired", dev, stream, ctypes.byref(d), _ptr(q2p, torch.int8, dev),
            _ptr(expert_cumsum, torch.int32, dev), _ptr(w2p, torch.int8, dev),
            _ptr(scale2, torch.float32, dev), _ptr(gmm2_out, torch.float16, dev),
            _ptr(acc_dbg, torch.int32, dev))


def megamoe_unpermute(d, gmm2_out, pts2, expanded_row_idx, probs, out, stream=None):
    dev = _device(gmm2_out)
    _launch("megamoe_unpermute", dev, stream, ctypes.byref(d), _ptr(gmm2_out, torch.float16, dev),
            _ptr(pts2, torch.float32, dev), _ptr(expanded_row_idx, torch.int32, dev),
            _ptr(probs, torch.float32, dev), _ptr(out, torch.bfloat16, dev))


def megamoe_last_error(workspace, stream=None) -> int:
    """The number of routes the last permute / forward on this workspace
    dropped (the library returns MEGAMOE_EDEVICE when it is not zero)."""
    v, dev = ctypes.c_int32(0), _device(workspace)
    with torch.cuda.device(dev):
        rc = load().megamoe_last_error(_ptr(workspace, None, dev), _handle(dev, stream), ctypes.byref(v))
    if rc != MEGAMOE_EDEVICE:
        _check("megamoe_last_error", rc)
    return v.value


def _type(t: torch.Tensor) -> int:
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"expected one of {sorted(map(str, _TYPES))}, got {t.dtype}")
    return kind


def _at(name: str, t: torch.Tensor | None, dtype, shape, dev: int) -> int | None:
    """The address of t, which has to be contiguous and of that type and shape (None: any) on
    device dev.  One function and plain integers: at one token the call takes longer than
    the kernel."""
    if t is None:
        return None
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        _device(t)
        raise ValueError("tensors must be on one device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def megamoe_route(d, logits, expert_idx, probs, bias=None, renormalize=True, stream=None):
    M, E, k, dev = d.M, d.E, d.top_k, _device(logits)
    _launch("megamoe_route", dev, stream, ctypes.byref(d), _at("logits", logits, None, (M, E), dev),
            0 if logits is None else _type(logits),
            None if bias is None else _at("bias", bias, torch.float32, (E,), dev),
            1 if renormalize else 0, _at("expert_idx", expert_idx, torch.int32, (M, k), dev),
            _at("probs", probs, torch.float32, (M, k), dev))


def _packed(name: str, w: torch.Tensor | None, d, k: int, n: int, dev: int) -> int | None:
    """Packed weights of E experts' k by n: columns in whole blocks of 256."""
    need = d.E * k * ((n + 255) // 256 * 256)
    if w is not None and w.numel() < need:
        raise ValueError(f"{name}: expected at least {need} elements, got {w.numel()}")
    return _at(name, w, torch.int8, None, dev)


def megamoe_few_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_few_workspace_bytes",
           load().megamoe_few_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_forward_few(d, x, expert_idx, probs, w1p, scale1, w2p, scale2, out, workspace,
                        stream=None):
    M, K, E, k, I, dev = d.M, d.K, d.E, d.top_k, d.I, _device(x)
    _launch("megamoe_forward_few", dev, stream, ctypes.byref(d),
            _at("x", x, torch.float16, (M, K), dev),
            _at("expert_idx", expert_idx, torch.int32, (M, k), dev),
            _at("probs", probs, torch.float32, (M, k), dev),
            _packed("w1p", w1p, d, K, 2 * I, dev),
            _at("scale1", scale1, torch.float32, (E, 2 * I), dev),
            _packed("w2p", w2p, d, I, K, dev),
            _at("scale2", scale2, torch.float32, (E, K), dev),
            _at("out", out, torch.bfloat16, (M, K), dev),
            _at("workspace", workspace, None, None, dev),
            workspace.numel() * workspace.element_size())


def _rows_cols(x: torch.Tensor) -> tuple[int, int]:
    if x.dim() != 2:
        raise ValueError(f"x: expected [rows, cols], got {tuple(x.shape)}")
    return x.shape


def _valid(valid_rows, dev: int):
    if valid_rows is None:
        return None
    if valid_rows.numel() != 1:
        raise ValueError("valid_rows: expected one element")
    return _at("valid_rows", valid_rows, torch.int32, None, dev)


def megamoe_mxfp4_quant(x, q, scale, valid_rows=None, stream=None):
    """x [rows, cols] fp32, fp16 or bf16 -> q uint8 [rows, cols / 2], scale uint8
    [rows, cols / 32].  valid_rows: int32 device tensor of one element."""
    (rows, cols), dev = _rows_cols(x), _device(x)
    _launch("megamoe_mxfp4_quant", dev, stream, _at("x", x, None, None, dev), _type(x), rows, cols,
            _valid(valid_rows, dev), _at("q", q, torch.uint8, (rows, cols // 2), dev),
            _at("scale", scale, torch.uint8, (rows, cols // 32), dev))


def megamoe_mxfp4_dequant(q, scale, x, valid_rows=None, stream=None):
    (rows, cols), dev = _rows_cols(x), _device(x)
    _launch("megamoe_mxfp4_dequant", dev, stream, _at("q", q, torch.uint8, (rows, cols // 2), dev),
            _at("scale", scale, torch.uint8, (rows, cols // 32), dev), rows, cols,
            _valid(valid_rows, dev), _at("x", x, None, None, dev), _type(x))


def megamoe_mxfp4_gmm1(d, xq, xs, sorted_route, expert_cumsum, w1q, w1s, y, stream=None):
    M, K, E, I, dev = d.M, d.K, d.E, d.I, _device(xq)
    R, u8, i32 = M * d.top_k, torch.uint8, torch.int32
    _launch("megamoe_mxfp4_gmm1", dev, stream, ctypes.byref(d), _at("xq", xq, u8, (M, K // 2), dev),
            _at("xs", xs, u8, (M, K // 32), dev), _at("sorted_route", sorted_route, i32, (R,), dev),
            _at("expert_cumsum", expert_cumsum, i32, (E,), dev),
            _at("w1q", w1q, u8, (E, 2 * I, K // 2), dev), _at("w1s", w1s, u8, (E, 2 * I, K // 32), dev),
            _at("y", y, torch.bfloat16, (R, I), dev))


def megamoe_mxfp4_gmm2(d, yq, ys, expert_cumsum, w2q, w2s, gmm2_out, stream=None):
    K, E, I, dev = d.K, d.E, d.I, _device(yq)
    R, u8 = d.M * d.top_k, torch.uint8
    _launch("megamoe_mxfp4_gmm2", dev, stream, ctypes.byref(d), _at("yq", yq, u8, (R, I // 2), dev),
            _at("ys", ys, u8, (R, I // 32), dev),
            _at("expert_cumsum", expert_cumsum, torch.int32, (E,), dev),
            _at("w2q", w2q, u8, (E, K, I // 2), dev), _at("w2s", w2s, u8, (E, K, I // 32), dev),
            _at("gmm2_out", gmm2_out, torch.float16, (R, K), dev))


def megamoe_mxfp4_workspace_bytes(d: megamoe_dims) -> int:
    n = ctypes.c_size_t(0)
    _check("megamoe_mxfp4_workspace_bytes",
           load().megamoe_mxfp4_workspace_bytes(ctypes.byref(d), ctypes.byref(n)))
    return n.value


def megamoe_forward_mxfp4(d, x, expert_idx, probs, w1q, w1s, w2q, w2s, out, workspace,
                          stream=None):
    M, K, E, k, I, dev, u8 = d.M, d.K, d.E, d.top_k, d.I, _device(x), torch.uint8
    _launch("megamoe_forward_mxfp4", dev, stream, ctypes.byref(d),
            _at("x", x, torch.float16, (M, K), dev),
            _at("expert_idx", expert_idx, torch.int32, (M, k), dev),
            _at("probs", probs, torch.float32, (M, k), dev),
            _at("w1q", w1q, u8, (E, 2 * I, K // 2), dev), _at("w1s", w1s, u8, (E, 2 * I, K // 32), dev),
            _at("w2q", w2q, u8, (E, K, I // 2), dev), _at("w2s", w2s, u8, (E, K, I // 32), dev),
            _at("out", out, torch.bfloat16, (M, K), dev),
            _at("workspace", workspace, None, None, dev),
            workspace.numel() * workspace.element_size())


def megamoe_set_overlap(mode: int) -> None:
    """0: GMM1 then SwiGLU (default); 1: SwiGLU overlaps GMM1's last round;
    2: as 1, with the overlap's waits giving up at once (its fallback path)."""
    _check("megamoe_set_overlap", load().megamoe_set_overlap(int(mode)))


class MegaMoE:
    """Convenience holder: packed weights + workspace for one set of dims.  forward and
    forward_few share the workspace: calls of one holder belong in one order."""

    def __init__(self, M: int, K: int, E: int, top_k: int, I: int, device="cuda"):
        self.d = dims(M, K, E, top_k, I)
        _check("megamoe_check_dims", megamoe_check_dims(self.d))
        self.device = torch.device(device)
        self.workspace = torch.empty(megamoe_workspace_bytes(self.d), dtype=torch.uint8,
                                     device=self.device)
        # forward_few, where the dims allow it, works in the same memory (it needs less), so that
        # the dropped-route word is that of the newest forward on the GPU, replayed graphs included
        self.few_workspace = self.workspace if M <= 16 and M * top_k <= 512 else None
        n1, n2 = megamoe_packed_weight_bytes(self.d)
        self.w1p = torch.empty(n1, dtype=torch.int8, device=self.device)
        self.w2p = torch.empty(n2, dtype=torch.int8, device=self.device)
        self.scale1 = None
        self.scale2 = None

    def load_weights(self, w1, scale1, w2, scale2):
        megamoe_prepack_w1(self.d, w1, self.w1p)
        megamoe_prepack_w2(self.d, w2, self.w2p)
        self.scale1 = scale1.contiguous()
        self.scale2 = scale2.contiguous()

    def route(self, logits, bias=None, renormalize=True):
        """Router logits [M, E] -> expert_idx and probs for forward and forward_few."""
        return _route(self.d, logits, bias, renormalize)

    def forward(self, x, expert_idx, probs, out=None):
        if out is None:
            out = torch.empty((self.d.M, self.d.K), dtype=torch.bfloat16, device=self.device)
        megamoe_forward(self.d, x, expert_idx, probs, self.w1p, self.scale1, self.w2p,
                        self.scale2, out, self.workspace)
        return out

    def forward_few(self, x, expert_idx, probs, out=None):
        """forward in two kernels, for M <= 16: the same result, sooner for the smallest batches."""
        if self.few_workspace is None:
            raise MegaMoEError("megamoe_forward_few", MEGAMOE_EUNSUPPORTED)
        if out is None:
            out = torch.empty((self.d.M, self.d.K), dtype=torch.bfloat16, device=self.device)
        megamoe_forward_few(self.d, x, expert_idx, probs, self.w1p, self.scale1, self.w2p,
                            self.scale2, out, self.few_workspace)
        return out

    def last_error(self) -> int:
        """Routes that the last forward dropped."""
        return megamoe_last_error(self.workspace)


class MegaMoEMXFP4:
    """Convenience holder: MXFP4 weights + workspace for one set of dims."""

    def __init__(self, M: int, K: int, E: int, top_k: int, I: int, device="cuda"):
        self.d = dims(M, K, E, top_k, I)
        _check("megamoe_check_dims", megamoe_check_dims(self.d))
        self.device = torch.device(device)

        def empty(*shape):
            return torch.empty(shape, dtype=torch.uint8, device=self.device)

        self.workspace = empty(megamoe_mxfp4_workspace_bytes(self.d))
        self.w1q, self.w1s = empty(E, 2 * I, K // 2), empty(E, 2 * I, K // 32)
        self.w2q, self.w2s = empty(E, K, I // 2), empty(E, K, I // 32)
        for s in (self.w1s, self.w2s):
            s.fill_(255)  # NaN: what a forward answers before load_weights

    def load_weights(self, w1, w2):
        """w1 [E, 2I, K], w2 [E, K, I], fp32, fp16 or bf16: rows over the reduction."""
        d = self.d
        weights = ((w1, self.w1q, self.w1s, (d.E, 2 * d.I, d.K)), (w2, self.w2q, self.w2s, (d.E, d.K, d.I)))
        for w, q, _, shape in weights:  # all of it before the first is written
            if w.shape != shape:
                raise ValueError(f"expected weights of shape {shape}, got {tuple(w.shape)}")
            if _device(w) != q.get_device():
                raise ValueError("weights must be on the holder's device")
            _type(w)
        for w, q, s, _ in weights:
            megamoe_mxfp4_quant(w.reshape(-1, w.shape[2]).contiguous(), q.view(-1, q.shape[2]),
                                s.view(-1, s.shape[2]))

    def route(self, logits, bias=None, renormalize=True):
        """Router logits [M, E] -> expert_idx and probs for forward."""
        return _route(self.d, logits, bias, renormalize)

    def forward(self, x, expert_idx, probs, out=None):
        if out is None:
            out = torch.empty((self.d.M, self.d.K), dtype=torch.bfloat16, device=self.device)
        megamoe_forward_mxfp4(self.d, x, expert_idx, probs, self.w1q, self.w1s, self.w2q,
                              self.w2s, out, self.workspace)
        return out

    def last_error(self) -> int:
        """Routes that the last forward dropped."""
        return megamoe_last_error(self.workspace)


def _route(d, logits, bias, renormalize):
    ids = torch.empty((d.M, d.top_k), dtype=torch.int32, device=logits.device)
    probs = torch.empty((d.M, d.top_k), dtype=torch.float32, device=logits.device)
    megamoe_route(d, logits, ids, probs, bias=bias, renormalize=renormalize)
    return ids, probs
