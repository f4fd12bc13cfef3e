"""Python binding of libqmx.so: the steps of an MoE layer around the expert
products on AMD Instinct MI355X (gfx950); include/qmx.h has the definitions.

Argument marshalling only, as for the products: there is no CPU fallback.

    import bit_block_quantized_amd as qmv
    x, xs, h = qmv.qmx_rmsnorm(y, weight, residual=h, fmt="mxfp4")   # codes, scales, new residual
    ids, w = qmv.qmx_router(logits, 4)                               # int32, float32 [M][top_k]
    g = qmv.qmv_gather_moe_swiglu("mxfp4", gc, gs, uc, us, ids, x, xs)
    a, as_ = qmv.qmx_quantize(g)                                     # [M][top_k][N/2], [M][top_k][N/32]
    y = qmv.qmv_gather_moe_combine("mxfp4", dc, ds, ids, w, a, as_)

Formats by name: "mxfp4" (uint8 codes [..][K/2], uint8 E8M0 scales
[..][K/32]), "q8" (int8 codes [..][K], float16 scales [..][K/32]) and, for
the norm's output, "bf16".  Tensors are C-contiguous and on one GPU; each
call runs on that GPU's current stream (or ``stream``).
"""
from __future__ import annotations

import ctypes
import os

import torch

import bit_block_quantized_amd as _q

__all__ = ["qmx_rmsnorm", "qmx_router", "qmx_quantize", "qmx_dequantize", "qmx_strerror", "qmx_lib",
           "QMX_LIB_PATH"]

QMX_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmx.so")

_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_FMT = {"bf16": 0, "q8": 1, "mxfp4": 2}
_SCORING = {"softmax": 0, "sigmoid": 1}

_lib = None


def qmx_lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(QMX_LIB_PATH):
        raise RuntimeError(f"{QMX_LIB_PATH} is not built; run __graft_entry__.build() "
                           "or python -m bit_block_quantized_amd.build")
    L = ctypes.CDLL(QMX_LIB_PATH)
    P, I, F, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
    for name, args in (("qmx_rmsnorm", [I, P, I, P, P, I, P, F, I, P, P, I, I, P]),
                       ("qmx_router", [I, P, I, I, I, I, I, F, P, P, P]),
                       ("qmx_quantize", [I, P, I, P, P, LL, I, P]),
                       ("qmx_dequantize", [I, P, P, I, P, LL, I, P])):
        f = getattr(L, name)
        f.restype, f.argtypes = I, args
    L.qmx_strerror.restype, L.qmx_strerror.argtypes = ctypes.c_char_p, [I]
    _lib = L
    return L


def qmx_strerror(status: int) -> str:
    return qmx_lib().qmx_strerror(int(status)).decode()


def _tensor(t, name, dtypes, device=None, shape=None):
    """``t`` is a contiguous tensor of one of ``dtypes`` (on ``device``, of ``shape``)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _choice(value, table, name):
    if value not in table:
        raise ValueError(f"{name} is {value!r}, expected one of {tuple(table)}")
    return table[value]


def _rows(t, name):
    """(rows, K) of a tensor [..][K]."""
    if t.dim() < 1 or t.shape[-1] < 1 or t.numel() < 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [..][K] with at least one value")
    K = t.shape[-1]
    return t.numel() // K, K


def _blocks(K, name):
    if K % 32:
        raise ValueError(f"{name} has rows of {K} values; blocks need a multiple of 32")


def _code_spec(fmt, lead, K):
    """((codes dtype, shape), (scales dtype, shape)) of rows of K values."""
    if fmt == "mxfp4":
        return (torch.uint8, lead + (K // 2,)), (torch.uint8, lead + (K // 32,))
    return (torch.int8, lead + (K,)), (torch.float16, lead + (K // 32,))


def _out(t, name, spec, device):
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(spec[1], dtype=spec[0], device=device)
    _tensor(t, name, (spec[0],), device, spec[1])
    return t


def _run(entry, device, stream, *args):
    """Call a library entry on the tensors' GPU and stream."""
    status = _q._on_device(getattr(_lib or qmx_lib(), entry), device, stream, *args)
    if status != 0:
        raise _q.QmvError(status, qmx_strerror(status))


def _gpu(t, entry):
    if t.device.type != "cuda":
        raise ValueError(f"{entry} runs on the GPU only; pass device tensors")


def qmx_rmsnorm(x, weight=None, eps=1e-5, residual=None, fmt="bf16", y=None, y_scales=None,
                residual_out=None, stream=None):
    """Residual addition and root-mean-square norm over x's last dimension;
    returns (y, y_scales, residual_out).

    h = x + residual, residual_out = h in the residual's type, y = h /
    sqrt(mean(h^2) + eps) * weight in ``fmt`` ("bf16", or "q8" / "mxfp4" codes
    with y_scales).  y_scales is None for "bf16", residual_out without a
    residual; ``residual_out`` may be ``residual`` itself.  x, residual and
    weight are float32, bfloat16 or float16 each."""
    f = _choice(fmt, _FMT, "fmt")
    _tensor(x, "x", _TYPE)
    M, K = _rows(x, "x")
    _q._ints(M, K)
    dev, shape = x.device, x.shape
    if fmt != "bf16":
        _blocks(K, "x")
    if weight is not None:
        _tensor(weight, "weight", _TYPE, dev, (K,))
    if residual is not None:
        _tensor(residual, "residual", _TYPE, dev, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fmt == "bf16" and y_scales is not None:
        raise ValueError("y_scales is only used with quantized outputs")
    _gpu(x, "qmx_rmsnorm")
    if fmt == "bf16":
        y = _out(y, "y", (torch.bfloat16, shape), dev)
    else:
        cs, ss = _code_spec(fmt, tuple(shape[:-1]), K)
        y, y_scales = _out(y, "y", cs, dev), _out(y_scales, "y_scales", ss, dev)
    if residual is not None:
        residual_out = _out(residual_out, "residual_out", (residual.dtype, shape), dev)
    _run("qmx_rmsnorm", dev, stream, _TYPE[x.dtype], x.data_ptr(),
         0 if residual is None else _TYPE[residual.dtype], None if residual is None else residual.data_ptr(),
         None if residual is None else residual_out.data_ptr(),
         0 if weight is None else _TYPE[weight.dtype], None if weight is None else weight.data_ptr(), eps, f,
         y.data_ptr(), None if y_scales is None else y_scales.data_ptr(), M, K)
    return y, y_scales, residual_out


def qmx_router(logits, top_k, scoring="softmax", normalize=True, scale=1.0, ids=None, weights=None,
               stream=None):
    """The top_k experts of each token and their weights from router logits
    [M][E] (float32 or bfloat16); returns (ids int32 [M][top_k], weights
    float32 [M][top_k]), the largest logit first, the lower index first among
    equals.  ``scoring`` "softmax" or "sigmoid"; ``normalize`` divides by the
    chosen experts' sum (softmax without it: by all experts' sum).  A logit of
    -inf or NaN masks its expert; slots left without one get id -1, weight 0."""
    sc = _choice(scoring, _SCORING, "scoring")
    _tensor(logits, "logits", (torch.float32, torch.bfloat16))
    if logits.dim() != 2 or logits.numel() < 1:
        raise ValueError(f"logits has shape {tuple(logits.shape)}, expected [M][E]")
    M, E = logits.shape
    _q._ints(M, E)
    top_k = int(top_k)
    if not 1 <= top_k <= min(16, E):
        raise ValueError(f"top_k is {top_k}, expected 1 to {min(16, E)}")
    _gpu(logits, "qmx_router")
    dev = logits.device
    ids = _out(ids, "ids", (torch.int32, (M, top_k)), dev)
    weights = _out(weights, "weights", (torch.float32, (M, top_k)), dev)
    _run("qmx_router", dev, stream, _TYPE[logits.dtype], logits.data_ptr(), M, E, top_k, sc, int(bool(normalize)),
         scale, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def qmx_quantize(x, fmt="mxfp4", codes=None, scales=None, stream=None):
    """x [..][K] (float32, bfloat16 or float16; K % 32 == 0) in blocks of 32:
    (codes, scales) in "mxfp4" or "q8"."""
    if fmt not in ("mxfp4", "q8"):
        raise ValueError(f"fmt is {fmt!r}, expected one of ('mxfp4', 'q8')")
    _tensor(x, "x", _TYPE)
    rows, K = _rows(x, "x")
    _q._ints(K)
    _blocks(K, "x")
    _gpu(x, "qmx_quantize")
    cs, ss = _code_spec(fmt, tuple(x.shape[:-1]), K)
    codes, scales = _out(codes, "codes", cs, x.device), _out(scales, "scales", ss, x.device)
    _run("qmx_quantize", x.device, stream, _TYPE[x.dtype], x.data_ptr(), _FMT[fmt], codes.data_ptr(),
         scales.data_ptr(), rows, K)
    return codes, scales


def qmx_dequantize(codes, scales, fmt="mxfp4", dtype=torch.bfloat16, y=None, stream=None):
    """The values [..][K] that (codes, scales) stand for, in ``dtype``."""
    if fmt not in ("mxfp4", "q8"):
        raise ValueError(f"fmt is {fmt!r}, expected one of ('mxfp4', 'q8')")
    if dtype not in _TYPE:
        raise ValueError(f"dtype is {dtype}, expected one of {tuple(_TYPE)}")
    _tensor(codes, "codes", (torch.uint8 if fmt == "mxfp4" else torch.int8,))
    rows, n = _rows(codes, "codes")
    K = 2 * n if fmt == "mxfp4" else n
    _q._ints(K)
    _blocks(K, "codes")
    _, ss = _code_spec(fmt, tuple(codes.shape[:-1]), K)
    _tensor(scales, "scales", (ss[0],), codes.device, ss[1])
    _gpu(codes, "qmx_dequantize")
    y = _out(y, "y", (dtype, tuple(codes.shape[:-1]) + (K,)), codes.device)
    _run("qmx_dequantize", codes.device, stream, _FMT[fmt], codes.data_ptr(), scales.data_ptr(), _TYPE[dtype],
         y.data_ptr(), rows, K)
    return y
