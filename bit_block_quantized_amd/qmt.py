"""Python binding of libqmt.so: the steps of a model around the 8-bit
floating-point products on AMD Instinct MI355X (gfx950); include/qmt.h has the
definitions.

Argument marshalling only, as for the products: there is no CPU fallback.

    import bit_block_quantized_amd as qmv
    wc, ws = qmv.qmt_quantize_weights(w)                             # [N][K] -> e4m3, float32 scales per 128 x 128
    x, xs, h = qmv.qmx_rmsnorm(y, weight, residual=h, fmt="f8")      # e4m3, float32 scales per 128
    qkv = qmv.qmv_dense("f8", wc, ws, x, xs)                         # float32 [M][(heads + 2 kv_heads) * D]
    q, k = qmv.qmt_qk_norm_rope(qkv, heads, kv_heads, D, table, positions, q_weight, k_weight)
    ...
    logits = qmv.qmv_dense("f8", hc, hs, x, xs)                      # float32 [M][V]
    logprobs, entropy, ids, top = qmv.qmt_logprobs(logits, tokens, 20)

Tensors are C-contiguous and on one GPU; each call runs on that GPU's current
stream (or ``stream``).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

import bit_block_quantized_amd as _q
from .qmx import _TYPE, _choice, _gpu, _out, _tensor

__all__ = ["qmt_quantize_weights", "qmt_dequantize_weights", "qmt_qk_norm_rope", "qmt_logprobs", "qmt_strerror",
           "qmt_lib", "QMT_LIB_PATH"]

QMT_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmt.so")

_STYLE = {"half": 0, "pairs": 1}
_F = torch.float32
_F32, _I32 = (torch.float32,), (torch.int32,)

_lib = None
_fn = {}                    # the library's entries by name


def qmt_lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(QMT_LIB_PATH):
        raise RuntimeError(f"{QMT_LIB_PATH} is not built; run __graft_entry__.build() "
                           "or python -m bit_block_quantized_amd.build")
    L = ctypes.CDLL(QMT_LIB_PATH)
    P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    for name, args in (("qmt_quantize_weights", [I, P, P, P, I, I, I, P]),
                       ("qmt_dequantize_weights", [P, P, I, P, I, I, I, P]),
                       ("qmt_qk_norm_rope", [I, P, I, I, I, I, P, I, I, P, I, P, P, F, I, I, P, P, I, P]),
                       ("qmt_logprobs", [I, P, I, I, P, I, P, P, P, P, P, P])):
        f = getattr(L, name)
        f.restype, f.argtypes = I, args
        _fn[name] = f
    L.qmt_logprobs_workspace.restype, L.qmt_logprobs_workspace.argtypes = ctypes.c_longlong, [I, I, I]
    L.qmt_strerror.restype, L.qmt_strerror.argtypes = ctypes.c_char_p, [I]
    _lib = L
    return L


def qmt_strerror(status: int) -> str:
    return qmt_lib().qmt_strerror(int(status)).decode()


def _run(entry, device, stream, *args):
    """Call a library entry on the tensors' GPU and stream."""
    if _lib is None:
        qmt_lib()
    status = _q._on_device(_fn[entry], device, stream, *args)
    if status != 0:
        raise _q.QmvError(status, qmt_strerror(status))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _matrices(t, name):
    """(E, N, K) of a tensor [N][K] or [..][N][K]."""
    if t.dim() < 2 or t.numel() < 1:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [..][N][K] with at least one value")
    N, K = t.shape[-2:]
    if K % 32:
        raise ValueError(f"{name} has rows of {K} values; blocks need a multiple of 32")
    E = t.numel() // (N * K)
    _q._ints(E, N, K)
    return E, N, K


def _scale_shape(shape):
    return tuple(shape[:-2]) + (_q._blocks128(shape[-2]), _q._blocks128(shape[-1]))


def qmt_quantize_weights(x, codes=None, scales=None, stream=None):
    """Matrices x [..][N][K] (float32, bfloat16 or float16; K % 32 == 0) as "f8"
    weights of the products: (codes float8_e4m3fn [..][N][K], scales float32
    [..][ceil(N/128)][ceil(K/128)])."""
    _tensor(x, "x", _TYPE)
    E, N, K = _matrices(x, "x")
    _gpu(x, "qmt_quantize_weights")
    codes = _out(codes, "codes", (_q.F8_DT, tuple(x.shape)), x.device)
    scales = _out(scales, "scales", (torch.float32, _scale_shape(x.shape)), x.device)
    _run("qmt_quantize_weights", x.device, stream, _TYPE[x.dtype], x.data_ptr(), codes.data_ptr(), scales.data_ptr(),
         E, N, K)
    return codes, scales


def qmt_dequantize_weights(codes, scales, dtype=torch.bfloat16, y=None, stream=None):
    """The values [..][N][K] that "f8" weights stand for, in ``dtype``."""
    if dtype not in _TYPE:
        raise ValueError(f"dtype is {dtype}, expected one of {tuple(_TYPE)}")
    _tensor(codes, "codes", _q.F8_DT)
    E, N, K = _matrices(codes, "codes")
    _tensor(scales, "scales", (torch.float32,), codes.device, _scale_shape(codes.shape))
    _gpu(codes, "qmt_dequantize_weights")
    y = _out(y, "y", (dtype, tuple(codes.shape)), codes.device)
    _run("qmt_dequantize_weights", codes.device, stream, codes.data_ptr(), scales.data_ptr(), _TYPE[dtype],
         y.data_ptr(), E, N, K)
    return y


# Sizes and options of the two small calls: checked once for each set of them,
# the tensors themselves each time (a call of one token is over in less time
# than its checks take).

@functools.lru_cache(maxsize=256)
def _qk_plan(x_shape, table_shape, H, Hk, D, style, dtype):
    """(M, row, H, Hk, D, P, R, rotation, ytype; shape and strides of q, of k)"""
    rotation = _choice(style, _STYLE, "style")
    if dtype not in _TYPE:
        raise ValueError(f"dtype is {dtype}, expected one of {tuple(_TYPE)}")
    if len(x_shape) != 2 or 0 in x_shape:
        raise ValueError(f"x has shape {tuple(x_shape)}, expected [M][row]")
    M, row = x_shape
    if H < 1 or Hk < 0 or D < 8 or D % 8 or D > 512:
        raise ValueError(f"{H} heads and {Hk} key heads of {D}: expected at least 1, at least 0, and a multiple of 8 "
                         "up to 512")
    if row < (H + Hk) * D or row % 4:
        raise ValueError(f"x has rows of {row} values, expected at least {(H + Hk) * D} and a multiple of 4")
    if len(table_shape) != 2 or 0 in table_shape or table_shape[1] % 8 or table_shape[1] > D:
        raise ValueError(f"table has shape {tuple(table_shape)}, expected [P][R] with R % 8 == 0 and 8 <= R <= {D}")
    P, R = table_shape
    _q._ints(M, row, P)
    return (M, row, H, Hk, D, P, R, rotation, _TYPE[dtype],
            ((M, H, D), (H * D, D, 1)), ((M, Hk, D), (Hk * D, D, 1)))


def qmt_qk_norm_rope(x, heads, kv_heads, head_dim, table, positions, q_weight=None, k_weight=None, eps=1e-5,
                     style="half", dtype=torch.bfloat16, q=None, k=None, stream=None):
    """Root-mean-square norm of each query and key head and the rotation by
    position; returns (q [M][heads][D], k [M][kv_heads][D]) in ``dtype`` (k is
    None with ``kv_heads`` 0).

    ``x`` [M][row] holds the query heads, then the key heads (what follows, the
    values say, is left alone); ``table`` float32 [P][R] the R / 2 cosines and
    R / 2 sines of each position; ``positions`` int32 [M], where one outside
    [0, P) gives zeros; ``q_weight`` and ``k_weight`` [D], of one type.
    ``style`` "half" rotates values i and i + R / 2, "pairs" values 2 i and 2 i
    + 1."""
    _tensor(x, "x", _TYPE)
    dev = x.device
    _tensor(table, "table", _F32, dev)
    M, row, H, Hk, D, P, R, rotation, ytype, qs, ks = _qk_plan(x.shape, table.shape, int(heads), int(kv_heads),
                                                               int(head_dim), style, dtype)
    _tensor(positions, "positions", _I32, dev, (M,))
    if q_weight is not None:
        _tensor(q_weight, "q_weight", _TYPE, dev, (D,))
    if k_weight is not None:
        _tensor(k_weight, "k_weight", _TYPE, dev, (D,))
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError(f"q_weight has dtype {q_weight.dtype}, k_weight {k_weight.dtype}; expected one type")
    if k is not None and Hk == 0:
        raise ValueError("k needs key heads")
    _gpu(x, "qmt_qk_norm_rope")
    q = torch.empty_strided(*qs, dtype=dtype, device=dev) if q is None else _out(q, "q", (dtype, qs[0]), dev)
    if Hk:
        k = torch.empty_strided(*ks, dtype=dtype, device=dev) if k is None else _out(k, "k", (dtype, ks[0]), dev)
    w = q_weight if q_weight is not None else k_weight
    _run("qmt_qk_norm_rope", dev, stream, _TYPE[x.dtype], x.data_ptr(), row, H, Hk, D, table.data_ptr(), P, R,
         positions.data_ptr(), 0 if w is None else _TYPE[w.dtype], _ptr(q_weight), _ptr(k_weight), eps, rotation,
         ytype, q.data_ptr(), _ptr(k), M)
    return q, k


@functools.lru_cache(maxsize=256)
def _logprobs_plan(shape, top_k):
    """(M, V, bytes of the workspace)"""
    if len(shape) != 2 or 0 in shape:
        raise ValueError(f"logits has shape {tuple(shape)}, expected [M][V]")
    M, V = shape
    _q._ints(M, V)
    if not 0 <= top_k <= 32:
        raise ValueError(f"top_k is {top_k}, expected 0 to 32")
    return M, V, qmt_lib().qmt_logprobs_workspace(M, V, top_k)


def qmt_logprobs(logits, tokens=None, top_k=0, logprobs=None, entropy=None, top_ids=None, top_logprobs=None,
                 workspace=None, stream=None):
    """Log probability of each row's token, the row's entropy and its top_k
    logits; returns (logprobs float32 [M] or None, entropy float32 [M], top_ids
    int32 [M][top_k], top_logprobs float32 [M][top_k]; the last two None with
    ``top_k`` 0).

    ``logits`` [M][V] (float32, bfloat16 or float16), ``tokens`` int32 [M] (one
    outside [0, V) gives 0).  A logit of -inf or NaN is masked; slots left
    without a logit get id -1 and -inf.  ``workspace``, a uint8 tensor of at
    least qmt_lib().qmt_logprobs_workspace(M, V, top_k) bytes, is taken from
    torch where it is not given."""
    _tensor(logits, "logits", _TYPE)
    top_k = int(top_k)
    M, V, need = _logprobs_plan(logits.shape, top_k)
    dev = logits.device
    if tokens is not None:
        _tensor(tokens, "tokens", _I32, dev, (M,))
    elif logprobs is not None:
        raise ValueError("logprobs needs tokens")
    if top_k == 0 and (top_ids is not None or top_logprobs is not None):
        raise ValueError("top_ids and top_logprobs need top_k")
    if workspace is not None:
        _tensor(workspace, "workspace", (torch.uint8,), dev)
    _gpu(logits, "qmt_logprobs")
    if tokens is not None:
        logprobs = torch.empty_strided((M,), (1,), dtype=_F, device=dev) if logprobs is None else \
            _out(logprobs, "logprobs", (_F, (M,)), dev)
    entropy = torch.empty_strided((M,), (1,), dtype=_F, device=dev) if entropy is None else \
        _out(entropy, "entropy", (_F, (M,)), dev)
    if top_k:
        top_ids = torch.empty_strided((M, top_k), (top_k, 1), dtype=torch.int32, device=dev) if top_ids is None else \
            _out(top_ids, "top_ids", (torch.int32, (M, top_k)), dev)
        top_logprobs = torch.empty_strided((M, top_k), (top_k, 1), dtype=_F, device=dev) if top_logprobs is None else \
            _out(top_logprobs, "top_logprobs", (_F, (M, top_k)), dev)
    if workspace is not None:
        if workspace.numel() < need:
            raise ValueError(f"workspace has {workspace.numel()} bytes, expected at least {need}")
    elif need:
        # (given back to the stream that used it, not to the one that is current here)
        if stream is None:
            workspace = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _run("qmt_logprobs", dev, stream, _TYPE[logits.dtype], logits.data_ptr(), M, V, _ptr(tokens), top_k, _ptr(logprobs),
         _ptr(entropy), _ptr(top_ids), _ptr(top_logprobs), _ptr(workspace) if need else None)
    return logprobs, entropy, top_ids, top_logprobs
