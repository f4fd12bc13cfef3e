"""Plain 64-bit forms of the MXFP4 x MXFP4 products and of the steps around
them (include/qmx.h), in numpy, one definition after the other.  Shares no
code with the package.  tests/test_mx_ref.py pins it to hand-worked values.
"""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def pow2(e):
    return np.ldexp(1.0, np.asarray(e))


def values(codes, scales):
    """MXFP4 codes uint8 (.., K/2) and scale bytes (.., K/32) -> values (.., K)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    v = np.stack((E2M1[codes & 15], E2M1[codes >> 4]), axis=-1).reshape(codes.shape[:-1] + (-1,))
    s = np.where(scales == 255, np.nan, pow2(scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def q8_values(codes, scales):
    """int8 codes (.., K) and fp16 scales (.., K/32) -> values."""
    return np.asarray(codes, np.float64) * np.repeat(np.asarray(scales).astype(np.float64), 32, axis=-1)


def quantize_mxfp4(x):
    """x (.., K) -> (codes uint8 (.., K/2), scale bytes uint8 (.., K/32))."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(axis=-1)
    fin = np.isfinite(amax)
    m, e = np.frexp(np.where(fin & (amax > 0), amax, 1.0))       # m in [1/2, 1)
    exp = np.where(m >= 0.875, e, e - 1)                        # 1.75 powers of two and above count as 2
    byte = np.where(amax > 0, np.maximum(exp - 2 + 127, 0), 0)
    byte = np.where(fin, byte, 255).astype(np.int64)
    a = np.abs(np.where(fin[..., None], b, 0.0)) / pow2(np.where(fin, byte, 127) - 127)[..., None]
    grid = E2M1[:8]
    code = np.zeros(b.shape, np.int64)
    best = np.full(b.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):                          # an even code wins a tie
        d = np.abs(a - grid[c])
        code, best = np.where(d < best, c, code), np.minimum(d, best)
    code = np.where(np.signbit(b) & fin[..., None], code + 8, code)
    code = code.reshape(x.shape[:-1] + (-1, 2)).astype(np.uint8)
    return code[..., 0] | (code[..., 1] << 4), byte.astype(np.uint8)


def quantize_q8(x):
    """fp32 x (.., K) -> (int8 codes, fp16 scales); every step in fp32 as defined."""
    x = np.asarray(x, np.float32)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(axis=-1)
    with np.errstate(all="ignore"):
        d16 = (amax / np.float32(127)).astype(np.float16)
        d16 = np.where(np.isfinite(amax), d16, np.float16("nan")).astype(np.float16)
        d = d16.astype(np.float32)[..., None]
        ok = (d > 0) & np.isfinite(d)
        r = np.float32(1) / np.where(ok, d, np.float32(1))
        q = np.where(ok, np.clip(np.rint(np.where(ok, b, 0) * r), -127, 127), 0)
    return q.astype(np.int8).reshape(x.shape), d16


def rmsnorm(x, weight=None, residual=None, eps=1e-5):
    """(normed, h): h is the fp32 sum; normed in 64 bits."""
    h = np.asarray(x, np.float32)
    if residual is not None:
        h = h + np.asarray(residual, np.float32)
    d = h.astype(np.float64)
    r = 1.0 / np.sqrt((d * d).mean(axis=-1, keepdims=True) + np.float64(np.float32(eps)))
    return d * r * (1.0 if weight is None else np.asarray(weight, np.float64)), h


def router(logits, top_k, scoring="softmax", normalize=True, scale=1.0):
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    ids, w = np.full((M, top_k), -1, np.int32), np.zeros((M, top_k))
    for t in range(M):
        live = [e for e in range(E) if l[t, e] > -np.inf]        # NaN compares false
        order = sorted(live, key=lambda e: (-l[t, e], e))[:top_k]
        if not order:
            continue
        top = l[t, order]
        if scoring == "softmax":
            z = np.exp(top - top[0])
            s = z / (z.sum() if normalize else np.exp(l[t, live] - top[0]).sum())
        else:
            # sigmoid times a common factor that keeps far negative logits apart from 0
            z = -np.logaddexp(0.0, -top)
            s = np.exp(z - z.max()) / np.exp(z - z.max()).sum() if normalize else np.exp(z)
        ids[t, :len(order)], w[t, :len(order)] = order, s * scale
    return ids, w


def gather(ids, wv, xv, per_slot):
    """Products of weight values wv (E, N, K) with xv (M, K) or (M, top_k, K):
    (y, A), A the sum of the magnitudes."""
    M, top_k = ids.shape
    y = np.zeros((M, top_k, wv.shape[1]))
    A = np.zeros_like(y)
    for t in range(M):
        for j in range(top_k):
            e = ids[t, j]
            if 0 <= e < wv.shape[0]:
                x = xv[t, j] if per_slot else xv[t]
                y[t, j], A[t, j] = wv[e] @ x, np.abs(wv[e]) @ np.abs(x)
    return y, A
