"""Plain 64-bit forms of the e4m3 products (include/qmv.h), of their quantizers
and of the steps around them (include/qmx.h, include/qmt.h), in numpy, one
definition after the other.  Shares no code with the package.
tests/test_f8_ref.py pins it to hand-worked values.
"""
import numpy as np

BLOCK = 128
# e4m3 by code: sign, four exponent bits (bias 7), three mantissa bits
E4M3 = np.array([(-1.0 if c & 128 else 1.0) *
                 (np.nan if c & 127 == 127 else
                  (c & 7) * 2.0 ** -9 if not c & 120 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
                 for c in range(256)])
GRID = E4M3[:127]                                              # 0 .. 448, rising


def blocks(n):
    return -(-n // BLOCK)


def spread(scales, n, axis):
    """One scale per block of 128 along `axis` -> one per value."""
    return np.take(np.repeat(scales, BLOCK, axis=axis), np.arange(n), axis=axis)


def row_values(codes, scales):
    """codes uint8 (.., K), scales fp32 (.., blocks) -> values."""
    codes = np.asarray(codes)
    return E4M3[codes] * spread(np.asarray(scales, np.float64), codes.shape[-1], -1)


def weight_values(codes, scales):
    """codes uint8 (.., N, K), scales fp32 (.., blocks, blocks) -> values."""
    codes = np.asarray(codes)
    s = spread(np.asarray(scales, np.float64), codes.shape[-1], -1)
    return E4M3[codes] * spread(s, codes.shape[-2], -2)


def scale_of(amax):
    """The scale of a block with the largest magnitude amax (fp32; not finite: NaN)."""
    with np.errstate(all="ignore"):
        d = np.maximum(np.asarray(amax, np.float32) / np.float32(448), np.float32(2.0 ** -126))
    return np.where(np.isfinite(amax), d, np.float32("nan")).astype(np.float32)


def codes_of(x, d):
    """The codes of fp32 values x with their scales d (same shape): the nearest
    of the quotient in 64 bits, ties to the even code; 0 where d is NaN."""
    ok = np.isfinite(d)
    q = np.abs(np.where(ok, x, 0).astype(np.float64)) / np.where(ok, d, 1).astype(np.float64)
    q = np.minimum(q, 448.0)
    hi = np.searchsorted(GRID, q)                              # GRID[hi - 1] < q <= GRID[hi]
    lo = np.maximum(hi - 1, 0)
    down, up = q - GRID[lo], GRID[hi] - q
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(ok, code | np.where(np.signbit(x), 128, 0), 0).astype(np.uint8)


def quantize_rows(x):
    """fp32 x (.., K) -> (codes uint8 (.., K), scales fp32 (.., blocks))."""
    x = np.asarray(x, np.float32)
    K = x.shape[-1]
    p = np.zeros(x.shape[:-1] + (blocks(K) * BLOCK,), np.float32)
    p[..., :K] = x
    with np.errstate(invalid="ignore"):
        d = scale_of(np.abs(p).reshape(x.shape[:-1] + (-1, BLOCK)).max(-1))
    return codes_of(x, spread(d, K, -1)), d


def quantize_weights(x):
    """fp32 x (.., N, K) -> (codes uint8 (.., N, K), scales fp32 (.., blocks, blocks))."""
    x = np.asarray(x, np.float32)
    N, K = x.shape[-2:]
    p = np.zeros(x.shape[:-2] + (blocks(N) * BLOCK, blocks(K) * BLOCK), np.float32)
    p[..., :N, :K] = x
    with np.errstate(invalid="ignore"):
        d = scale_of(np.abs(p).reshape(x.shape[:-2] + (blocks(N), BLOCK, blocks(K), BLOCK)).max((-3, -1)))
    return codes_of(x, spread(spread(d, K, -1), N, -2)), d


def qk_norm_rope(x, heads, kv_heads, D, table, positions, qw=None, kw=None, eps=1e-5, style="half"):
    """(q (M, heads, D), k (M, kv_heads, D)) in 64 bits."""
    x = np.asarray(x, np.float64)
    M, (P, R) = x.shape[0], table.shape
    out = []
    for lo, H, w in ((0, heads, qw), (heads, kv_heads, kw)):
        y = np.zeros((M, H, D))
        for t in range(M):
            p = int(positions[t])
            if not 0 <= p < P:
                continue
            for h in range(H):
                v = x[t, (lo + h) * D:(lo + h + 1) * D]
                n = v / np.sqrt((v * v).mean() + np.float64(np.float32(eps))) * (1.0 if w is None else np.asarray(w, np.float64))
                o = n.copy()
                for i in range(R // 2):
                    a, b = (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)
                    c, s = float(table[p, i]), float(table[p, R // 2 + i])
                    o[a], o[b] = n[a] * c - n[b] * s, n[b] * c + n[a] * s
                y[t, h] = o
        out.append(y)
    return out


def logprobs(l, tokens, top_k):
    """(logprob (M,), entropy (M,), ids (M, top_k), top logprobs (M, top_k)) in 64 bits."""
    l = np.asarray(l, np.float64)
    M, V = l.shape
    lp, H = np.zeros(M), np.zeros(M)
    ids, top = np.full((M, top_k), -1, np.int32), np.full((M, top_k), -np.inf)
    for r in range(M):
        live = l[r] > -np.inf                                  # NaN compares false
        if live.any():
            with np.errstate(invalid="ignore", over="ignore"):
                m = l[r][live].max()
                z = l[r][live] - m
                e = np.exp(z)
                # log1p of the others: e is exactly 1 at the first largest
                others = np.delete(e, np.argmax(l[r][live])).sum()
                lse = np.log1p(others)
                H[r] = lse - (e * z).sum() / (1.0 + others)
                every = np.where(live, l[r] - m - lse, -np.inf)
                if m == np.inf:
                    H[r], every = np.nan, np.where(live, np.nan, -np.inf)
        else:
            every = np.full(V, -np.inf)
        lp[r] = every[tokens[r]] if 0 <= tokens[r] < V else 0.0
        order = np.argsort(-np.where(live, l[r], -np.inf), kind="stable")[:top_k]
        order = order[live[order]]
        ids[r, :len(order)], top[r, :len(order)] = order, every[order]
    return lp, H, ids, top
