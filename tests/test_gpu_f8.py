"""e4m3 products with a scale per block of 128 (QMV_W_F8B128 x QMV_A_F8B128)
against the 64-bit forms of f8_ref.py (needs an MI355X).

Tolerance of a product: a product of two codes is exact in fp32; each of a
block's 128 additions may lose a last place (2^-23) of a partial sum, which is
at most the sum of the magnitudes A; the two scales' product, its
multiplication and each block's addition round once more (2^-24 each), and
four waves' partial sums join.  So |error| <= (128 + blocks + 4) 2^-23 A.
Where every step is exact in fp32, the results are equal.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import f8_ref as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.double().cpu().numpy()


def codes(rng, shape):
    c = rng.integers(0, 256, shape, dtype=np.uint8)
    return np.where(c & 127 == 127, c ^ 1, c).astype(np.uint8)  # no NaN


def scales(rng, shape):
    return np.exp(rng.standard_normal(shape)).astype(np.float32)


def weights(rng, lead, N, K):
    return codes(rng, lead + (N, K)), scales(rng, lead + (F.blocks(N), F.blocks(K)))


def vectors(rng, lead, K):
    return codes(rng, lead + (K,)), scales(rng, lead + (F.blocks(K),))


def bound(K):
    return (128 + F.blocks(K) + 4) * U


def routed(ids, wv, xv, per_slot):
    """(y, A) of every (token, slot)."""
    M, top_k = ids.shape
    y = np.zeros((M, top_k, wv.shape[1]))
    A = np.zeros_like(y)
    for e in range(wv.shape[0]):
        t, j = np.nonzero(ids == e)
        if len(t):
            x = xv[t, j] if per_slot else xv[t]
            y[t, j], A[t, j] = x @ wv[e].T, np.abs(x) @ np.abs(wv[e]).T
    return y, A


def inside_buffer(shape, fill=7.0):
    """A float32 output between 8 sentinels on either side, off 16-byte alignment."""
    n = int(np.prod(shape))
    buf = torch.full((n + 17,), fill, device="cuda")
    return buf, buf[9:9 + n].view(shape)


def untouched(buf, fill=7.0):
    return bool((buf[:9] == fill).all() and (buf[-8:] == fill).all())


DENSE = [(1, 1, 32), (1, 16, 128), (2, 17, 160), (3, 130, 2880), (4, 300, 16384), (1, 2048, 7168), (5, 128, 128),
         (16, 257, 288), (17, 96, 512), (33, 129, 416), (64, 256, 1024), (65, 384, 160), (130, 200, 7168),
         (64, 4096, 288), (100, 3200, 160), (200, 3210, 416), (20, 8200, 96), (16, 300, 16384), (40, 7000, 2880),
         (300, 700, 544), (1000, 515, 384),
         (2000, 3101, 160), (1300, 5000, 1056), (200, 17000, 288), (8192, 900, 96)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    (wc, ws), (xc, xs) = weights(rng, (), N, K), vectors(rng, (M,), K)
    buf, y = inside_buffer((M, N))
    got = q.qmv_dense("f8", dev(wc), dev(ws), dev(xc), dev(xs), y=y)
    assert got is y and untouched(buf)
    wv, xv = F.weight_values(wc, ws), F.row_values(xc, xs)
    want, A = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert (np.abs(host(y) - want) <= bound(K) * A).all(), (np.abs(host(y) - want) / A).max() / bound(K)
    aligned = q.qmv_dense("f8", dev(wc).view(torch.float8_e4m3fn), dev(ws), dev(xc).view(torch.float8_e4m3fn), dev(xs))
    assert torch.equal(aligned, y)


ROUTED = [(1, 4, 1, 40, 96), (1, 32, 4, 100, 2880), (2, 2000, 3, 33, 160), (4, 8, 16, 50, 256), (3, 1, 1, 129, 7168),
          (5, 7, 3, 65, 288), (20, 16, 4, 130, 512), (40, 300, 8, 64, 128), (64, 4, 2, 300, 416), (150, 3, 2, 96, 1024),
          (200, 5, 5, 257, 160), (33, 9, 2, 70, 16384), (4, 3, 4, 64, 16384), (130, 2, 2, 512, 2080), (700, 6, 4, 200, 96),
          (300, 40, 8, 1030, 64)]


def routing(rng, M, E, top_k, holes):
    ids = rng.integers(0, E, (M, top_k)).astype(np.int32)       # the same expert twice now and then
    if holes:
        bad = rng.random((M, top_k)) < 0.3
        ids = np.where(bad, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (M, top_k)), ids).astype(np.int32)
        ids[rng.integers(M)] = -1
    return ids


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("M,E,top_k,N,K", ROUTED)
def test_gather(M, E, top_k, N, K, per_slot):
    rng = np.random.default_rng(M + E + N + K)
    ids = routing(rng, M, E, top_k, holes=not per_slot)
    (wc, ws), (xc, xs) = weights(rng, (E,), N, K), vectors(rng, (M, top_k) if per_slot else (M,), K)
    buf, y = inside_buffer((M, top_k, N))
    q.qmv_gather_moe("f8", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs), y=y)
    assert untouched(buf)
    want, A = routed(ids, F.weight_values(wc, ws), F.row_values(xc, xs), per_slot)
    assert (np.abs(host(y) - want) <= bound(K) * A).all(), np.nanmax(np.abs(host(y) - want) / A) / bound(K)


@pytest.mark.parametrize("M,E,top_k,N,K", ROUTED)
def test_swiglu(M, E, top_k, N, K):
    rng = np.random.default_rng(M + E + N + K + 1)
    ids = routing(rng, M, E, top_k, holes=M % 2 == 0)
    (gc, gs), (uc, us), (xc, xs) = weights(rng, (E,), N, K), weights(rng, (E,), N, K), vectors(rng, (M,), K)
    gs /= 2e3 * np.sqrt(K)                                      # gates of about 1
    buf, y = inside_buffer((M, top_k, N))
    q.qmv_gather_moe_swiglu("f8", dev(gc), dev(gs), dev(uc), dev(us), dev(ids), dev(xc), dev(xs), y=y)
    assert untouched(buf)
    xv = F.row_values(xc, xs)
    gate, Ag = routed(ids, F.weight_values(gc, gs), xv, False)
    up, Au = routed(ids, F.weight_values(uc, us), xv, False)
    b = bound(K)
    with np.errstate(over="ignore"):
        silu = gate / (1 + np.exp(-gate))
    # silu's slope is at most 1.1; the exponential's argument |gate| 2^-24, and a few roundings
    tol = 1.1 * b * Ag * (np.abs(up) + b * Au) + np.abs(silu) * b * Au + (np.abs(gate) + 8) * 2 * U * np.abs(silu * up)
    assert (np.abs(host(y) - silu * up) <= tol + 1e-30).all()


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("M,E,top_k,N,K", ROUTED)
def test_combine(M, E, top_k, N, K, per_slot):
    rng = np.random.default_rng(M + E + N + K + 2)
    ids = routing(rng, M, E, top_k, holes=per_slot)
    (wc, ws), (xc, xs) = weights(rng, (E,), N, K), vectors(rng, (M, top_k) if per_slot else (M,), K)
    rw = rng.standard_normal((M, top_k)).astype(np.float32)
    buf, y = inside_buffer((M, N))
    args = ("f8", dev(wc), dev(ws), dev(ids), dev(rw), dev(xc))
    q.qmv_gather_moe_combine(*args, dev(xs), y=y)
    assert untouched(buf)
    g, A = routed(ids, F.weight_values(wc, ws), F.row_values(xc, xs), per_slot)
    r = rw.astype(np.float64)[:, :, None]
    tol = ((bound(K) + (top_k + 3) * U) * np.abs(r) * A).sum(1)
    assert (np.abs(host(y) - (r * g).sum(1)) <= tol).all()
    free = torch.empty((M, N), device="cuda")
    q.qmv_gather_moe_combine_noalloc(*args, free, dev(xs))
    assert torch.equal(free, y)


# up to 4 tokens whose slots take more than 64 KB of LDS, of two groups of them the first
BIG_COMBINE = [(4, 16, 8, 100, 7168), (1, 16, 16, 100, 7168), (2, 20, 8, 257, 7072), (3, 9, 11, 70, 6144)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("M,E,top_k,N,K", BIG_COMBINE)
def test_combine_of_many_slots_of_long_rows(M, E, top_k, N, K, per_slot):
    test_combine(M, E, top_k, N, K, per_slot)


def small_exact(rng, shape):
    """Codes of -2 .. 2 in steps of a half: sums of up to 16384 products stay whole quarters below 2^18."""
    v = rng.integers(-4, 5, shape) * 0.5
    return F.codes_of(v.astype(np.float32), np.ones(shape, np.float32)), v


@pytest.mark.parametrize("M,N,K", [(1, 64, 16384), (4, 100, 288), (16, 80, 1024), (64, 4096, 288), (200, 700, 160),
                                   (130, 3300, 416), (600, 1300, 2080), (2100, 260, 544),
                                   (1900, 3400, 544), (700, 9000, 416)])
def test_dense_exact(M, N, K):
    rng = np.random.default_rng(N)
    wc, wv = small_exact(rng, (N, K))
    xc, xv = small_exact(rng, (M, K))
    ws = np.exp2(rng.integers(-1, 2, (F.blocks(N), F.blocks(K)))).astype(np.float32)
    xs = np.exp2(rng.integers(-1, 2, (M, F.blocks(K)))).astype(np.float32)
    y = q.qmv_dense("f8", dev(wc), dev(ws), dev(xc), dev(xs))
    assert np.array_equal(host(y), F.row_values(xc, xs) @ F.weight_values(wc, ws).T)


@pytest.mark.parametrize("M,E,top_k,N,K", [(4, 5, 4, 70, 544), (40, 6, 3, 300, 288), (300, 3, 2, 150, 416),
                                           (500, 9, 8, 1100, 160)])
def test_gather_and_combine_exact(M, E, top_k, N, K):
    rng = np.random.default_rng(E)
    ids = routing(rng, M, E, top_k, True)
    wc, wv = small_exact(rng, (E, N, K))
    xc, xv = small_exact(rng, (M, top_k, K))
    one = np.ones((E, F.blocks(N), F.blocks(K)), np.float32)
    ones = np.ones((M, top_k, F.blocks(K)), np.float32)
    want, _ = routed(ids, wv, xv, True)
    y = q.qmv_gather_moe("f8", dev(wc), dev(one), dev(ids), dev(xc), dev(ones))
    assert np.array_equal(host(y), want)
    rw = np.exp2(rng.integers(-2, 1, (M, top_k))).astype(np.float32)
    c = q.qmv_gather_moe_combine("f8", dev(wc), dev(one), dev(ids), dev(rw), dev(xc), dev(ones))
    assert np.array_equal(host(c), (rw.astype(np.float64)[:, :, None] * want).sum(1))


@pytest.mark.parametrize("M,N,K", [(3, 300, 288), (64, 4096, 288), (600, 1300, 160), (2000, 3101, 160)])
def test_nan_reaches_its_own_outputs_only(M, N, K):
    rng = np.random.default_rng(N)
    (wc, ws), (xc, xs) = weights(rng, (), N, K), vectors(rng, (M,), K)
    wc[17, K - 1], wc[140, 0] = 0x7F, 0xFF
    xc[M - 1, 40] = 0x7F
    ws[2, F.blocks(K) - 1] = np.nan
    y = host(q.qmv_dense("f8", dev(wc), dev(ws), dev(xc), dev(xs)))
    nan = np.zeros((M, N), bool)
    nan[:, [17, 140]] = nan[M - 1] = nan[:, 256:min(N, 384)] = True
    assert np.array_equal(np.isnan(y), nan)


def test_a_slot_without_an_expert_is_zero_whatever_its_vector_holds():
    rng = np.random.default_rng(1)
    for M in (2, 9):
        (wc, ws), (xc, xs) = weights(rng, (4,), 40, 160), vectors(rng, (M, 3), 160)
        ids = rng.integers(0, 4, (M, 3)).astype(np.int32)
        ids[0, 1] = -1
        xc[0, 1], xs[0, 1] = 0x7F, np.nan
        rw = np.ones((M, 3), np.float32)
        y = q.qmv_gather_moe("f8", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs))
        assert not y[0, 1].any() and torch.isfinite(y).all()
        assert torch.isfinite(q.qmv_gather_moe_combine("f8", dev(wc), dev(ws), dev(ids), dev(rw), dev(xc), dev(xs))).all()
        ids[:] = 99
        y = q.qmv_gather_moe("f8", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs), y=torch.full_like(y, 3.0))
        assert not y.any()


def test_repeats_replays_and_streams():
    """Every kernel: the same bits again, from a captured graph with eager work
    between its replays, and on a stream of its own."""
    rng = np.random.default_rng(3)
    sets = []
    for M, E, top_k, N, K in ((2, 8, 4, 96, 544), (90, 8, 3, 300, 288), (600, 4, 4, 260, 160)):
        wc, ws = weights(rng, (E,), N, K)
        uc, us = weights(rng, (E,), N, K)
        xc, xs = vectors(rng, (M,), K)
        sets.append([dev(a) for a in (wc, ws, uc, us, rng.integers(-1, E, (M, top_k)).astype(np.int32),
                                      rng.standard_normal((M, top_k)).astype(np.float32), xc, xs)])
    dw = [dev(a) for a in weights(rng, (), 4100, 288)]
    dx = [dev(a) for a in vectors(rng, (1800,), 288)]

    def calls(stream=None):
        out = [q.qmv_dense("f8", *dw, dx[0][:m], dx[1][:m], stream=stream) for m in (1, 40, 300, 1800)]
        for wc, ws, uc, us, ids, rw, xc, xs in sets:
            out.append(q.qmv_gather_moe("f8", wc, ws, ids, xc, xs, stream=stream))
            out.append(q.qmv_gather_moe_swiglu("f8", wc, ws, uc, us, ids, xc, xs, stream=stream))
            out.append(q.qmv_gather_moe_combine("f8", wc, ws, ids, rw, xc, xs, stream=stream))
        return out

    want = calls()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(calls(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = calls(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls()
    for k in range(4):
        for st in sets:
            st[6].copy_(dev(codes(rng, tuple(st[6].shape))))
        dx[0].copy_(dev(codes(rng, tuple(dx[0].shape))))
        g.replay()
        torch.cuda.synchronize()
        want = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k


# ------------------------------------------------------------- quantizers

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def values(rng, shape, t):
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape[:-1] + (1,)))
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[t]).cuda()


def same_codes(got, want):
    assert np.array_equal(got[1].cpu().numpy(), want[1], equal_nan=True)
    assert np.array_equal(got[0].view(torch.uint8).cpu().numpy(), want[0])


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 128), (5, 160), (2, 2880), (700, 96), (33, 7168), (2, 16384), (5000, 416)])
def test_quantize(rows, K, t):
    x = values(np.random.default_rng(rows + K), (rows, K), t)
    c, s = q.qmx_quantize(x, "f8")
    assert c.dtype == torch.float8_e4m3fn and s.shape == (rows, F.blocks(K))
    want = F.quantize_rows(x.float().cpu().numpy())
    same_codes((c, s), want)
    v = F.row_values(*want)
    for yt in TYPES.values():
        y = q.qmx_dequantize(c, s, "f8", yt)
        assert torch.equal(y.cpu(), torch.from_numpy(v.astype(np.float32)).to(yt))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("lead,N,K", [((), 1, 32), ((), 128, 128), ((3,), 130, 160), ((2, 2), 60, 2880), ((5,), 257, 96),
                                      ((), 1000, 1056)])
def test_quantize_weights(lead, N, K, t):
    x = values(np.random.default_rng(N + K), lead + (N, K), t)
    c, s = q.qmt_quantize_weights(x)
    want = F.quantize_weights(x.float().cpu().numpy())
    same_codes((c, s), want)
    for yt in TYPES.values():
        y = q.qmt_dequantize_weights(c, s, yt)
        assert torch.equal(y.cpu(), torch.from_numpy(F.weight_values(*want).astype(np.float32)).to(yt))


def test_quantize_borders_and_extremes():
    """Values on and next to every border between two codes, with scales that
    make the quotient exact and ones that do not; largest and smallest values;
    blocks with NaN or infinities."""
    rng = np.random.default_rng(4)
    middle = (F.GRID[1:] + F.GRID[:-1]) / 2
    rows = []
    for d in [1.0, 2.0 ** -20, 3.0, 0.7, 1.1e-5] + list(np.exp(rng.standard_normal(40))):
        d32 = np.float32(d)
        top = np.float32(448) * d32                              # may round: the scale is then another one
        b = (middle * np.float64(d32)).astype(np.float32)
        for v in (b, np.nextafter(b, np.float32(1e30)), np.nextafter(b, np.float32(0))):
            rows.append(np.concatenate([[top], v, [0.0]])[:128] * np.where(np.arange(128) % 3 == 1, -1, 1))
    for e in range(-149, 128, 3):
        rows.append(np.ldexp(rng.uniform(0.5, 1, 128), e + 1 - rng.integers(0, 12, 128)))
    rows.append(np.zeros(128))
    rows.append(np.full(128, -0.0))
    rows.append(np.full(128, 2.0 ** -149))
    rows.append(np.full(128, np.finfo(np.float32).max))
    for v in (np.nan, np.inf, -np.inf):
        r = rng.standard_normal(128)
        r[rng.integers(128)] = v
        rows.append(r)
    with np.errstate(over="ignore"):
        x = np.stack(rows).astype(np.float32)
    x[:-3] = np.where(np.isinf(x[:-3]), 1.0, x[:-3])
    same_codes(q.qmx_quantize(dev(x), "f8"), F.quantize_rows(x))
    w = np.repeat(x[:, None], 3, axis=1)                         # the same as matrices of three rows
    same_codes(q.qmt_quantize_weights(dev(w)), F.quantize_weights(w))


@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (1, 2880), (5, 512), (9, 544), (2, 2048), (7, 2080), (4, 4096), (1030, 2080),
                                 (3, 4128), (2, 7168), (2, 8224), (1, 16384), (130, 96)])
def test_rmsnorm(M, K):
    rng = np.random.default_rng(M + K)
    for xt, rt, wt in (("f32", "bf16", "bf16"), ("bf16", None, None), ("f16", "f32", "f16")):
        x = values(rng, (M, K), xt)
        r = None if rt is None else values(rng, (M, K), rt)
        w = None if wt is None else values(rng, (K,), wt)
        y, ys, h = q.qmx_rmsnorm(x, w, residual=r, fmt="f8")
        s = x.float().cpu().numpy()
        if r is not None:
            s = s + r.float().cpu().numpy()
            assert torch.equal(h.cpu(), torch.from_numpy(s).to(r.dtype))
        d = s.astype(np.float64)
        n = d / np.sqrt((d * d).mean(-1, keepdims=True) + np.float64(np.float32(1e-5)))
        n = n * (1.0 if w is None else host(w))
        same_codes((y, ys), F.quantize_rows(n.astype(np.float32)))


def test_quantize_past_32_bit_offsets():
    rows, K = 270000, 16384                                      # 4.4e9 values
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    at = [0, 131071, 131072, 262144, rows - 1]
    vals = values(rng, (len(at), K), "bf16")
    for i, r in enumerate(at):
        x[r] = vals[i]
    want = F.quantize_rows(vals.float().cpu().numpy())
    c, s = q.qmx_quantize(x, "f8")
    for i, r in enumerate(at):
        same_codes((c[r], s[r]), (want[0][i], want[1][i]))
    assert not c.view(torch.uint8)[1:131071].any()
    wc, ws = q.qmt_quantize_weights(x)
    for i, r in enumerate(at):
        lo = r // 128 * 128
        block = x[lo:lo + 128].float().cpu().numpy()
        same_codes((wc[lo:lo + 128], ws[r // 128:r // 128 + 1]), F.quantize_weights(block))
    del x
    y = q.qmx_dequantize(c, s, "f8")
    assert torch.equal(y[rows - 1].float().cpu(), torch.from_numpy(F.row_values(want[0][-1], want[1][-1])).bfloat16().float())
    y = q.qmt_dequantize_weights(wc, ws, y=y)
    assert not y[200000].any() and y[rows - 1].any()
