"""Each kernel of the e4m3 products at the sizes where its tiles, chunks and
halves of K begin and end, and calls of more workgroups than one launch takes
(needs an MI355X).  test_f8_launches.py holds each case to the kernel that it
names.  Tolerances are those of test_gpu_f8.py.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import f8_ref as F
import test_gpu_f8 as T
from test_gpu_f8 import bound, dev, host, inside_buffer, routed, untouched, vectors, weights

pytestmark = pytest.mark.gpu

FEW, FEW_GU, FEW_COMB = (f"qmv_f8_few_kernel<{m}>" for m in range(3))
TILE, TILE_GU = "qmv_f8_tile_kernel<0, 1>", "qmv_f8_tile_kernel<1, 1>"         # all of K
HALVES, HALVES_GU = "qmv_f8_tile_kernel<0, 2>", "qmv_f8_tile_kernel<1, 2>"
WIDE = "qmv_f8_wide_kernel"

# rows that end inside a wave's 32, a tile's 128, and on them
DENSE = [(FEW, 31, 16400, 160), (FEW, 33, 9000, 32), (FEW, 64, 8190, 288), (FEW, 65, 7168, 416),
         (FEW, 96, 6500, 128), (HALVES, 97, 8193, 544), (HALVES, 256, 4100, 672),
         (HALVES, 31, 30000, 160), (HALVES, 40, 32700, 32), (HALVES, 32, 32700, 64), (HALVES, 65, 14000, 416),
         (HALVES, 96, 12000, 128), (HALVES, 64, 16390, 800), (HALVES, 40, 32700, 288), (HALVES, 180, 16300, 160),
         (TILE, 32, 33000, 160), (TILE, 64, 32897, 96), (TILE, 200, 11000, 32), (TILE, 97, 16513, 160),
         (TILE, 200, 11100, 288), (TILE, 256, 11000, 544),
         (WIDE, 97, 32800, 160), (WIDE, 129, 16500, 288), (WIDE, 1030, 3700, 96),
         (FEW, 1, 33, 32), (FEW, 8, 1000, 16384), (FEW, 17, 2000, 96), (FEW, 64, 300, 7200)]


@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_dense(kernel, M, N, K):
    rng = np.random.default_rng(M + N + K)
    (wc, ws), (xc, xs) = weights(rng, (), N, K), vectors(rng, (M,), K)
    buf, y = inside_buffer((M, N))
    q.qmv_dense("f8", dev(wc), dev(ws), dev(xc), dev(xs), y=y)
    assert untouched(buf)
    wv, xv = F.weight_values(wc, ws), F.row_values(xc, xs)
    want, A = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert (np.abs(host(y) - want) <= bound(K) * A).all(), (np.abs(host(y) - want) / A).max() / bound(K)


# experts' vectors around a fragment's 32, two, three, and past one chunk's 96
COUNTS = [0, 1, 31, 32, 33, 64, 65, 95, 96, 97, 200]
ROUTED = [(HALVES, 300, 160), (HALVES, 129, 32), (HALVES, 890, 416), (TILE, 5500, 160), (TILE, 5504, 288), (TILE, 5377, 32)]
GU = {HALVES: HALVES_GU, TILE: TILE_GU}


def counted(rng, top_k):
    """ids int32 [M][top_k]: expert e in COUNTS[e] pairs, in any order, and some pairs without one."""
    flat = np.concatenate([np.full(n, e) for e, n in enumerate(COUNTS)] + [np.full(9, -1), np.full(3, len(COUNTS))])
    flat = np.concatenate([flat, np.full(-len(flat) % top_k, -5)])
    return rng.permutation(flat).astype(np.int32).reshape(-1, top_k)


@pytest.mark.parametrize("top_k", [1, 5])
@pytest.mark.parametrize("kernel,N,K", ROUTED)
def test_gather_and_combine(kernel, N, K, top_k):
    rng = np.random.default_rng(N + K + top_k)
    ids, E = counted(rng, top_k), len(COUNTS)
    M = len(ids)
    (wc, ws), (xc, xs) = weights(rng, (E,), N, K), vectors(rng, (M, top_k), K)
    buf, y = inside_buffer((M, top_k, N))
    q.qmv_gather_moe("f8", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs), y=y)
    assert untouched(buf)
    want, A = routed(ids, F.weight_values(wc, ws), F.row_values(xc, xs), True)
    assert (np.abs(host(y) - want) <= bound(K) * A).all()
    rw = rng.standard_normal((M, top_k)).astype(np.float32)
    c = q.qmv_gather_moe_combine("f8", dev(wc), dev(ws), dev(ids), dev(rw), dev(xc), dev(xs))
    r = rw.astype(np.float64)[:, :, None]
    assert (np.abs(host(c) - (r * want).sum(1)) <= ((bound(K) + (top_k + 3) * T.U) * np.abs(r) * A).sum(1)).all()


@pytest.mark.parametrize("kernel,N,K", ROUTED)
def test_swiglu(kernel, N, K):
    rng = np.random.default_rng(N + K)
    ids, E = counted(rng, 3), len(COUNTS)
    (gc, gs), (uc, us), (xc, xs) = weights(rng, (E,), N, K), weights(rng, (E,), N, K), vectors(rng, (len(ids),), K)
    gs /= 2e3 * np.sqrt(K)                                      # gates of about 1
    buf, y = inside_buffer((*ids.shape, N))
    q.qmv_gather_moe_swiglu("f8", dev(gc), dev(gs), dev(uc), dev(us), dev(ids), dev(xc), dev(xs), y=y)
    assert untouched(buf)
    xv = F.row_values(xc, xs)
    gate, Ag = routed(ids, F.weight_values(gc, gs), xv, False)
    up, Au = routed(ids, F.weight_values(uc, us), xv, False)
    b = bound(K)
    with np.errstate(over="ignore"):
        silu = gate / (1 + np.exp(-gate))
    # (as in test_gpu_f8.py)
    tol = 1.1 * b * Ag * (np.abs(up) + b * Au) + np.abs(silu) * b * Au + (np.abs(gate) + 8) * 2 * T.U * np.abs(silu * up)
    assert (np.abs(host(y) - silu * up) <= tol + 1e-30).all()


@pytest.mark.parametrize("kernel,M,N,K", [c for c in DENSE if c[2] > 256 and c[3] >= 160])
def test_a_nan_or_an_infinite_scale_stays_in_its_block_row(kernel, M, N, K):
    """K's last block is a half's missing one, and rows past N repeat the last row."""
    rng = np.random.default_rng(N)
    (wc, ws), (xc, xs) = weights(rng, (), N, K), vectors(rng, (M,), K)
    wc[130, K - 1] = 0x7F
    ws[0, F.blocks(K) - 1] = np.inf
    wc[:128, -32:], xc[:, -32:] = 0x38, 0x38                    # (ones there: the infinite sums have one sign)
    wc[:128, 128 * (K // 128):], xc[:, 128 * (K // 128):] = 0x38, 0x38
    if K % 128 == 0:
        wc[:128, -128:], xc[:, -128:] = 0x38, 0x38
    y = host(q.qmv_dense("f8", dev(wc), dev(ws), dev(xc), dev(xs)))
    assert np.isposinf(y[:, :128]).all() and np.isnan(y[:, 130]).all()
    rest = np.ones(N, bool)
    rest[:128] = rest[130] = False
    assert np.isfinite(y[:, rest]).all()


def test_two_streams_at_once():
    """Calls that overlap on two streams, with each of the kernels, and replays of both in one graph."""
    rng = np.random.default_rng(5)
    E, top_k, N, K = 8, 2, 700, 416
    w = [(dev(c), dev(s)) for c, s in (weights(rng, (E,), N, K), weights(rng, (E,), N, K))]
    calls = []
    for M in (1, 4, 70, 300):
        ids, (xc, xs) = dev(T.routing(rng, M, E, top_k, True)), vectors(rng, (M,), K)
        x, s = dev(xc), dev(xs)
        for c, sc in w:
            calls.append(lambda c=c, sc=sc, ids=ids, x=x, s=s: q.qmv_gather_moe("f8", c, sc, ids, x, s))
            calls.append(lambda c=c, sc=sc, x=x, s=s: q.qmv_dense("f8", c[0], sc[0], x, s))
        calls.append(lambda ids=ids, x=x, s=s: q.qmv_gather_moe_swiglu("f8", *w[0], *w[1], ids, x, s))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None] * len(calls)
    for i, f in enumerate(calls):
        with torch.cuda.stream((a, b)[i % 2]):
            got[i] = f()
    torch.cuda.synchronize()
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [f() for f in calls]
    for _ in range(3):
        for o in out:
            o.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(out, want))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
def test_ties_of_short_values(t):
    """Quotients of 16-bit values by their block's largest: many lie on a border between two codes, more next to one."""
    rng = np.random.default_rng(6)
    largest = torch.from_numpy(np.concatenate([np.arange(128, 256) / 32.0, [3.5 / 2 ** 9, 7 / 2 ** 12]])).to(t)
    x = torch.from_numpy(rng.integers(128, 256, (len(largest), 128)) * np.exp2(rng.integers(-18, -7, (len(largest), 128)))).to(t)
    x = torch.where(x > largest[:, None], largest[:, None], x) * torch.from_numpy(rng.choice([-1.0, 1.0], x.shape)).to(t)
    x[:, 5] = largest
    T.same_codes(q.qmx_quantize(x.cuda(), "f8"), F.quantize_rows(x.float().numpy()))
    m = x[:, None, :].repeat(1, 3, 1)
    T.same_codes(q.qmt_quantize_weights(m.cuda()), F.quantize_weights(m.float().numpy()))


# ------------------------------------------- more workgroups than one launch takes
def test_a_million_matrices():
    E, N, K = (1 << 20) + 100, 1, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(E, N, K, device="cuda", generator=g).to(torch.bfloat16)
    c, s = q.qmt_quantize_weights(x)
    y = q.qmt_dequantize_weights(c, s, torch.float32)
    last = x[-200:].contiguous()
    c1, s1 = q.qmt_quantize_weights(last)
    assert torch.equal(c[-200:].view(torch.uint8), c1.view(torch.uint8)) and torch.equal(s[-200:], s1)
    # a code is off by half a step of its 3 bits, and by half of 2^-9 steps below 2^-6 times the scale
    v = x.float()
    assert ((y - v).abs() <= v.abs() / 16 + s.view(E, 1, 1) * 2.0 ** -10).all()


def test_a_million_rows_of_logits():
    M, V = (1 << 20) + 77, 9
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.randn(M, V, device="cuda", generator=g)
    t = torch.randint(0, V, (M,), device="cuda", generator=g).int()
    lp, H, ids, top = q.qmt_logprobs(l, t, 2)
    all_lp = torch.log_softmax(l.double(), 1)
    # (fp32 exponentials of arguments up to 12, each off by 12 2^-24 of itself and a few roundings; log probabilities up to 12)
    tol = 30 * 2.0 ** -24
    assert ((lp - all_lp.gather(1, t.long()[:, None])[:, 0]).abs() <= tol).all()
    assert ((H + (all_lp.exp() * all_lp).sum(1)).abs() <= 12 * tol).all()
    v, i = l.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), i[:, :2])
    assert ((top - all_lp.gather(1, i[:, :2])).abs() <= tol).all()


def test_sixteen_million_heads():
    M, H, D = 4100, 4096, 264                                   # 16 heads a workgroup: 2^20 + 1024 of them
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(M, H * D, device="cuda", generator=g, dtype=torch.bfloat16)
    a = torch.rand(64, 8, device="cuda", generator=g)
    table = torch.cat([a.cos(), a.sin()], 1).contiguous()
    pos = torch.randint(0, 64, (M,), device="cuda", generator=g).int()
    y, _ = q.qmt_qk_norm_rope(x, H, 0, D, table, pos)
    for t in (0, 2050, M - 5, M - 1):
        want, _ = q.qmt_qk_norm_rope(x[t:t + 1].contiguous(), H, 0, D, table, pos[t:t + 1].contiguous())
        assert torch.equal(y[t:t + 1], want)
