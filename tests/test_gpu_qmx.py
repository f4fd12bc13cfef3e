"""The norm, the router and the block quantizers (include/qmx.h) against the
64-bit forms of mx_ref.py, and a whole MoE layer of them (needs an MI355X).

Tolerances.  Codes, scales and ids are compared exactly.  A bf16 output is
half a step (2^-8 of the value) from the fp32 value, which is 2^-24 from the
64-bit one.  A router weight is a few exponentials (2 ulp each, and
|l - top| 2^-24 from the rounded argument), a sum of at most 16 (1024 without
normalize) terms and a division.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import mx_ref as R

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rand(rng, shape, t, spread=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * spread).astype(np.float32)).to(TYPES[t]).cuda()


def f32(t):
    return t.float().cpu().numpy()


def check_blocks(fmt, codes, scales, x32):
    """codes and scales are exactly those of the fp32 values x32."""
    if fmt == "mxfp4":
        c, s = R.quantize_mxfp4(x32)
        assert np.array_equal(scales.cpu().numpy(), s)
        assert np.array_equal(codes.cpu().numpy(), c)
    else:
        c, s = R.quantize_q8(x32)
        assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
        assert np.array_equal(codes.cpu().numpy(), c)


def check_norm(x, weight, residual, fmt, eps=1e-5):
    y, ys, h = q.qmx_rmsnorm(x, weight, eps=eps, residual=residual, fmt=fmt)
    want, h32 = R.rmsnorm(f32(x), None if weight is None else f32(weight), None if residual is None else f32(residual), eps)
    if residual is None:
        assert h is None
    else:
        assert h.dtype == residual.dtype and torch.equal(h.cpu(), torch.from_numpy(h32).to(residual.dtype))
    if fmt == "bf16":
        got = y.double().cpu().numpy()
        assert ys is None and (np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133).all()
    else:
        check_blocks(fmt, y, ys, want.astype(np.float32))


@pytest.mark.parametrize("fmt", ["bf16", "q8", "mxfp4"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (1, 2880), (5, 512), (9, 544), (2, 2048), (7, 2080), (4, 4096),
                                 (3, 4128), (2, 7168), (3, 8192), (2, 8224), (1, 16384), (130, 96)])
def test_rmsnorm_sizes(M, K, fmt):
    rng = np.random.default_rng(M * 31 + K)
    check_norm(rand(rng, (M, K), "f32", 3.0), rand(rng, (K,), "bf16"), rand(rng, (M, K), "bf16", 20.0), fmt)


@pytest.mark.parametrize("fmt", ["bf16", "q8", "mxfp4"])
@pytest.mark.parametrize("M,K", [(1024, 2080), (1030, 4096), (1023, 2880)])
def test_rmsnorm_many_rows(M, K, fmt):
    rng = np.random.default_rng(M + K)
    check_norm(rand(rng, (M, K), "bf16", 3.0), rand(rng, (K,), "bf16"), rand(rng, (M, K), "f32", 20.0), fmt)


@pytest.mark.parametrize("fmt", ["bf16", "q8", "mxfp4"])
@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("rt", [None, "f32", "bf16", "f16"])
def test_rmsnorm_types(xt, rt, fmt):
    rng = np.random.default_rng(5)
    wt = {None: None, "f32": "bf16", "bf16": "f32", "f16": "f16"}[rt]
    check_norm(rand(rng, (6, 352), xt), None if wt is None else rand(rng, (352,), wt),
               None if rt is None else rand(rng, (6, 352), rt), fmt)


@pytest.mark.parametrize("M,K", [(1, 1), (5, 7), (3, 63), (2, 250), (2, 257), (4, 1001), (777, 37), (3, 4095), (2, 4097),
                                 (2, 8191), (1, 16383), (9, 12), (2, 2890)])
@pytest.mark.parametrize("rt", [None, "bf16", "f32"])
def test_rmsnorm_odd_widths(M, K, rt):
    rng = np.random.default_rng(M * 31 + K)
    for xt, wt in (("bf16", "bf16"), ("f32", "f16"), ("f16", None)):
        check_norm(rand(rng, (M, K), xt), None if wt is None else rand(rng, (K,), wt),
                   None if rt is None else rand(rng, (M, K), rt), "bf16")


def test_rmsnorm_extremes():
    rng = np.random.default_rng(2)
    x = rand(rng, (8, 256), "f32")
    x[0] = 0.0
    x[1] *= 1e-30                                               # squares underflow in fp32
    x[2] *= 1e25                                                # and overflow
    x[3, 7], x[4, 9], x[5, 0] = float("nan"), float("inf"), -float("inf")
    y, _, _ = q.qmx_rmsnorm(x, eps=1e-5)
    want, _ = R.rmsnorm(f32(x), eps=1e-5)
    got = y.double().cpu().numpy()
    fine = [0, 1, 2, 6, 7]
    assert (np.abs(got[fine] - want[fine]) <= np.abs(want[fine]) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133).all()
    assert np.isnan(got[3]).all() and np.isnan(got[4, 9]) and np.isnan(got[5, 0]) and not got[4, :9].any()
    for fmt, bad in (("mxfp4", 255), ("q8", None)):
        c, s, _ = q.qmx_rmsnorm(x, fmt=fmt)
        v = q.qmx_dequantize(c, s, fmt, torch.float32).cpu().numpy()
        assert np.isnan(v[3]).all() and np.isnan(v[4, :32]).all() and not v[4, 32:].any()
        assert np.isfinite(v[fine]).all()


def test_rmsnorm_in_place_residual_and_given_outputs():
    rng = np.random.default_rng(4)
    x, w, r = rand(rng, (5, 320), "f32"), rand(rng, (320,), "bf16"), rand(rng, (5, 320), "bf16")
    y0, s0, h0 = q.qmx_rmsnorm(x, w, residual=r, fmt="mxfp4")
    keep = r.clone()
    y, s = torch.empty_like(y0), torch.empty_like(s0)
    got = q.qmx_rmsnorm(x, w, residual=r, fmt="mxfp4", y=y, y_scales=s, residual_out=r)
    assert got[0] is y and got[1] is s and got[2] is r
    assert torch.equal(y, y0) and torch.equal(s, s0) and torch.equal(r, h0) and not torch.equal(r, keep)


@pytest.mark.parametrize("fmt", ["mxfp4", "q8"])
@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (4, 2880), (2, 5, 544), (1000, 32), (130, 4128), (64,)])
def test_quantize_and_back(shape, xt, fmt):
    rng = np.random.default_rng(7)
    x = rand(rng, shape, xt, 0.3)
    c, s = q.qmx_quantize(x, fmt)
    check_blocks(fmt, c, s, f32(x))
    want = R.values(c.cpu().numpy(), s.cpu().numpy()) if fmt == "mxfp4" else \
        R.q8_values(c.cpu().numpy(), s.cpu().numpy())
    for t in TYPES.values():
        got = q.qmx_dequantize(c, s, fmt, t)
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(t))


@pytest.mark.parametrize("fmt", ["mxfp4", "q8"])
def test_quantize_edges(fmt):
    """Every rounding border, every power of two, zeros, subnormal numbers and
    blocks with NaN or infinities."""
    rng = np.random.default_rng(9)
    rows = []
    for top in (6.0, 6.99, 7.0, 7.01, 4.0, 1.75, 1.7499999):
        borders = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5])
        near = np.concatenate([borders, np.nextafter(borders, 9, dtype=np.float32),
                               np.nextafter(borders, -9, dtype=np.float32)])
        rows.append(np.concatenate([[top], near, -near])[:32])
    for e in range(-149, 128):
        rows.append(np.ldexp(rng.uniform(1, 2, 32), e - rng.integers(0, 4, 32)))
    rows.append(np.zeros(32))
    rows.append(-np.zeros(32))
    for v in (np.nan, np.inf, -np.inf):
        r = rng.standard_normal(32)
        r[rng.integers(32)] = v
        rows.append(r)
    with np.errstate(over="ignore"):
        x = np.stack(rows).astype(np.float32)
    x = x[~np.isinf(x).any(1) | (np.arange(len(x)) >= len(x) - 3)]
    c, s = q.qmx_quantize(torch.from_numpy(x).cuda(), fmt)
    check_blocks(fmt, c, s, x)


def test_dequantize_every_code_and_scale():
    codes = np.arange(256, dtype=np.uint8)
    c = np.tile(codes.reshape(16, 16), (256, 1))                # 16 blocks hold every byte; once per scale
    s = np.repeat(codes, 16)[:, None]
    got = q.qmx_dequantize(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), "mxfp4", torch.float32)
    with np.errstate(over="ignore"):
        want = R.values(c, s).astype(np.float32)
    assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


def test_quantize_past_32_bit_offsets():
    rows, K = 270000, 16384                                     # 4.4e9 values
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    at = [0, 131071, 131072, 262144, rows - 1]
    vals = rand(rng, (len(at), K), "bf16")
    for i, r in enumerate(at):
        x[r] = vals[i]
    c, s = q.qmx_quantize(x)
    for i, r in enumerate(at):
        check_blocks("mxfp4", c[r], s[r], f32(vals[i]))
    assert not c[1:131071].any() and not s[262145:rows - 1].any()
    del x
    y = q.qmx_dequantize(c, s)
    for i, r in enumerate(at):
        assert torch.equal(y[r].float().cpu(), torch.from_numpy(R.values(c[r].cpu().numpy(), s[r].cpu().numpy())).float())
    assert not y[200000].any()


def check_router(l, top_k, **kw):
    ids, w = q.qmx_router(l, top_k, **kw)
    x = f32(l).astype(np.float64)
    want_ids, want = R.router(x, top_k, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    live = np.where(np.isfinite(x), x, 0.0)
    far = np.abs(live).max() + (live.max() - live.min())
    tol = np.abs(want) * (far + 2 * min(l.shape[1], 64) + 16) * 2.0 ** -22 + 2.0 ** -140
    got = w.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / np.maximum(np.abs(want), 1e-30)).max()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("M,E,top_k", [(1, 32, 4), (1, 1, 1), (5, 64, 2), (7, 65, 16), (3, 128, 8), (9, 256, 8),
                                       (2, 300, 3), (33, 512, 10), (2, 1024, 16), (130, 17, 16), (4, 4, 4)])
def test_router(M, E, top_k, scoring, normalize):
    rng = np.random.default_rng(M + E)
    for t in ("f32", "bf16"):
        check_router(rand(rng, (M, E), t, 2.0), top_k, scoring=scoring, normalize=normalize)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_router_ties_masks_and_far_logits(scoring, normalize):
    rng = np.random.default_rng(1)
    for E in (8, 100, 1000):
        l = torch.from_numpy(rng.integers(-2, 3, (40, E)).astype(np.float32)).cuda()   # many ties
        check_router(l, min(8, E), scoring=scoring, normalize=normalize, scale=2.5)
        l[:, ::2] = -float("inf")
        l[3], l[4, 1:], l[5] = -float("inf"), float("nan"), float("nan")
        l[6] = 0.0
        l[6, 0], l[6, 1] = -0.0, 0.0                            # equal: the lower index first
        check_router(l, min(8, E), scoring=scoring, normalize=normalize)
    l = rand(rng, (6, 64), "f32", 1.0) - 300.0                  # every sigmoid underflows in fp32
    check_router(l, 4, scoring=scoring, normalize=True)
    l = rand(rng, (6, 64), "f32", 40.0)
    check_router(l, 8, scoring=scoring, normalize=normalize)
    l[:, 3] = torch.finfo(torch.float32).min                    # the lowest finite logit is no mask
    check_router(l[:, :8].contiguous(), 8, scoring="sigmoid", normalize=False)


def test_calls_repeat_bit_for_bit_and_replay_in_a_graph():
    rng = np.random.default_rng(11)
    x, w, r = rand(rng, (40, 2880), "f32"), rand(rng, (2880,), "bf16"), rand(rng, (40, 2880), "bf16")
    l = rand(rng, (40, 32), "bf16")
    out = {}

    def call():
        out["n"] = q.qmx_rmsnorm(x, w, residual=r, fmt="mxfp4")
        out["r"] = q.qmx_router(l, 4)
        out["q"] = q.qmx_quantize(x, "q8")
        out["d"] = (q.qmx_dequantize(*out["n"][:2]), q.qmx_dequantize(*out["q"], "q8"))

    call()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    held = dict(out)
    for k in range(4):
        x.copy_(rand(rng, (40, 2880), "f32"))
        l.copy_(rand(rng, (40, 32), "bf16"))
        g.replay()
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        for name in out:
            for a, b in zip(held[name], out[name]):
                assert torch.equal(a, b), (k, name)


def test_layer_on_another_stream():
    rng = np.random.default_rng(12)
    x = rand(rng, (9, 512), "f32")
    want = q.qmx_quantize(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = q.qmx_quantize(x, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("M", [1, 4, 37, 200])
def test_moe_layer(M):
    """norm -> router -> gate/up -> quantize -> down + combine, as a layer runs
    them, each step from the step before; the products' inputs are the GPU's
    own codes, so every step is held to its own tolerance."""
    rng = np.random.default_rng(M)
    K, N, E, top_k = 320, 160, 8, 2
    h = rand(rng, (M, K), "bf16", 3.0)
    x, w = rand(rng, (M, K), "f32"), rand(rng, (K,), "bf16")
    router_w = rand(rng, (E, K), "f32", 0.2)
    gw, uw, dw = (q.qmx_quantize(rand(rng, s, "bf16", 0.1)) for s in ((E, N, K), (E, N, K), (E, K, N)))

    a, a_s, h2 = q.qmx_rmsnorm(x, w, residual=h, fmt="mxfp4")
    logits = q.qmx_dequantize(a, a_s, dtype=torch.float32) @ router_w.t()
    ids, rw = q.qmx_router(logits, top_k)
    g = q.qmv_gather_moe_swiglu("mxfp4", *gw, *uw, ids, a, a_s)
    b, b_s = q.qmx_quantize(g)
    y = q.qmv_gather_moe_combine("mxfp4", *dw, ids, rw, b, b_s)

    n, h32 = R.rmsnorm(f32(x), f32(w), f32(h))
    assert torch.equal(h2.cpu(), torch.from_numpy(h32).bfloat16())
    check_blocks("mxfp4", a, a_s, n.astype(np.float32))
    check_router(logits, top_k)
    av, wv = R.values(a.cpu().numpy(), a_s.cpu().numpy()), [R.values(c.cpu().numpy(), s.cpu().numpy()) for c, s in (gw, uw, dw)]
    i = ids.cpu().numpy()
    gate, Ag = R.gather(i, wv[0], av, False)
    up, Au = R.gather(i, wv[1], av, False)
    silu = gate / (1 + np.exp(-gate))
    U = 2.0 ** -23
    tol = 1.1 * K * U * Ag * (np.abs(up) + K * U * Au) + np.abs(silu) * K * U * Au + (np.abs(gate) + 8) * 2 * U * np.abs(silu * up)
    assert (np.abs(f32(g) - silu * up) <= tol).all()
    check_blocks("mxfp4", b, b_s, f32(g))
    d, A = R.gather(i, wv[2], R.values(b.cpu().numpy(), b_s.cpu().numpy()), True)
    r = rw.double().cpu().numpy()[:, :, None]
    assert (np.abs(f32(y) - (r * d).sum(1)) <= ((N + 2 * top_k) * U * np.abs(r) * A).sum(1)).all()
