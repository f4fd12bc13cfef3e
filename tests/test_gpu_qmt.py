"""Norm and rotation of heads and log probabilities (include/qmt.h) against the
64-bit forms of f8_ref.py, and a decode step of them with the e4m3 products
(needs an MI355X).

Tolerances.  A head's normed values are formed in 64 bits and rounded to fp32
(2^-24 each); the rotation is two products and a sum in fp32 (2^-24 each of
|a cos| + |b sin|), and the output's rounding is half a step.  A log
probability's exponentials are fp32: the argument's two roundings |l - m|
2^-23, 2 ulp of the function; the sum's relative error is then at most that of
its terms, weighted by their size (where e^-z z is at most 1/e, so 2^-23 of the
terms in all): 8 2^-24 of log s's change, and the output's rounding to fp32.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import f8_ref as F

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def values(rng, shape, t, spread=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * spread).astype(np.float32)).to(TYPES[t]).cuda()


def host(t):
    return t.double().cpu().numpy()


def table(rng, P, R):
    a = rng.uniform(-np.pi, np.pi, (P, R // 2))
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def check_qk(rng, M, H, Hk, D, R, rest, xt, yt, wt, style, P=50, x=None, pos=None, eps=1e-5):
    x = values(rng, (M, (H + Hk) * D + rest), xt, 3.0) if x is None else x
    tb = table(rng, P, R)
    pos = rng.integers(0, P, M).astype(np.int32) if pos is None else pos
    qw, kw = (None, None) if wt is None else (values(rng, (D,), wt), values(rng, (D,), wt))
    n = M * (H + Hk) * D
    buf = torch.full((n + 64,), 5.0, dtype=TYPES[yt], device="cuda")
    qo, ko = buf[32:32 + M * H * D].view(M, H, D), buf[32 + M * H * D:32 + n].view(M, Hk, D)
    got = q.qmt_qk_norm_rope(x, H, Hk, D, torch.from_numpy(tb).cuda(), torch.from_numpy(pos).cuda(), qw, kw, eps=eps,
                             style=style, dtype=TYPES[yt], q=qo, k=ko if Hk else None)
    assert (buf[:32] == 5.0).all() and (buf[32 + n:] == 5.0).all()
    want = F.qk_norm_rope(host(x), H, Hk, D, tb, pos, None if qw is None else host(qw), None if kw is None else host(kw),
                          eps, style)
    # |a cos| + |b sin| of each output: the same with magnitudes only
    mag = F.qk_norm_rope(np.abs(host(x)), H, Hk, D, np.concatenate([np.abs(tb[:, :R // 2]), -np.abs(tb[:, R // 2:])], 1),
                         pos, None if qw is None else np.abs(host(qw)), None if kw is None else np.abs(host(kw)), eps, style)
    for g, w, m, heads in zip(got, want, mag, (H, Hk)):
        if heads == 0:
            assert g is None
            continue
        # the first of a pair's magnitudes is a |cos| + b |sin|; the second's differs in sign
        hi = np.abs(m)
        if R:
            a, b = (slice(0, R // 2), slice(R // 2, R)) if style == "half" else (slice(0, R, 2), slice(1, R, 2))
            both = np.maximum(np.abs(w[..., a]), np.abs(w[..., b])) + hi[..., a]
            hi[..., a] = hi[..., b] = 2 * both                  # (at least either output's own)
        tol = HALF_STEP[yt] * np.abs(w) + 4 * 2.0 ** -24 * hi + 2.0 ** -24 * np.abs(w) + (2.0 ** -24 if yt == "f16" else 2.0 ** -133)
        assert (np.abs(host(g) - w) <= tol).all(), (np.abs(host(g) - w) / np.maximum(tol, 1e-300)).max()
    return got


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("M,H,Hk,D,R,rest", [(1, 1, 1, 8, 8, 0), (1, 64, 8, 64, 64, 512), (3, 4, 2, 128, 128, 256),
                                             (5, 3, 1, 80, 40, 24), (2, 5, 5, 96, 96, 4), (7, 2, 1, 256, 64, 0),
                                             (4, 3, 2, 192, 128, 8), (2, 2, 1, 512, 512, 0), (3, 2, 2, 32, 16, 0),
                                             (2, 4, 0, 64, 64, 0), (2, 3, 1, 72, 8, 12), (3, 1, 1, 264, 8, 0)])
def test_qk_shapes(M, H, Hk, D, R, rest, style):
    rng = np.random.default_rng(M + D + R)
    check_qk(rng, M, H, Hk, D, R, rest, "f32", "bf16", "bf16", style)


@pytest.mark.parametrize("xt", list(TYPES))
@pytest.mark.parametrize("yt", list(TYPES))
@pytest.mark.parametrize("wt", [None, "f32", "bf16", "f16"])
def test_qk_types(xt, yt, wt):
    rng = np.random.default_rng(7)
    check_qk(rng, 5, 6, 2, 64, 32, 64, xt, yt, wt, "half")
    check_qk(rng, 5, 6, 2, 64, 64, 64, xt, yt, wt, "pairs")


@pytest.mark.parametrize("D,R,style", [(128, 128, "half"), (64, 32, "half"), (80, 80, "pairs"), (256, 256, "half"), (32, 32, "pairs")])
def test_qk_many_heads(D, R, style):
    """Enough heads that a group of lanes takes four of a token, with a head count that four does not divide."""
    rng = np.random.default_rng(D)
    check_qk(rng, 1700, 7, 3, D, R, 40, "bf16", "bf16", "bf16", style)


def test_qk_positions_outside_and_odd_inputs():
    rng = np.random.default_rng(8)
    pos = np.array([0, -1, 49, 50, 2 ** 31 - 1, -2 ** 31, 7], np.int32)
    got = check_qk(rng, 7, 4, 2, 64, 64, 0, "f32", "f32", "f32", "half", pos=pos)
    for g in got:
        assert not g[[1, 3, 4, 5]].any() and g[[0, 2, 6]].any()
    x = values(rng, (4, 3 * 64), "f32")
    x[0] = 0.0
    x[1] *= 1e-25                                               # squares underflow in fp32
    x[2] *= 1e25                                                # and overflow
    check_qk(rng, 4, 2, 1, 64, 64, 0, "f32", "f32", None, "half", x=x)
    x[3, 5] = float("nan")
    tb = torch.from_numpy(table(rng, 9, 64)).cuda()
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    qo, ko = q.qmt_qk_norm_rope(x, 2, 1, 64, tb, p)
    assert qo[3, 0].isnan().all() and qo[:3].isfinite().all() and qo[3, 1].isfinite().all() and ko.isfinite().all()
    p[3] = -1                                                   # a padded row's values do not matter
    qo, ko = q.qmt_qk_norm_rope(x, 2, 1, 64, tb, p)
    assert not qo[3].any() and qo.isfinite().all()


# ------------------------------------------------------- log probabilities

def check_logprobs(l, t, top_k):
    M, V = l.shape
    x = host(l)
    got = q.qmt_logprobs(l, torch.from_numpy(t).cuda(), top_k)
    lp, H, ids, top = F.logprobs(x, t, top_k)
    assert got[0].shape == got[1].shape == (M,)
    if top_k:
        assert np.array_equal(got[2].cpu().numpy(), ids)
    else:
        assert got[2] is None and got[3] is None
    E = 2.0 ** -24
    live = np.where(np.isfinite(x), x, -np.inf)
    m = live.max(1, initial=-np.inf)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(np.isfinite(live) & np.isfinite(m)[:, None], live - m[:, None], -np.inf)
        e = np.exp(z)
        others = np.maximum(e.sum(1) - 1.0, 0.0)
        # log(1 + others): others is off by 16 roundings of its own (and |z| <= 40 where it counts), a term of 2^-24 z
        zs = np.where(e > 0, e * np.abs(np.where(e > 0, z, 0)), 0).sum(1)
        # the sum itself is fp64 and starts from the largest's 1: each of at most V / 256 + 20 additions to the
        # partial sum that holds it loses up to 2^-53 of 1 + others, which moves the logarithm by as much
        dlog = (16 * others + 2 * zs) * E / np.maximum(1 + others, 1) + (V / 256 + 20) * 2.0 ** -53
    for g, w in ((host(got[0])[:, None], lp[:, None]), (host(got[3]) if top_k else None, top)):
        if g is None:
            continue
        tol = dlog[:, None] + E * np.abs(np.where(np.isfinite(w), w, 0)) + 2.0 ** -149
        with np.errstate(invalid="ignore"):
            ok = (g == w) | (np.isnan(g) & np.isnan(w)) | (np.abs(g - w) <= tol)
        assert ok.all(), (g[~ok], w[~ok])
    # the entropy: log s, and a sum of e z with 16 roundings of each term and its argument's
    zz = np.where(e > 0, e * np.where(e > 0, z, 0) ** 2, 0).sum(1)
    tolH = 2 * dlog + (20 * zs + 2 * zz + 16 * np.abs(np.where(np.isfinite(H), H, 0))) * E / np.maximum(1 + others, 1) + E * np.abs(H) + 1e-44
    g = host(got[1])
    with np.errstate(invalid="ignore"):
        ok = (g == H) | (np.isnan(g) & np.isnan(H)) | (np.abs(g - H) <= tolH)
    assert ok.all(), (g[~ok], H[~ok], tolH[~ok])
    return got


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("M,V,top_k", [(1, 1, 1), (1, 5, 8), (2, 37, 20), (3, 2048, 5), (1, 2047, 32), (4, 2042, 1),
                                       (5, 4099, 7), (1, 20000, 20), (2, 131071, 5), (1, 201088, 20), (9, 3001, 0),
                                       (33, 513, 32), (700, 1001, 3), (1030, 2051, 6)])
def test_logprobs_shapes(M, V, top_k, t):
    rng = np.random.default_rng(M + V)
    l = values(rng, (M, V), t, 3.0)
    check_logprobs(l, rng.integers(0, V, M).astype(np.int32), top_k)


@pytest.mark.parametrize("M", [2, 1100])
def test_logprobs_masks_ties_and_far_logits(M):
    rng = np.random.default_rng(9)
    V = 5003
    l = torch.from_numpy(rng.integers(-3, 3, (M, V)).astype(np.float32)).cuda()          # many ties
    t = rng.integers(-2, V + 2, M).astype(np.int32)
    t[0] = 2 ** 31 - 1
    check_logprobs(l, t, 32)
    l[:, ::2] = -float("inf")
    l[1, 7:] = float("nan")
    check_logprobs(l, t, 6)
    l[0], l[1] = -float("inf"), 0.0
    l[1, 9], l[1, 4] = -0.0, 0.0                                # equal: the lower index first
    check_logprobs(l, t, 5)
    l[0, 100], l[1, 3] = float("inf"), float("inf")
    check_logprobs(l, t, 3)
    check_logprobs(values(rng, (M, V), "f32", 200.0), t, 4)
    l = values(rng, (M, V), "f32")
    l[:, 4321] += 25.0                                          # a token that is nearly certain
    t[:] = 4321
    got = check_logprobs(l, t, 2)
    assert (got[0] < 0).all()
    l[:, 3] = torch.finfo(torch.float32).min                    # the lowest finite logit is no mask
    l[:, 4:] = -float("inf")
    got = check_logprobs(l, t, 5)
    assert (got[2][:, 3] == 3).all() and (got[2][:, 4] == -1).all()
    l[:, 0] = torch.finfo(torch.float32).max
    check_logprobs(l, t, 3)


@pytest.mark.parametrize("M", [1, 1100])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "late"])
def test_logprobs_orders(M, order):
    """Every logit a new largest one, the largest first, all alike, all the top ones in the last group."""
    V = 70001 if M == 1 else 9001
    l = torch.linspace(-9, 9, V).repeat(M, 1)
    if order == "falling":
        l = l.flip(1)
    elif order == "equal":
        l = torch.full((M, V), 1.5)
    elif order == "late":
        l = torch.zeros(M, V)
        l[:, -40:] = torch.arange(40.0)
    check_logprobs(l.contiguous().cuda(), np.full(M, V - 1, np.int32), 32)


@pytest.mark.parametrize("t", list(TYPES))
def test_logprobs_off_alignment(t):
    """Logits that start at any of their elements (rows of an odd width do, and so may the array)."""
    rng = np.random.default_rng(10)
    M, V = 3, 4001
    flat = values(rng, (M * V + 32,), t)
    for off in range(9):
        check_logprobs(flat[off:off + M * V].view(M, V), rng.integers(0, V, M).astype(np.int32), 4)


def test_logprobs_past_32_bit_offsets():
    M, V = 33000, 131071                                        # 4.3e9 logits
    l = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(11)
    at = [0, 16383, 16384, 32768, M - 1]
    vals = values(rng, (len(at), V), "bf16", 3.0)
    for i, r in enumerate(at):
        l[r] = vals[i]
    t = torch.full((M,), 77, dtype=torch.int32, device="cuda")
    lp, H, ids, top = q.qmt_logprobs(l, t, 3)
    want = q.qmt_logprobs(vals, t[:len(at)].contiguous(), 3)
    for i, r in enumerate(at):
        assert torch.equal(ids[r], want[2][i])
        assert torch.allclose(top[r], want[3][i], rtol=1e-6) and torch.allclose(lp[r], want[0][i], rtol=1e-6)
        assert torch.allclose(H[r], want[1][i], rtol=1e-6)
    rest = torch.ones(M, dtype=torch.bool)
    rest[at] = False
    assert (ids[rest.cuda()] == torch.tensor([0, 1, 2], device="cuda")).all()
    assert torch.allclose(lp[rest.cuda()], torch.full((), -np.log(V), dtype=torch.float32, device="cuda"))


def test_logprobs_optional_outputs_and_workspace():
    rng = np.random.default_rng(12)
    l, t = values(rng, (3, 30000), "f32", 2.0), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    lp, H, ids, top = q.qmt_logprobs(l, t, 4)
    none = q.qmt_logprobs(l)
    assert none[0] is None and torch.equal(none[1], H) and none[2] is None
    need = q.qmt_lib().qmt_logprobs_workspace(3, 30000, 4)
    assert need > 0 and q.qmt_lib().qmt_logprobs_workspace(2000, 30000, 4) == 0
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    o = [torch.empty_like(a) for a in (lp, H, ids, top)]
    got = q.qmt_logprobs(l, t, 4, *o, workspace=ws)
    assert all(a is b for a, b in zip(got, o)) and all(torch.equal(a, b) for a, b in zip(got, (lp, H, ids, top)))
    assert (ws[need:] == 255).all()
    with pytest.raises(ValueError, match="workspace"):
        q.qmt_logprobs(l, t, 4, workspace=ws[:need - 1])


# ------------------------------------------------------------ a decode step

@pytest.mark.parametrize("M", [1, 4, 37, 300])
def test_decode_step(M):
    """norm -> codes -> q/k/v product -> heads; norm -> router -> experts; norm
    -> head product -> log probabilities, each step from the one before and
    held to its own tolerance."""
    rng = np.random.default_rng(M)
    K, D, H, Hk, E, I, top_k, V = 288, 32, 4, 2, 6, 160, 2, 1501
    h = values(rng, (M, K), "bf16", 3.0)
    x, nw = values(rng, (M, K), "f32"), values(rng, (K,), "bf16")
    qkvw, headw = (q.qmt_quantize_weights(values(rng, (n, K), "bf16", 0.1)) for n in ((H + 2 * Hk) * D, V))
    gw, uw, dw = (q.qmt_quantize_weights(values(rng, s, "bf16", 0.1)) for s in ((E, I, K), (E, I, K), (E, K, I)))
    rw_ = values(rng, (E, K), "f32", 0.2)
    tb = torch.from_numpy(table(rng, 64, D)).cuda()
    pos = torch.from_numpy(rng.integers(0, 64, M).astype(np.int32)).cuda()
    tok = torch.from_numpy(rng.integers(0, V, M).astype(np.int32)).cuda()

    def step():
        a, s, h2 = q.qmx_rmsnorm(x, nw, residual=h, fmt="f8")
        qkv = q.qmv_dense("f8", *qkvw, a, s)
        qo, ko = q.qmt_qk_norm_rope(qkv, H, Hk, D, tb, pos)
        ids, w = q.qmx_router(q.qmx_dequantize(a, s, "f8", torch.float32) @ rw_.t(), top_k)
        g = q.qmv_gather_moe_swiglu("f8", *gw, *uw, ids, a, s)
        b, bs = q.qmx_quantize(g, "f8")
        y = q.qmv_gather_moe_combine("f8", *dw, ids, w, b, bs)
        c, cs, _ = q.qmx_rmsnorm(y, nw, residual=h2, fmt="f8")
        logits = q.qmv_dense("f8", *headw, c, cs)
        return [a, s, qkv, qo, ko, ids, w, g, b, bs, y, c, cs, logits, *q.qmt_logprobs(logits, tok, 4)]

    a, s, qkv, qo, ko, ids, w, g, b, bs, y, c, cs, logits, lp, ent, tid, top = out = step()

    def u8(t):
        return t.view(torch.uint8).cpu().numpy()

    def close(got, xv, wv, blocks_k):
        want, A = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        assert (np.abs(host(got) - want) <= (132 + blocks_k) * 2.0 ** -23 * A).all()

    wvals = [F.weight_values(u8(cc), ss.cpu().numpy()) for cc, ss in (qkvw, headw, gw, uw, dw)]
    av, bv, cv = (F.row_values(u8(cc), ss.cpu().numpy()) for cc, ss in ((a, s), (b, bs), (c, cs)))
    close(qkv, av, wvals[0], 3)
    close(logits, cv, wvals[1], 3)
    want = F.qk_norm_rope(host(qkv), H, Hk, D, tb.cpu().numpy(), pos.cpu().numpy())
    for got, w64 in ((qo, want[0]), (ko, want[1])):
        assert (np.abs(host(got) - w64) <= 2.0 ** -8 * np.abs(w64) + 2.0 ** -20).all()
    i = ids.cpu().numpy()
    for t in range(M):
        total = 0.0
        for j in range(top_k):
            e = i[t, j]
            gate, up = wvals[2][e] @ av[t], wvals[3][e] @ av[t]
            want_g = gate / (1 + np.exp(-gate)) * up
            assert np.allclose(host(g)[t, j], want_g, rtol=1e-4, atol=1e-4 * np.abs(want_g).max())
            total = total + host(w)[t, j] * (wvals[4][e] @ bv[t, j])
        assert np.allclose(host(y)[t], total, rtol=1e-4, atol=1e-4 * np.abs(total).max())
    assert np.array_equal(u8(b).reshape(M, top_k, I), F.quantize_rows(g.cpu().numpy())[0])
    check_logprobs(logits, tok.cpu().numpy(), 4)

    # captured: replays with other inputs, eager work between them
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(values(rng, (M, K), "f32"))
        graph.replay()
        torch.cuda.synchronize()
        now = step()
        torch.cuda.synchronize()
        for n, (p, r) in enumerate(zip(held, now)):
            assert torch.equal(p.view(torch.uint8), r.view(torch.uint8)), (k, n)


def test_another_stream_with_its_own_workspace():
    rng = np.random.default_rng(13)
    l, t = values(rng, (2, 60000), "bf16", 2.0), torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    x = values(rng, (6, 256), "f32")
    tb, pos = torch.from_numpy(table(rng, 9, 64)).cuda(), torch.arange(6, dtype=torch.int32, device="cuda")
    want = (*q.qmt_logprobs(l, t, 4), *q.qmt_qk_norm_rope(x, 2, 2, 64, tb, pos), *q.qmt_quantize_weights(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        got.append((*q.qmt_logprobs(l, t, 4, stream=s), *q.qmt_qk_norm_rope(x, 2, 2, 64, tb, pos, stream=s),
                    *q.qmt_quantize_weights(x, stream=s)))
        other = q.qmt_logprobs(l, t, 8)                         # at the same time, on the current one
    s.synchronize()
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(one, want))
    assert torch.equal(other[2][:, :4], want[2])
