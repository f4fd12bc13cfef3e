"""Every kernel of the MXFP4 x MXFP4 products, each case with the kernel that
it is meant for (needs an MI355X; test_mx4_launches.py checks on the host that
each case reaches its kernel, so that no case loses its point when the choice
between the kernels changes).

All inputs have exact sums (mx4_exact.py): products are compared bit for bit.
Gate/up and route weights say their own bounds.
"""
import pytest
import torch

import bit_block_quantized_amd as q
import mx4_exact as X

pytestmark = pytest.mark.gpu

FEW, FEW_GU, FEW_COMB = "qmv_mx4_few_kernel<0>", "qmv_mx4_few_kernel<1>", "qmv_mx4_few_kernel<2>"
TILE64, GU64 = "qmv_mx4_tile_kernel<0, 64>", "qmv_mx4_tile_kernel<1, 64>"
TILE128, GU128 = "qmv_mx4_tile_kernel<0, 128>", "qmv_mx4_tile_kernel<1, 128>"
WIDE = "qmv_mx4_wide_kernel"


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def equal(y, want, what):
    """Bit for bit the 64-bit values (-0 and 0 are equal; NaN where they are NaN)."""
    assert y.shape == want.shape, what
    y = y.double()
    ok = (y == want) | (y.isnan() & want.isnan())
    assert ok.all(), (what, int((~ok).sum()), torch.nonzero(~ok)[:3].tolist(), y[~ok][:3].tolist(), want[~ok][:3].tolist())


def nan_like(*shape):
    return torch.full(shape, float("nan"), device="cuda")


# ------------------------------------------------------------ exact products
# (kernel, M, N, K): tails of K in the last unit and slab, the longest rows
DENSE = [(FEW, 3, 100, 16384), (FEW, 16, 200, 7168), (FEW, 20, 90, 16352),
         (TILE64, 17, 6200, 16384), (TILE64, 70, 2900, 7168), (TILE64, 64, 3100, 16352), (TILE64, 33, 4100, 544),
         (WIDE, 257, 8300, 7168), (WIDE, 1030, 3400, 16352), (WIDE, 300, 8300, 16384), (WIDE, 2050, 2100, 2880),
         (WIDE, 4100, 1030, 32), (WIDE, 2300, 7500, 288), (TILE64, 8192, 200, 96), (FEW, 8192, 16, 64)]


@pytest.mark.parametrize("kernel,M,N,K", DENSE)
def test_dense(kernel, M, N, K):
    g = gen(M + N + K)
    wc, ws = X.codes(g, (N,), K, X.W_LO)
    xc, xs = X.codes(g, (M,), K, X.X_LO)
    want, A = X.dense(wc, ws, X.values(xc, xs))
    X.held(A)
    equal(q.qmv_dense("mxfp4", wc, ws, xc, xs, y=nan_like(M, N)), want, (kernel, M, N, K))


# (kernel, M, E, top_k, N, K)
GATHER = [(FEW, 4, 8, 4, 100, 7168), (FEW, 40, 8, 2, 130, 7168), (FEW, 33, 1000, 2, 33, 16384),
          (TILE64, 60, 40, 2, 300, 7168), (TILE64, 60, 5, 2, 300, 16384), (TILE64, 100, 40, 2, 301, 16352),
          (TILE64, 4, 40, 8, 1000, 544), (TILE64, 300, 3, 2, 400, 3616),
          (TILE128, 150, 4, 4, 96, 3584), (TILE128, 300, 8, 4, 70, 3552), (TILE128, 700, 3, 2, 200, 1024)]
# as many pairs as a call may have, and as many as the few-vector kernel takes
GATHER += [(TILE64, 512, 1023, 16, 33, 96), (TILE128, 512, 100, 16, 33, 96), (TILE128, 8192, 5, 1, 20, 64),
           (FEW, 112, 1023, 16, 16, 96), (FEW, 1792, 40, 1, 9, 64)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("kernel,M,E,top_k,N,K", GATHER)
def test_gather(kernel, M, E, top_k, N, K, per_slot):
    g = gen(M + N + K)
    wc, ws = X.codes(g, (E, N), K, X.W_LO)
    xc, xs = X.codes(g, (M, top_k) if per_slot else (M,), K, X.X_LO)
    for skew in (False, True):
        ids = X.make_ids(g, M, top_k, E, skew=skew)
        want, A = X.gather(ids, wc, ws, X.values(xc, xs))
        X.held(A)
        y = q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs, y=nan_like(M, top_k, N))
        equal(y, want, (kernel, M, E, top_k, N, K, per_slot, skew))


SWIGLU = [(FEW_GU, 4, 8, 4, 100, 7168), (FEW_GU, 40, 8, 2, 70, 2880), (FEW_GU, 1, 1500, 15, 50, 15392),
          (GU64, 60, 40, 2, 300, 7168), (GU64, 60, 5, 2, 200, 16384), (GU64, 100, 40, 2, 201, 544),
          (GU128, 150, 4, 4, 96, 3584), (GU128, 300, 8, 4, 70, 3552), (GU128, 700, 3, 2, 100, 288)]


def check_swiglu(y, g, u, what):
    """g and u are exact, so y = g / (1 + e^-g) u has only its own roundings:
    e^-g is 2^(-g log2 e), whose argument is off by |g| 2^-23 of e^-g at most
    and whose result by 2 steps, a sum, a quotient and a product by half a step
    each; |g| < 80 keeps e^-g and the quotient inside fp32's normal range."""
    assert g.abs().max() < 80
    want = g / (1 + torch.exp(-g)) * u
    tol = (g.abs() + 8) * 2.0 ** -22 * want.abs() + 2.0 ** -126
    bad = ~((y.double() - want).abs() <= tol) & ~(y.isnan() & want.isnan())
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(), y[bad][:3].tolist(), want[bad][:3].tolist())


def swiglu_bytes(K):
    """Lowest scale bytes of the weights and of the vectors that keep |g| well below 80: a product of two codes is
    about 8 in root mean square, a sum of K of them 8 sqrt(K)."""
    x = 127
    w = 127 - 3 - (K.bit_length() + 1) // 2
    return w, x


@pytest.mark.parametrize("kernel,M,E,top_k,N,K", SWIGLU)
def test_swiglu(kernel, M, E, top_k, N, K):
    g = gen(M + N + K)
    w_lo, x_lo = swiglu_bytes(K)
    gc, gs = X.codes(g, (E, N), K, w_lo)
    uc, us = X.codes(g, (E, N), K, w_lo)
    xc, xs = X.codes(g, (M,), K, x_lo)
    for skew in (False, True):
        ids = X.make_ids(g, M, top_k, E, skew=skew)
        x = X.values(xc, xs)
        (gate, Ag), (up, Au) = X.gather(ids, gc, gs, x), X.gather(ids, uc, us, x)
        X.held(torch.maximum(Ag, Au), w_lo, x_lo)
        y = q.qmv_gather_moe_swiglu("mxfp4", gc, gs, uc, us, ids, xc, xs, y=nan_like(M, top_k, N))
        check_swiglu(y, gate, up, (kernel, M, E, top_k, N, K, skew))


COMBINE = [(FEW_COMB, 4, 8, 8, 100, 16384), (FEW_COMB, 3, 40, 16, 33, 7168), (FEW_COMB, 1, 300, 4, 70, 16352),
           (FEW, 9, 8, 4, 100, 7168), (TILE64, 60, 40, 2, 300, 7168), (TILE128, 200, 16, 4, 36, 3584)]


@pytest.mark.parametrize("kernel,M,E,top_k,N,K", COMBINE)
def test_combine(kernel, M, E, top_k, N, K):
    """Route weights 1/2, 1, 2 and -1: the weighted sums are whole numbers of 1/8 of the smallest step."""
    g = gen(M + N + K)
    wc, ws = X.codes(g, (E, N), K, X.W_LO, 2)
    xc, xs = X.codes(g, (M, top_k), K, X.X_LO, 1)
    ids = X.make_ids(g, M, top_k, E)
    rw = torch.tensor([0.5, 1.0, 2.0, -1.0], device="cuda")[torch.randint(0, 4, (M, top_k), device="cuda", generator=g)]
    rows, A = X.gather(ids, wc, ws, X.values(xc, xs))
    X.held((rw.abs().double()[:, :, None] * A).sum(1), parts=8)
    want = (rw.double()[:, :, None] * rows).sum(1)
    args = ("mxfp4", wc, ws, ids, rw, xc)
    equal(q.qmv_gather_moe_combine(*args, xs, y=nan_like(M, N)), want, (kernel, M, E, top_k, N, K))
    y = nan_like(M, N)
    q.qmv_gather_moe_combine_noalloc(*args, y, x_scales=xs)
    equal(y, want, (kernel, M, E, top_k, N, K, "no allocation"))


# ------------------------------------------------- runs of several row tiles
# (kernel, entry, M, E, top_k, N, K): calls of so many tiles that a workgroup
# takes two or more of an item one after another; runs that end short, rows of
# every remainder by 4, one and several slabs of K
RUNS = [(TILE64, "gather", 200, 128, 2, 8050, 96), (TILE64, "gather", 200, 128, 2, 8060, 544),
        (TILE64, "gather", 500, 1000, 2, 2600, 32), (TILE128, "gather", 512, 16, 2, 43801, 64),
        (TILE128, "gather", 512, 16, 2, 43804, 1056), (GU64, "swiglu", 100, 100, 2, 5151, 64),
        (GU64, "swiglu", 100, 100, 2, 5152, 544), (GU128, "swiglu", 400, 8, 2, 37641, 96),
        (GU128, "swiglu", 400, 8, 2, 37644, 544), (TILE64, "dense", 100, 1, 1, 524901, 32),
        (TILE64, "dense", 128, 1, 1, 524904, 96)]


@pytest.mark.parametrize("kernel,entry,M,E,top_k,N,K", RUNS)
def test_runs_of_row_tiles(kernel, entry, M, E, top_k, N, K):
    g = gen(M + N + K)
    what = (kernel, entry, M, E, top_k, N, K)
    w_lo, x_lo = swiglu_bytes(K) if entry == "swiglu" else (X.W_LO, X.X_LO)
    lead = (N,) if entry == "dense" else (E, N)
    wc, ws = X.codes(g, lead, K, w_lo)
    xc, xs = X.codes(g, (M,), K, x_lo)
    x = X.values(xc, xs)
    if entry == "dense":
        want, A = X.dense(wc, ws, x)
        X.held(A)
        equal(q.qmv_dense("mxfp4", wc, ws, xc, xs, y=nan_like(M, N)), want, what)
        return
    ids = X.make_ids(g, M, top_k, E)
    rows, A = X.gather(ids, wc, ws, x)
    X.held(A, w_lo, x_lo)
    if entry == "gather":
        equal(q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs, y=nan_like(M, top_k, N)), rows, what)
        return
    uc, us = X.codes(g, lead, K, w_lo)
    up, A = X.gather(ids, uc, us, x)
    X.held(A, w_lo, x_lo)
    y = q.qmv_gather_moe_swiglu("mxfp4", wc, ws, uc, us, ids, xc, xs, y=nan_like(M, top_k, N))
    check_swiglu(y, rows, up, what)


# ----------------------------------------------------------- edges of inputs
# (kernel, M, E, top_k, N): E = 0 is a dense call
EDGES = [(FEW, 3, 0, 1, 70), (FEW, 40, 8, 2, 130), (TILE64, 33, 0, 1, 4101), (TILE64, 60, 40, 2, 300),
         (TILE128, 150, 4, 4, 97), (WIDE, 300, 0, 1, 8301), (WIDE, 1030, 0, 1, 3400)]


def product(E, wc, ws, ids, xc, xs, **kw):
    if E:
        return q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs, **kw)
    return q.qmv_dense("mxfp4", wc, ws, xc, xs, **kw)


def reference(E, wc, ws, ids, xc, xs):
    return X.gather(ids, wc, ws, X.values(xc, xs)) if E else X.dense(wc, ws, X.values(xc, xs))


def edge_inputs(M, E, top_k, N, K, seed, **kw):
    g = gen(seed)
    wc, ws = X.codes(g, (E, N) if E else (N,), K, X.W_LO)
    xc, xs = X.codes(g, (M,), K, X.X_LO)
    return wc, ws, X.make_ids(g, M, top_k, E, **kw) if E else None, xc, xs


@pytest.mark.parametrize("K", [288, 1056])
@pytest.mark.parametrize("kernel,M,E,top_k,N", EDGES)
def test_nan_stays_in_its_row_and_vector(kernel, M, E, top_k, N, K):
    wc, ws, ids, xc, xs = edge_inputs(M, E, top_k, N, K, M)
    want, A = reference(E, wc, ws, ids, xc, xs)
    X.held(A)
    w2 = ws[1] if E else ws
    # a row's first, a middle and the last row's last block; a vector's last block and the last vector's first
    for r, b in ((0, 0), (N // 2, 3), (N - 1, K // 32 - 1)):
        w2[r, b] = 255
    xs[M // 2, K // 32 - 1] = 255
    xs[M - 1, 0] = 255
    nan_want, _ = reference(E, wc, ws, ids, xc, xs)
    want = torch.where(nan_want.isnan(), nan_want, want)
    assert want.isnan().any() and not want.isnan().all()
    equal(product(E, wc, ws, ids, xc, xs), want, (kernel, M, E, N, K))


@pytest.mark.parametrize("K", [64, 544])
@pytest.mark.parametrize("kernel,M,E,top_k,N", EDGES)
def test_every_scale_byte(kernel, M, E, top_k, N, K):
    """Row n's blocks have scale byte n % 256 and a vector's blocks one byte:
    2^-127 to 2^127 and NaN reach the instruction unchanged."""
    wc, ws, ids, xc, xs = edge_inputs(M, E, top_k, N, K, M)
    ws[:] = (torch.arange(N, device="cuda") % 256).to(torch.uint8)[:, None]
    for xb in (127, 100, 154):
        xs[:] = xb
        y = product(E, wc, ws, ids, xc, xs).double()
        want, A = reference(E, wc, ws, ids, xc, xs)
        assert (y.isnan() == want.isnan())[~(A >= 2.0 ** 128)].all(), (kernel, xb)
        byte = torch.arange(N, device="cuda") % 256
        # the smallest step of a row's sums; sums of normal numbers are exact
        step = torch.ldexp(torch.ones(N, dtype=torch.float64, device="cuda"), (byte + xb - 254).double()) / 4
        exact = (step >= 2.0 ** -126) & ~(A >= 2.0 ** 128)
        assert (y == want)[exact & ~want.isnan()].all(), (kernel, xb)
        # a sum whose terms pass fp32's largest may be infinite or NaN from there on; where the terms
        # themselves are below its normal range each of them and each partial sum may be flushed (2 K)
        low = (step < 2.0 ** -126).expand_as(y)
        assert ((y - want).abs()[low] <= 2 * K * 2.0 ** -126).all(), (kernel, xb)


@pytest.mark.parametrize("off_w,off_x", [(1, 0), (2, 3), (3, 1), (0, 2)])
@pytest.mark.parametrize("kernel,M,E,top_k,N", EDGES)
def test_scales_start_at_any_byte(kernel, M, E, top_k, N, off_w, off_x):
    K = 1120                                                   # 35 scale bytes a row

    def shifted(a, off):
        buf = torch.full((a.numel() + 16,), 255, dtype=torch.uint8, device="cuda")
        buf[off:off + a.numel()] = a.reshape(-1)
        return buf[off:off + a.numel()].view(a.shape)

    wc, ws, ids, xc, xs = edge_inputs(M, E, top_k, N, K, M + 4 * off_w)
    want, A = reference(E, wc, ws, ids, xc, xs)
    X.held(A)
    equal(product(E, wc, shifted(ws, off_w), ids, xc, shifted(xs, off_x)), want, (kernel, off_w, off_x))


# (kernel, entry, M, E, top_k, N)
SHIFTED = [(FEW_GU, "swiglu", 4, 8, 4, 100), (FEW_GU, "swiglu", 40, 8, 2, 70), (GU64, "swiglu", 60, 40, 2, 301),
           (GU128, "swiglu", 150, 4, 4, 97), (FEW_COMB, "combine", 4, 8, 4, 101)]


@pytest.mark.parametrize("kernel,entry,M,E,top_k,N", SHIFTED)
def test_gate_up_and_combine_scales_start_at_any_byte(kernel, entry, M, E, top_k, N):
    K = 1120
    w_lo, x_lo = swiglu_bytes(K)
    g = gen(M + N)

    def shifted(a, off):
        buf = torch.full((a.numel() + 16,), 255, dtype=torch.uint8, device="cuda")
        buf[off:off + a.numel()] = a.reshape(-1)
        return buf[off:off + a.numel()].view(a.shape)

    (wc, ws), (uc, us) = (X.codes(g, (E, N), K, w_lo) for _ in range(2))
    for offs in ((1, 2, 3), (3, 0, 1), (2, 3, 0)):
        xc, xs = X.codes(g, (M, top_k) if entry == "combine" else (M,), K, x_lo)
        ids = X.make_ids(g, M, top_k, E)
        rows, A = X.gather(ids, wc, ws, X.values(xc, xs))
        X.held(A, w_lo, x_lo)
        ws_, us_, xs_ = (shifted(t, o) for t, o in zip((ws, us, xs), offs))
        if entry == "combine":
            ones = torch.ones(M, top_k, device="cuda")
            X.held(A.sum(1), w_lo, x_lo)
            equal(q.qmv_gather_moe_combine("mxfp4", wc, ws_, ids, ones, xc, xs_), rows.sum(1), (kernel, offs))
        else:
            up, A = X.gather(ids, uc, us, X.values(xc, xs))
            X.held(A, w_lo, x_lo)
            check_swiglu(q.qmv_gather_moe_swiglu("mxfp4", wc, ws_, uc, us_, ids, xc, xs_), rows, up, (kernel, offs))


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("kernel,M,E,top_k,N", EDGES)
def test_rows_around_the_output_stay(kernel, M, E, top_k, N, at):
    """y from its buffer's element 64 + at on (16-byte aligned and not)."""
    wc, ws, ids, xc, xs = edge_inputs(M, E, top_k, N, 96, M)
    want, A = reference(E, wc, ws, ids, xc, xs)
    n, o = want.numel(), 64 + at
    buf = torch.full((n + 1024,), 7.0, device="cuda")
    equal(product(E, wc, ws, ids, xc, xs, y=buf[o:o + n].view(want.shape)), want, (kernel, at))
    assert (buf[:o] == 7.0).all() and (buf[o + n:] == 7.0).all()


# (kernel, entry, M, E, top_k, N): more than 64 pairs, none of them with an expert
EMPTY = [(FEW, "gather", 40, 8, 2, 130), (FEW, "gather", 70, 1000, 1, 33), (TILE64, "gather", 60, 40, 2, 301),
         (TILE128, "gather", 150, 4, 4, 96), (FEW_GU, "swiglu", 40, 8, 2, 70), (GU64, "swiglu", 60, 40, 2, 301),
         (GU128, "swiglu", 150, 4, 4, 96), (FEW, "combine", 40, 8, 2, 130), (TILE64, "combine", 60, 40, 2, 301)]


@pytest.mark.parametrize("kernel,entry,M,E,top_k,N", EMPTY)
def test_no_pair_has_an_expert(kernel, entry, M, E, top_k, N):
    K = 544
    g = gen(M)
    w = X.codes(g, (E, N), K, X.W_LO)
    xc, xs = X.codes(g, (M,), K, X.X_LO)
    xs[:] = 255                                                # nothing of the vectors reaches the zeros
    for bad in (-1, E, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((M, top_k), bad, dtype=torch.int32, device="cuda")
        out = nan_like(*((M, N) if entry == "combine" else (M, top_k, N)))
        if entry == "gather":
            q.qmv_gather_moe("mxfp4", *w, ids, xc, xs, y=out)
        elif entry == "swiglu":
            q.qmv_gather_moe_swiglu("mxfp4", *w, *w, ids, xc, xs, y=out)
        else:
            q.qmv_gather_moe_combine("mxfp4", *w, ids, torch.ones(M, top_k, device="cuda"), xc, xs, y=out)
        assert (out == 0).all(), (kernel, bad)


# (kernel, entry, M, E, top_k, N, K): codes past 2^32 bytes (few: past 2^31)
FAR = [(TILE64, "gather", 60, 1000, 2, 1024, 9216), (GU64, "swiglu", 60, 1000, 2, 1024, 9216),
       (FEW, "gather", 33, 1023, 2, 420, 16384)]


@pytest.mark.parametrize("kernel,entry,M,E,top_k,N,K", FAR)
def test_far_experts(kernel, entry, M, E, top_k, N, K):
    g = gen(K)
    w_lo, x_lo = swiglu_bytes(K) if entry == "swiglu" else (X.W_LO, X.X_LO)
    used = (E - 1, E // 2)
    wc = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N, K // 32), 255, dtype=torch.uint8, device="cuda")
    c, s = X.codes(g, (2, N), K, w_lo)
    for i, e in enumerate(used):
        wc[e], ws[e] = c[i], s[i]
    xc, xs = X.codes(g, (M,), K, x_lo)
    small = torch.randint(0, 2, (M, top_k), device="cuda", generator=g)
    ids = torch.tensor(used, device="cuda")[small].int()
    want, A = X.gather(small, c, s, X.values(xc, xs))
    X.held(A, w_lo, x_lo)
    if entry == "gather":
        equal(q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs), want, kernel)
    else:
        check_swiglu(q.qmv_gather_moe_swiglu("mxfp4", wc, ws, wc, ws, ids, xc, xs), want, want, kernel)
