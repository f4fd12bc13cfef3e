"""MXFP4 weights x MXFP4 activations (QMV_A_MXFP4) on every product entry
point against the 64-bit forms of mx_ref.py (needs an MI355X).

Tolerance.  The products of two e2m1 values and the powers of two are exact;
only sums round.  A sum of K terms in any order with a unit roundoff of 2^-23
(an adder that truncates) is off by at most K 2^-23 sum |w x| = K 2^-23 A.
Where all scales are one power of two every partial sum is a multiple of 1/4
of it below 2^24 quarters, so the result is exact whatever the order.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import mx_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(rng, lead, K, lo=118, hi=126):
    """Random codes and scale bytes of rows of K values."""
    return (rng.integers(0, 256, lead + (K // 2,), dtype=np.uint8),
            rng.integers(lo, hi + 1, lead + (K // 32,), dtype=np.uint8))


def make_ids(rng, M, top_k, E, holes=True):
    ids = np.stack([rng.permutation(max(E, top_k))[:top_k] % E for _ in range(M)]).astype(np.int32)
    if holes:
        ids[rng.random(ids.shape) < 0.15] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31])
    return ids


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN pattern"
    bad = np.abs(np.nan_to_num(got) - np.nan_to_num(want)) > np.nan_to_num(tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} want {want[bad][0]} tol {tol[bad][0]}")


DENSE = [(1, 1, 32), (1, 17, 64), (1, 2880, 2880), (2, 33, 96), (4, 64, 544), (5, 16, 128), (16, 100, 160),
         (17, 47, 2048), (33, 130, 2880), (64, 96, 512), (65, 31, 1056), (130, 257, 640), (300, 64, 7168),
         (1, 40, 16384), (20, 24, 16384), (513, 513, 1024), (1025, 300, 256)]


# thousands of vectors: tiles of 256 x 256, odd edges and every tail of K; and
# tiles of 128 x 64 with few vectors and many rows
DENSE += [(600, 130, 2880), (520, 70, 32), (777, 260, 544), (512, 256, 1536), (1100, 515, 1056), (2049, 300, 128),
          (4100, 33, 96), (2050, 3600, 32), (1900, 4097, 160), (4100, 2050, 544), (2049, 3850, 1056), (8192, 900, 96),
          (1025, 7001, 512), (17, 12400, 64), (70, 2900, 96), (200, 1100, 544), (96, 2700, 2880), (33, 5000, 1056),
          (1, 33000, 96), (4, 12320, 64), (5, 12320, 64), (16, 13000, 160), (128, 16500, 64), (129, 16400, 96),
          (600, 7000, 544), (700, 7041, 96), (257, 16600, 1056), (4100, 4200, 64), (2300, 7500, 32)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    wc, ws = make(rng, (N,), K)
    xc, xs = make(rng, (M,), K)
    y = q.qmv_dense("mxfp4", dev(wc), dev(ws), dev(xc), dev(xs))
    w, x = R.values(wc, ws), R.values(xc, xs)
    close(y, x @ w.T, K * U * (np.abs(x) @ np.abs(w).T), f"dense {M} {N} {K}")


GATHER = [(1, 1, 1, 5, 32), (1, 32, 4, 70, 2880), (2, 8, 3, 33, 96), (4, 40, 8, 48, 512), (4, 2, 4, 100, 224),
          (5, 64, 2, 50, 160), (6, 3, 2, 65, 544), (37, 8, 4, 130, 288), (64, 200, 4, 20, 128), (100, 4, 4, 96, 1024),
          (16, 1023, 2, 9, 64), (512, 16, 4, 40, 96), (1, 2000, 16, 24, 256), (4, 70000, 2, 3, 32),
          (70, 1, 3, 200, 320), (129, 2, 2, 40, 2880), (65, 1, 1, 130, 3584), (300, 3, 2, 33, 3616),
         (1000, 8, 2, 20, 64), (96, 2, 1, 129, 1504), (4, 30, 8, 1000, 288), (3, 1023, 16, 700, 160),
         (2, 1024, 16, 1000, 64), (9, 5, 3, 2000, 96), (60, 40, 2, 300, 1056)]


@pytest.mark.parametrize("M,E,top_k,N,K", GATHER)
@pytest.mark.parametrize("per_slot", [False, True])
def test_gather(M, E, top_k, N, K, per_slot):
    rng = np.random.default_rng(M + E * 3 + N * 5 + K)
    wc, ws = make(rng, (E, N), K)
    xc, xs = make(rng, (M, top_k) if per_slot else (M,), K)
    ids = make_ids(rng, M, top_k, E)
    out = torch.full((M, top_k, N), float("nan"), device="cuda")
    y = q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs), y=out)
    used = np.unique(ids[(ids >= 0) & (ids < E)])
    remap = {int(e): i for i, e in enumerate(used)}
    small = np.vectorize(lambda e: remap.get(int(e), -1), otypes=[np.int64])(ids)
    w = R.values(wc[used], ws[used])
    want, A = R.gather(small, w, R.values(xc, xs), per_slot)
    close(y, want, K * U * A, f"gather {M} {E} {top_k} {N} {K} {per_slot}")


SWIGLU = [(1, 32, 4, 70, 2880), (4, 6, 2, 33, 96), (5, 64, 2, 50, 160), (37, 8, 4, 130, 288), (150, 4, 4, 96, 1024),
          (3, 300, 8, 17, 64), (2, 1, 1, 5, 32), (300, 2, 2, 70, 544), (129, 2, 2, 40, 2880), (65, 1, 1, 66, 3584),
          (200, 3, 2, 33, 3616), (4, 1100, 16, 3, 16384), (4, 2, 16, 20, 16384), (1, 1500, 15, 5, 15392), (4, 30, 8, 600, 288), (2, 1024, 16, 500, 64),
          (9, 5, 3, 1000, 96)]


@pytest.mark.parametrize("M,E,top_k,N,K", SWIGLU)
def test_swiglu(M, E, top_k, N, K):
    rng = np.random.default_rng(M + E * 3 + N * 5 + K)
    gc, gs = make(rng, (E, N), K, 116, 120)
    uc, us = make(rng, (E, N), K, 116, 120)
    xc, xs = make(rng, (M,), K, 122, 124)
    ids = make_ids(rng, M, top_k, E)
    out = torch.full((M, top_k, N), float("nan"), device="cuda")
    y = q.qmv_gather_moe_swiglu("mxfp4", dev(gc), dev(gs), dev(uc), dev(us), dev(ids), dev(xc), dev(xs), y=out)
    x = R.values(xc, xs)
    g, Ag = R.gather(ids, R.values(gc, gs), x, False)
    u, Au = R.gather(ids, R.values(uc, us), x, False)
    silu = g / (1 + np.exp(-g))
    want = silu * u
    # |silu'| < 1.1; exp of a rounded product is off by |g| 2^-23 of itself, and four roundings more
    tol = 1.1 * K * U * Ag * (np.abs(u) + K * U * Au) + np.abs(silu) * K * U * Au + (np.abs(g) + 8) * 2 * U * np.abs(want)
    close(y, want, tol, f"swiglu {M} {E} {top_k} {N} {K}")


COMBINE = [(1, 8, 4, 70, 2880), (1, 32, 1, 16, 32), (2, 5, 16, 33, 96), (4, 40, 8, 100, 2048), (3, 9, 3, 17, 544),
           (5, 8, 4, 48, 160), (40, 6, 2, 130, 288), (200, 16, 4, 36, 128), (4, 3, 16, 20, 16384)]


@pytest.mark.parametrize("M,E,top_k,N,K", COMBINE)
@pytest.mark.parametrize("per_slot", [True, False])
def test_combine(M, E, top_k, N, K, per_slot):
    rng = np.random.default_rng(M + E * 3 + N * 5 + K)
    wc, ws = make(rng, (E, N), K)
    xc, xs = make(rng, (M, top_k) if per_slot else (M,), K)
    ids = make_ids(rng, M, top_k, E)
    rw = rng.standard_normal((M, top_k)).astype(np.float32)
    args = ("mxfp4", dev(wc), dev(ws), dev(ids), dev(rw), dev(xc))
    out = torch.full((M, N), float("nan"), device="cuda")
    y = q.qmv_gather_moe_combine(*args, dev(xs), y=out)
    g, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), per_slot)
    want = (rw[:, :, None].astype(np.float64) * g).sum(axis=1)
    tol = ((K + 2 * top_k) * U * np.abs(rw[:, :, None]) * A).sum(axis=1)
    close(y, want, tol, f"combine {M} {E} {top_k} {N} {K} {per_slot}")
    z = torch.full((M, N), float("nan"), device="cuda")
    q.qmv_gather_moe_combine_noalloc(*args, z, x_scales=dev(xs))
    assert torch.equal(y, z)


@pytest.mark.parametrize("M", [1, 4, 5, 40])
def test_slots_without_an_expert_hide_nan(M):
    """NaN scales of a slot whose id is outside [0, E), and of the expert that
    no pair has, reach no output."""
    E, top_k, N, K = 6, 4, 50, 544
    rng = np.random.default_rng(M)
    wc, ws = make(rng, (E, N), K)
    ws[0] = 255
    xc, xs = make(rng, (M, top_k), K)
    ids = rng.integers(1, E, (M, top_k)).astype(np.int32)
    for t in range(M):
        ids[t, t % top_k] = (-1, E, -2 ** 31, 2 ** 31 - 1)[t % 4]
        xs[t, t % top_k] = 255
    rw = rng.standard_normal((M, top_k)).astype(np.float32)
    y = q.qmv_gather_moe_combine("mxfp4", dev(wc), dev(ws), dev(ids), dev(rw), dev(xc), dev(xs))
    rows = q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs))
    ws[0], xs[xs == 255] = 120, 120
    g, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), True)
    close(rows, g, K * U * A, f"gather {M}")
    want = (rw[:, :, None].astype(np.float64) * g).sum(axis=1)
    close(y, want, ((K + 2 * top_k) * U * np.abs(rw[:, :, None]) * A).sum(axis=1), f"combine {M}")


@pytest.mark.parametrize("M,N,K", [(1, 48, 2880), (4, 100, 512), (40, 70, 1056), (200, 300, 2048)])
def test_one_scale_is_exact(M, N, K):
    rng = np.random.default_rng(K)
    wc, ws = make(rng, (N,), K, 120, 120)
    xc, xs = make(rng, (M,), K, 130, 130)
    y = q.qmv_dense("mxfp4", dev(wc), dev(ws), dev(xc), dev(xs))
    want = R.values(xc, xs) @ R.values(wc, ws).T
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("M", [1, 40])
def test_every_scale_byte(M):
    """Row n has weight scale n (its opposite in x): 2^-127 to 2^127 and NaN
    reach the instruction unchanged."""
    N, K = 256, 64
    rng = np.random.default_rng(M)
    wc, _ = make(rng, (N,), K)
    ws = np.repeat(np.arange(256, dtype=np.uint8)[:, None], K // 32, axis=1)
    xc, _ = make(rng, (M,), K)
    for xb in (127, 100, 154):
        xs = np.full((M, K // 32), xb, np.uint8)
        y = q.qmv_dense("mxfp4", dev(wc), dev(ws), dev(xc), dev(xs)).cpu().numpy()
        w, x = R.values(wc, ws), R.values(xc, xs)
        with np.errstate(over="ignore", invalid="ignore"):
            want = (x @ w.T).astype(np.float32)
            blocks = np.stack([x[:, b:b + 32] @ w[:, b:b + 32].T for b in range(0, K, 32)])
        # The sum is formed in fp32 from the blocks' sums.  A block's sum of
        # 2^128 or more has no finite fp32 value: a running sum that rounds it
        # is infinite from there on, whatever the 64-bit sum of all blocks
        # comes to (one that adds two blocks before it rounds may stay finite).
        past = (np.abs(blocks) >= 2.0 ** 128).any(axis=0)
        assert (~np.isfinite(y[past]) | (y[past] == want[past])).all(), xb
        # results below fp32's normal range may be flushed: they are held to its smallest normal number
        normal = ~(np.abs(want) < 2.0 ** -126)
        held = normal & ~past
        assert np.array_equal(y[held], want[held], equal_nan=True), xb
        assert (np.abs(y[~normal] - want[~normal]) <= 2.0 ** -126).all(), xb


@pytest.mark.parametrize("M", [1, 3, 40, 150])
def test_nan_stays_in_its_row_and_vector(M):
    rng = np.random.default_rng(M)
    N, K, E, top_k = 70, 288, 4, 2
    wc, ws = make(rng, (E, N), K)
    xc, xs = make(rng, (M,), K)
    ids = make_ids(rng, M, top_k, E, holes=False)
    ws[1, 5, 3] = 255
    xs[M // 2, 8] = 255
    y = q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs))
    want, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), False)
    close(y, want, K * U * A, f"nan {M}")


def test_a_token_that_names_one_expert_twice():
    rng = np.random.default_rng(8)
    for M in (1, 4, 9):
        wc, ws = make(rng, (3, 40), 96)
        xc, xs = make(rng, (M, 4), 96)
        ids = np.full((M, 4), 1, np.int32)
        y = q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs))
        want, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), True)
        close(y, want, 96 * U * A, f"same expert {M}")


@pytest.mark.parametrize("off_w,off_x", [(1, 0), (2, 3), (3, 1), (0, 2)])
@pytest.mark.parametrize("M", [1, 3, 20, 150])
def test_scales_start_at_any_byte(M, off_w, off_x):
    rng = np.random.default_rng(off_w + 4 * off_x)
    N, K, E = 37, 96, 3                                        # odd row and expert strides of the scales
    wc, ws = make(rng, (E, N), K)
    xc, xs = make(rng, (M,), K)
    ids = make_ids(rng, M, 2, E)

    def shifted(a, off):
        buf = torch.full((a.size + 16,), 255, dtype=torch.uint8, device="cuda")
        buf[off:off + a.size] = dev(a).reshape(-1)
        return buf[off:off + a.size].view(a.shape)

    y = q.qmv_gather_moe("mxfp4", dev(wc), shifted(ws, off_w), dev(ids), dev(xc), shifted(xs, off_x))
    want, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), False)
    close(y, want, K * U * A, "shifted scales")


@pytest.mark.parametrize("M,E,top_k,N,K", [(1, 8, 2, 96, 512), (4, 8, 2, 96, 512), (33, 4, 2, 100, 320),
                                           (260, 4, 2, 130, 512)])
def test_graph_replays_and_other_streams_equal_the_eager_call(M, E, top_k, N, K):
    rng = np.random.default_rng(M)
    wc, ws = (dev(a) for a in make(rng, (E, N), K))
    rw = dev(rng.random((M, top_k)).astype(np.float32))
    sets = []
    for _ in range(3):
        xc, xs = make(rng, (M,), K)
        sets.append((dev(make_ids(rng, M, top_k, E)), dev(xc), dev(xs)))
    ids, xc, xs = (t.clone() for t in sets[0])
    out, comb = torch.empty(M, top_k, N, device="cuda"), torch.empty(M, N, device="cuda")

    def call():
        q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs, y=out)
        q.qmv_gather_moe_combine_noalloc("mxfp4", wc, ws, ids, rw, xc, comb, x_scales=xs)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    side = torch.cuda.Stream()
    for k in (1, 2, 0, 1):
        for a, b in zip((ids, xc, xs), sets[k]):
            a.copy_(b)
        call()
        torch.cuda.synchronize()
        eager = out.clone(), comb.clone()
        out.fill_(float("nan"))
        comb.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(comb, eager[1])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = q.qmv_gather_moe("mxfp4", wc, ws, ids, xc, xs)
        side.synchronize()
        assert torch.equal(y, eager[0])


def test_large_expert_offsets():
    """An expert table whose byte offsets pass 2^32."""
    E, N, K = 1000, 1024, 9216                                 # 4.7 GB of codes
    rng = np.random.default_rng(1)
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    wc, ws = make(rng, (2, N), K)
    for i, e in enumerate((999, 500)):
        codes[e], scales[e] = dev(wc[i]), dev(ws[i])
    for M in (1, 6):
        xc, xs = make(rng, (M,), K)
        ids = np.tile(np.array([[999, 500]], np.int32), (M, 1))
        y = q.qmv_gather_moe("mxfp4", codes, scales, dev(ids), dev(xc), dev(xs))
        small = np.tile(np.array([[0, 1]], np.int32), (M, 1))
        want, A = R.gather(small, R.values(wc, ws), R.values(xc, xs), False)
        close(y, want, K * U * A, "large offsets")


def test_rows_behind_the_output_stay():
    rng = np.random.default_rng(3)
    for M in (1, 5, 40):
        wc, ws = make(rng, (4, 33), 96)
        xc, xs = make(rng, (M,), 96)
        buf = torch.full((M * 2 * 33 + 64,), 7.0, device="cuda")
        q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(make_ids(rng, M, 2, 4)), dev(xc), dev(xs),
                         y=buf[:M * 2 * 33].view(M, 2, 33))
        assert (buf[M * 2 * 33:] == 7.0).all()


@pytest.mark.parametrize("M,E,top_k,N,K", [(16, 64, 2, 20, 16384), (3, 500, 16, 33, 8192), (20, 300, 2, 100, 1088)])
def test_long_rows_with_few_pairs(M, E, top_k, N, K):
    """The widest vectors that a workgroup stages at once, gate/up and plain."""
    rng = np.random.default_rng(M + K)
    used = np.sort(rng.permutation(E)[:12]).astype(np.int32)
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 255, dtype=torch.uint8, device="cuda")
    wc, ws = make(rng, (12, N), K, 116, 120)
    codes[torch.from_numpy(used).long()], scales[torch.from_numpy(used).long()] = dev(wc), dev(ws)
    xc, xs = make(rng, (M,), K, 122, 124)
    small = rng.integers(0, 12, (M, top_k)).astype(np.int32)
    ids = dev(used[small])
    x, w = R.values(xc, xs), R.values(wc, ws)
    g, A = R.gather(small, w, x, False)
    close(q.qmv_gather_moe("mxfp4", codes, scales, ids, dev(xc), dev(xs)), g, K * U * A, "long rows")
    y = q.qmv_gather_moe_swiglu("mxfp4", codes, scales, codes, scales, ids, dev(xc), dev(xs))
    silu = g / (1 + np.exp(-g))
    tol = 1.1 * K * U * A * (np.abs(g) + K * U * A) + np.abs(silu) * K * U * A + (np.abs(g) + 8) * 2 * U * np.abs(silu * g)
    close(y, silu * g, tol, "long rows, gate/up")


@pytest.mark.parametrize("M,top_k,E", [(10, 4, 100), (16, 4, 40), (40, 2, 200), (3, 6, 50), (64, 1, 64), (200, 3, 1000)])
def test_many_pairs_of_one_expert_among_few_pairs(M, top_k, E):
    """More than 16 pairs of one expert where the call has fewer than two
    pairs per expert (chunks of 16 of the expert's pairs)."""
    rng = np.random.default_rng(M)
    N, K = 40, 288
    wc, ws = make(rng, (E, N), K)
    xc, xs = make(rng, (M,), K)
    for ids in (np.full((M, top_k), 7, np.int32), np.where(rng.random((M, top_k)) < 0.7, 7, -1).astype(np.int32),
                rng.integers(0, 2, (M, top_k)).astype(np.int32)):
        out = torch.full((M, top_k, N), float("nan"), device="cuda")
        y = q.qmv_gather_moe("mxfp4", dev(wc), dev(ws), dev(ids), dev(xc), dev(xs), y=out)
        want, A = R.gather(ids, R.values(wc, ws), R.values(xc, xs), False)
        close(y, want, K * U * A, f"one expert {M} {top_k}")


def test_dense_and_gate_up_replayed_and_on_two_streams_at_once():
    """Every kernel (few vectors, tiles of 64 and of 128, wide tiles): bit for
    bit the eager call's, under graph replays and beside each other on two
    streams."""
    rng = np.random.default_rng(3)
    K = 544
    dense = []
    for M, N in ((3, 100), (70, 12400), (1100, 6600)):
        wc, ws = (dev(a) for a in make(rng, (N,), K))
        xc, xs = (dev(a) for a in make(rng, (M,), K))
        dense.append((wc, ws, xc, xs, torch.empty(M, N, device="cuda")))
    routed = []
    for M, E, top_k, N in ((2, 8, 2, 96), (40, 4, 2, 1000), (150, 4, 2, 1000)):
        gu = [dev(a) for _ in range(2) for a in make(rng, (E, N), K)]
        xc, xs = (dev(a) for a in make(rng, (M,), K))
        routed.append((*gu, dev(make_ids(rng, M, top_k, E)), xc, xs, torch.empty(M, top_k, N, device="cuda")))

    def call():
        for *a, y in dense:
            q.qmv_dense("mxfp4", *a, y=y)
        for *a, y in routed:
            q.qmv_gather_moe_swiglu("mxfp4", *a, y=y)

    outs = [t[-1] for t in dense + routed]
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        for t in dense + routed:
            for x in t[-3:-1]:                                   # other codes and scales of the vectors
                x.copy_(x.flip(0))
        call()
        torch.cuda.synchronize()
        eager = [y.clone() for y in outs]
        for y in outs:
            y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, e) for y, e in zip(outs, eager)), k
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append([q.qmv_dense("mxfp4", *a) for *a, _ in dense] +
                              [q.qmv_gather_moe_swiglu("mxfp4", *a) for *a, _ in routed])
    for st in streams:
        st.synchronize()
    for rounds in got:
        for r in rounds:
            assert all(torch.equal(y, e) for y, e in zip(r, eager))
