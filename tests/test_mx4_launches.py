"""On the host (no GPU needed): every case of test_gpu_mx4_kernels.py reaches
the kernel that it names, and the 64-bit forms of mx4_exact.py are those of
mx_ref.py.
"""
import numpy as np
import pytest
import torch

import launches
import mx4_exact as X
import mx_ref as R
import test_gpu_mx4_kernels as G
from launches import mx4_combine, mx4_dense, mx4_gather, mx4_swiglu


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    with launches.Launches(tmp_path_factory.mktemp("recorder")) as l:
        yield l


def first(ls, kernel):
    assert ls[0].kernel == kernel, ls
    return ls[0]


def test_products(L):
    for kernel, M, N, K in G.DENSE:
        first(mx4_dense(L, M, N, K), kernel)
    for kernel, *case in G.GATHER:
        for per_slot in (False, True):
            first(mx4_gather(L, *case, per_slot), kernel)
    for kernel, *case in G.SWIGLU:
        first(mx4_swiglu(L, *case), kernel)
    for kernel, *case in G.COMBINE:
        for entry in ("qmv_gather_moe_combine", "qmv_gather_moe_combine_noalloc"):
            ls = mx4_combine(L, *case, entry=entry)
            first(ls, kernel)
            assert len(ls) == (1 if kernel == G.FEW_COMB else 2)


def test_runs_of_row_tiles(L):
    """Fewer workgroups than tiles: each takes a run of them."""
    runs = set()
    for kernel, entry, M, E, top_k, N, K in G.RUNS:
        if entry == "dense":
            l = first(mx4_dense(L, M, N, K), kernel)
        else:
            l = first((mx4_gather if entry == "gather" else mx4_swiglu)(L, M, E, top_k, N, K), kernel)
        chunk = 128 if "128" in kernel else 64
        rows = 64 if entry == "swiglu" else 128
        pairs = M * top_k
        items = -(-M // chunk) if entry == "dense" else min(pairs, E) + pairs // chunk
        tiles = -(-N // rows)
        run = next(r for r in range(1, tiles + 1) if 8 * -(-items * -(-tiles // r) // 8) == l.grid[0])
        assert run >= 2, (kernel, entry, M, N, K, l)
        runs.add((kernel, tiles % run != 0, N % 4 == 0))
    for kernel in (G.TILE64, G.TILE128, G.GU64, G.GU128):
        assert {r[1] for r in runs if r[0] == kernel} >= {True}, kernel      # a run that ends short
        assert {r[2] for r in runs if r[0] == kernel} == {True, False}, kernel


def test_edges(L):
    for K in (64, 96, 288, 544, 1056, 1120):
        for kernel, M, E, top_k, N in G.EDGES:
            first(mx4_gather(L, M, E, top_k, N, K) if E else mx4_dense(L, M, N, K), kernel)
    entries = {"gather": mx4_gather, "swiglu": mx4_swiglu,
               "combine": lambda *a: mx4_combine(*a, per_slot=False)}
    for kernel, entry, M, E, top_k, N in G.EMPTY:
        assert M * top_k > 64
        first(entries[entry](L, M, E, top_k, N, 544), kernel)
    for kernel, entry, M, E, top_k, N in G.SHIFTED:
        first((mx4_swiglu if entry == "swiglu" else mx4_combine)(L, M, E, top_k, N, 1120), kernel)
    for kernel, entry, M, E, top_k, N, K in G.FAR:
        first(entries[entry](L, M, E, top_k, N, K), kernel)
        assert (E - 1) * N * (K // 2) > (2 ** 31 if kernel == G.FEW else 2 ** 32)


def test_every_kernel_is_named(L):
    named = {c[0] for cases in (G.DENSE, G.GATHER, G.SWIGLU, G.COMBINE, G.RUNS, G.EDGES, G.EMPTY, G.FAR) for c in cases}
    assert named == {G.FEW, G.FEW_GU, G.FEW_COMB, G.TILE64, G.TILE128, G.GU64, G.GU128, G.WIDE}


# ------------------------------------------------------- the 64-bit forms

def test_values_and_products():
    g = torch.Generator()
    g.manual_seed(1)
    c, s = X.codes(g, (3, 5), 96, 0, 256)
    s[0, 0, 0], s[1, 2, 1] = 255, 0
    assert np.array_equal(X.values(c, s).numpy(), R.values(c.numpy(), s.numpy()), equal_nan=True)
    wc, ws = X.codes(g, (4, 7), 64, X.W_LO)
    for lead in ((6,), (6, 2)):
        xc, xs = X.codes(g, lead, 64, X.X_LO)
        ids = X.make_ids(g, 6, 2, 4)
        y, A = X.gather(ids, wc, ws, X.values(xc, xs))
        want, B = R.gather(ids.numpy(), R.values(wc.numpy(), ws.numpy()), R.values(xc.numpy(), xs.numpy()), len(lead) == 2)
        assert np.array_equal(y.numpy(), want) and np.array_equal(A.numpy(), B)
    with pytest.raises(AssertionError):
        X.held(torch.tensor(2.0 ** 22 * 2.0 ** (X.W_LO + X.X_LO - 254)))
