"""On the host (no GPU needed): the calls of test_gpu_qmx_large.py pass one
launch's 2^20 workgroups, and what is launched covers their rows.
"""
import pytest

import launches
from launches import P

LIMIT = 1 << 20


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    with launches.Launches(tmp_path_factory.mktemp("recorder")) as l:
        yield l


def groups(ls, n):
    assert [l.grid[1:] for l in ls] == [(1, 1)] * len(ls)
    assert sum(l.grid[0] for l in ls) == n and all(l.grid[0] <= LIMIT for l in ls), ls
    return ls


@pytest.mark.parametrize("K,M,rows", [(520, LIMIT + 5, 1), (257, LIMIT + 5, 1), (8, 4 * LIMIT + 5, 4), (5, 4 * LIMIT + 5, 4)])
def test_norm(L, K, M, rows):
    ls = L.call("qmx_rmsnorm", 1, P(), 0, P(), P(), 1, P(), 1e-5, 0, P(), None, M, K, None)
    assert len(groups(ls, -(-M // rows))) == 2


def test_norm_to_blocks(L):
    for fmt in (1, 2):
        assert len(groups(L.call("qmx_rmsnorm", 1, P(), 0, None, None, 0, None, 1e-5, fmt, P(), P(), LIMIT + 5, 544, None),
                          LIMIT + 5)) == 2


def test_router(L):
    for E, top_k in ((4, 2), (70, 8)):
        M = 4 * LIMIT + 5
        assert len(groups(L.call("qmx_router", 1, P(), M, E, top_k, 0, 1, 1.0, P(), P(), None), LIMIT + 2)) == 2


def test_quantizers_loop(L):
    K = 4096
    M = (1 << 33) // K + 33
    for fmt in (1, 2):
        for ls in (L.call("qmx_quantize", 1, P(), fmt, P(), P(), M, K, None),
                   L.call("qmx_dequantize", fmt, P(), P(), 1, P(), M, K, None)):
            assert len(groups(ls, LIMIT)) == 1 and M * K > LIMIT * 1024 * 8
