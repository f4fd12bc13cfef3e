"""Hand-worked values of the plain forms in mx_ref.py (no GPU needed)."""
import numpy as np
import pytest

import mx_ref as R


def block(*v):
    return np.array(list(v) + [0.0] * (32 - len(v)))


def test_mxfp4_scale_follows_the_rounded_maximum():
    # amax 6 = 1.5 * 4: scale 1; 6.99 still counts as 6; 7 = 1.75 * 4 as 8
    for amax, byte, top in ((6.0, 127, 7), (6.99, 127, 7), (7.0, 128, 6), (8.0, 128, 6), (4.0, 127, 6),
                            (1.0, 125, 6), (0.0, 0, 0)):
        c, s = R.quantize_mxfp4(block(amax))
        assert s[0] == byte and c[0] & 15 == top, (amax, s[0], c[0])


def test_mxfp4_rounds_ties_to_even_codes():
    x = block(6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -5.0, .2500001, .26)
    c, s = R.quantize_mxfp4(x)
    got = R.values(c, s)
    assert s[0] == 127
    assert got[:13].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, .5, .5]


def test_mxfp4_edges():
    c, s = R.quantize_mxfp4(block(np.inf, 1.0))
    assert s[0] == 255 and not c.any() and np.isnan(R.values(c, s)).all()
    c, s = R.quantize_mxfp4(block(2.0 ** -130, -(2.0 ** -128)))    # the scale stops at 2^-127
    assert s[0] == 0 and R.values(c, s)[:2].tolist() == [0.0, -(2.0 ** -128)]
    c, s = R.quantize_mxfp4(block(3.0e38))                          # 1.76 * 2^127 counts as 2^128
    assert s[0] == 253 and R.values(c, s)[0] == 4 * 2.0 ** 126


def test_q8():
    q, d = R.quantize_q8(block(127.0, -63.5, 0.5, 1.5).astype(np.float32))
    assert d[0] == 1.0 and q[:4].tolist() == [127, -64, 0, 2]
    q, d = R.quantize_q8(block(np.nan, 4.0).astype(np.float32))
    assert np.isnan(d[0]) and not q.any()
    q, d = R.quantize_q8(np.zeros(32, np.float32))
    assert d[0] == 0 and not q.any()


def test_rmsnorm():
    y, h = R.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), np.array([[0.0, 0.0]]), eps=0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]) and h.tolist() == [[3, 4]]


def test_router():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [np.nan, -np.inf, -np.inf, -np.inf], [-1e4, -1e4 - 1, -2e4, -3e4]])
    ids, w = R.router(l, 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 2]]
    assert np.allclose(w[0], np.exp([0, 0, -2]) / (2 + np.exp(-2.0))) and not w[1].any()
    ids, w = R.router(l, 2, "sigmoid")
    assert np.allclose(w[2], [1 / (1 + np.exp(-1.0)), 1 / (1 + np.exp(1.0))])
    _, w = R.router(l[:1], 1, "softmax", normalize=False, scale=2.0)
    assert w[0, 0] == pytest.approx(2 / (2 + np.exp(-2.0)))
