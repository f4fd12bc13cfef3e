"""The 64-bit forms of f8_ref.py against hand-worked values, and against the
same things said another way (no GPU needed).
"""
import math

import numpy as np
import pytest
import torch

import f8_ref as F


def test_values_of_the_codes():
    assert F.E4M3[0x00] == 0 and F.E4M3[0x01] == 2.0 ** -9 and F.E4M3[0x07] == 7 * 2.0 ** -9
    assert F.E4M3[0x08] == 2.0 ** -6 and F.E4M3[0x38] == 1.0 and F.E4M3[0x39] == 1.125
    assert F.E4M3[0x7E] == 448.0 and F.E4M3[0xFE] == -448.0 and np.isnan(F.E4M3[[0x7F, 0xFF]]).all()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F.E4M3, t, equal_nan=True)
    assert (np.diff(F.GRID) > 0).all() and len(F.GRID) == 127


def test_codes_round_to_nearest_even():
    d = np.ones(8, np.float32)
    x = np.array([1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, 447.0, 448.0, 1e9], np.float32)
    # 1.0625 lies between 1 (0x38) and 1.125 (0x39), 1.1875 between 1.125 and 1.25 (0x3A)
    assert F.codes_of(x, d).tolist() == [0x38, 0x3A, 0xB8, 0x00, 0x02, 0x7E, 0x7E, 0x7E]


def test_codes_are_the_nearest_by_search():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(4000) * np.exp(3 * rng.standard_normal(4000))).astype(np.float32)
    d = np.full(4000, np.abs(x).max() / 448, np.float32)
    got = np.abs(F.E4M3[F.codes_of(x, d)])
    q = np.abs(x.astype(np.float64) / d)
    assert np.array_equal(np.abs(got - np.minimum(q, 448)), np.abs(F.GRID[None] - np.minimum(q, 448)[:, None]).min(1))


def test_scales_of_short_blocks():
    x = np.zeros((3, 160), np.float32)
    x[0, 5], x[0, 130], x[1, 159] = -896.0, 448.0, np.inf
    c, s = F.quantize_rows(x)
    assert s.shape == (3, 2) and s[0].tolist() == [2.0, 1.0] and s[2].tolist() == [2.0 ** -126] * 2
    assert np.isnan(s[1, 1]) and c[1, 159] == 0 and c[0, 5] == 0xFE and c[0, 130] == 0x7E
    w = np.zeros((130, 160), np.float32)
    w[0, 0], w[129, 159] = 448.0, 44.8
    c, s = F.quantize_weights(w)
    assert s.shape == (2, 2) and s[0, 0] == 1.0 and s[1, 1] == np.float32(44.8) / np.float32(448) and c[129, 159] == 0x7E
    assert F.weight_values(c, s)[0, 0] == 448.0


def test_rotation_by_hand():
    table = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 1.0, 1.0, 0.0]])       # cosines, sines of two pairs
    x = np.array([[3.0, 1.0, 1.0, 1.0], [2.0, 2.0, 2.0, 2.0], [1.0, 1.0, 1.0, 1.0]])
    q, k = F.qk_norm_rope(x, 1, 0, 4, table, [1, 0, 2], eps=0.0)
    r = 1 / math.sqrt(3.0)
    assert np.allclose(q[0, 0], [-r, r, 3 * r, r]) and np.allclose(q[1, 0], 1.0) and not q[2].any() and k.shape == (3, 0, 4)
    q, _ = F.qk_norm_rope(x, 1, 0, 4, table, [1, 0, -1], eps=0.0, style="pairs")
    assert np.allclose(q[0, 0], [-r, 3 * r, r, r]) and not q[2].any()


def test_logprobs_by_hand():
    inf = math.inf
    l = np.log(np.array([[1.0, 2.0, 5.0], [1.0, 1.0, 2.0]]))
    lp, H, ids, top = F.logprobs(l, [1, 5], 2)
    assert np.allclose(lp, [math.log(0.25), 0.0]) and ids.tolist() == [[2, 1], [2, 0]]
    assert np.allclose(H, [-(0.125 * math.log(0.125) + 0.25 * math.log(0.25) + 0.625 * math.log(0.625)),
                           -(0.5 * math.log(0.5) + 0.5 * math.log(0.25))])
    lp, H, ids, top = F.logprobs([[-inf, math.nan, 0.0], [-inf] * 3, [inf, 0.0, -inf]], [1, 1, 2], 2)
    assert lp.tolist() == [-inf] * 3 and H[:2].tolist() == [0.0, 0.0] and math.isnan(H[2])
    assert ids.tolist() == [[2, -1], [-1, -1], [0, 1]] and top[0].tolist() == [0.0, -inf] and np.isnan(top[2]).all()


@pytest.mark.parametrize("scale", [1.0, 8.0])
def test_logprobs_against_torch(scale):
    rng = np.random.default_rng(2)
    l = rng.standard_normal((5, 400)) * scale
    t = rng.integers(0, 400, 5)
    lp, H, ids, top = F.logprobs(l, t, 7)
    p = torch.log_softmax(torch.from_numpy(l), 1)
    assert np.allclose(lp, p[torch.arange(5), torch.from_numpy(t)]) and np.allclose(H, torch.special.entr(p.exp()).sum(1))
    assert np.allclose(top, p.topk(7, 1).values) and np.array_equal(ids, p.topk(7, 1).indices)
