"""Router weights where their formula leaves fp32's normal range (needs an
MI355X)."""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import mx_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [None, 3.0])
def test_sigmoid_weights_below_the_normal_range(top):
    """1 / (1 + e^-l) is about e^l: a subnormal number from l = -87.4 on, the smallest of them at -103.3.  The
    exponential and the quotient are off by 2 steps of 2^-149 each at most there (2^-22 of the value above)."""
    l = np.float32(-np.linspace(80, 103, 16 * 64).reshape(64, 16))
    if top is not None:
        l[:, 0] = top
    ids, w = q.qmx_router(torch.from_numpy(l).cuda(), 16, scoring="sigmoid", normalize=False)
    want_ids, want = R.router(l, 16, "sigmoid", False)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.double().cpu().numpy()
    tol = 2.0 ** -21 * want + 4 * 2.0 ** -149
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
