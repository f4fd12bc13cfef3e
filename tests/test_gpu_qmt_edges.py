"""Log probabilities (include/qmt.h) where their arithmetic is at its edge, against
the 64-bit forms of f8_ref.py (needs an MI355X): logits further apart than fp32
holds, rows that rise at every step.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import f8_ref as F
import test_gpu_qmt
from test_gpu_qmt import host

pytestmark = pytest.mark.gpu

E = 2.0 ** -24                                                  # half a step of fp32
PLANS = [2, 1500]                                               # rows of 5003: parts and a join, a workgroup each
FAR = 3e38                                                      # FAR + FAR passes fp32's largest, 3.4e38


@pytest.mark.parametrize("M", PLANS)
@pytest.mark.parametrize("live,top_k,want", [
    ({8: FAR, 4104: -FAR}, 2, [8, 4104]),                       # in one wave's first two steps
    ({8: FAR, 16: -FAR, 4104: -2e38}, 2, [8, 4104]),            # with two logits to begin with
    ({8: FAR, 16: -FAR, 4104: -2e38}, 3, [8, 4104, 16]),
    ({8: FAR, 16: -2e38, 4104: -FAR}, 2, [8, 16]),
    ({8: -FAR, 4104: FAR}, 2, [4104, 8]),
    ({8: FAR, 5002: -FAR}, 4, [8, 5002, -1, -1]),               # behind the row's last whole group
    ({0: FAR, 1: -FAR, 4999: -FAR}, 3, [0, 1, 4999]),
    ({8: float("inf"), 16: -1.0, 4104: 1.0, 4105: -FAR}, 4, [8, 4104, 16, 4105]),
    ({8: float("inf"), 4104: float("inf"), 4100: -FAR}, 3, [8, 4104, 4100]),
])
@pytest.mark.parametrize("masked", [-float("inf"), float("nan")])
def test_logprobs_of_logits_further_apart_than_fp32_holds(M, live, top_k, want, masked):
    """The top logits are found by their values, not by differences."""
    V = 5003
    l = torch.full((M, V), masked)
    for i, v in live.items():
        l[:, i] = v
    t = torch.full((M,), next(iter(live)), dtype=torch.int32, device="cuda")
    lp, H, ids, top = (o.cpu() for o in q.qmt_logprobs(l.cuda(), t, top_k))
    assert (ids == torch.tensor(want, dtype=torch.int32)).all(), ids[(ids != torch.tensor(want)).any(1)][:3]
    with np.errstate(over="ignore"):                            # (a difference beyond fp32 is -infinity in it)
        ref = [np.asarray(o).astype(np.float32) for o in F.logprobs(l[:1].numpy(), t[:1].cpu().numpy(), top_k)]
    for g, w in ((lp, ref[0]), (H, ref[1]), (top, ref[3])):
        assert np.array_equal(g.numpy(), np.broadcast_to(w, g.shape), equal_nan=True)


def test_logprobs_masks_ties_and_far_logits_in_one_workgroup_a_row():
    """More rows than short parts are taken for."""
    test_gpu_qmt.test_logprobs_masks_ties_and_far_logits(PLANS[1])


@pytest.mark.parametrize("M", [520, 3])
@pytest.mark.parametrize("rise", [0.01, 0.1, 1.0, 30.0])
def test_logprobs_of_rows_that_rise_slowly(M, rise):
    """A new largest logit in every group: the sums move from one maximum to the
    next up to 512 times a row, and what a move rounds adds up.

    Tolerance: a term's argument is rounded twice and its constant once (2.3
    |z| 2^-24 of it), its exponential to 2^-23, a sum of eight three times, fp64's
    conversions not at all; the waves' and the parts' joins multiply it by two more
    exponentials (2^-23 each, and the arguments' share is in z's); a step's move
    adds 2^-26 in all.  So a term is off by (10.25 + 2.3 |z|) 2^-24 at most: with Z
    and Z2 the means of |z| and z^2 weighted by the terms, log s by (10.25 + 2.3
    Z) 2^-24, an output half a step more.  The entropy's second sum has two more
    roundings of a term, and the first one's error once more as its divisor.
    """
    V = 1 << 21
    row = torch.linspace(0.0, rise, V, dtype=torch.float64).to(torch.float32)
    l = row.cuda().expand(M, V).contiguous()
    t = np.full(M, V // 3, np.int32)
    lp, H, ids, top = q.qmt_logprobs(l, torch.from_numpy(t).cuda(), 4)
    for o in (lp, H, ids, top):
        assert (o == o[:1]).all()                               # (every row is the same, whichever workgroup has it)
    want = F.logprobs(row.numpy()[None], t[:1], 4)
    z = row.double().numpy() - float(row[-1])
    e = np.exp(z)
    Z, Z2 = (e * -z).sum() / e.sum(), (e * z * z).sum() / e.sum()
    dlog = (10.25 + 2.3 * Z) * E
    assert np.array_equal(ids[:1].cpu().numpy(), want[2])
    for g, w in ((host(lp[:1]), want[0]), (host(top[0]), want[3][0])):
        assert (np.abs(g - w) <= dlog + E * np.abs(w)).all(), (np.abs(g - w) / E, dlog / E)
    assert abs(host(H)[0] - want[1][0]) <= dlog + (12.25 * Z + 2.3 * Z2) * E + Z * dlog + E * abs(want[1][0])
