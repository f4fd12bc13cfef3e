"""Log probabilities and head norms (include/qmt.h) where their arithmetic is at
its edge, against 64-bit forms (needs an MI355X): logits further apart than fp32
holds, rows that rise at every step; a normed value's one rounding, in every
kernel for many heads.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import f8_ref as F
import test_gpu_qmt
from test_gpu_qmt import HALF_STEP, TYPES, host, values

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


LONG = [(130, 70001, 3), (513, 20001, 1), (2, 300001, 74), (1500, 4097, 1)]     # M, V, parts of a row


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("top_k", [0, 1, 32])
@pytest.mark.parametrize("M,V,parts", LONG)
def test_logprobs_in_long_parts(M, V, parts, top_k, t):
    """Rows, or several parts of them, that a workgroup takes in many steps, at every alignment; some masked."""
    rng = np.random.default_rng(M + V + top_k)
    off = int(rng.integers(8))
    l = values(rng, (M * V + 8,), t, 3.0)[off:off + M * V].view(M, V)
    l[:, rng.integers(0, V, V // 4)] = -float("inf")
    l[1] = -float("inf")
    l[0, rng.integers(0, V, 9)] = float("nan")
    test_gpu_qmt.check_logprobs(l, rng.integers(-1, V + 1, M).astype(np.int32), top_k)


def heads64(x, heads, kv_heads, D, table, pos, qw, kw, eps, style):
    """f8_ref.qk_norm_rope on the GPU, all heads at a time, and |a cos| + |b sin| of each output."""
    M, R = x.shape[0], table.shape[1]
    h = x[:, :(heads + kv_heads) * D].double().view(M, heads + kv_heads, D)
    w = torch.cat([qw.double().expand(heads, D), kw.double().expand(kv_heads, D)])
    n = h / ((h * h).mean(2, keepdim=True) + float(np.float32(eps))).sqrt() * w
    inside = ((pos >= 0) & (pos < table.shape[0]))[:, None, None]
    row = table[pos.long().clamp(0, table.shape[0] - 1)].double()[:, None]
    c, s = row[..., :R // 2], row[..., R // 2:]
    a, b = (slice(0, R // 2), slice(R // 2, R)) if style == "half" else (slice(0, R, 2), slice(1, R, 2))
    y, mag = n.clone(), n.abs()
    y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
    mag[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
    mag[..., b] = (n[..., b] * c).abs() + (n[..., a] * s).abs()
    return torch.where(inside, y, 0.0), torch.where(inside, mag, 0.0)


MANY = (3300, 7, 3)                                             # tokens, heads and key heads: 33000 heads
STYLES = ["half", "pairs"]
HEADS = [(MANY, D, xt, yt, style) for D in (32, 56, 128, 200, 264) for xt in TYPES for yt in TYPES for style in STYLES] + \
        [((5, 7, 3), D, xt, yt, style) for D, xt, yt, style in ((32, "f32", "f32", "half"), (56, "bf16", "f32", "pairs"),
         (128, "f16", "f32", "half"), (200, "f32", "f32", "pairs"), (264, "bf16", "f32", "half"))]


@pytest.mark.parametrize("sizes,D,xt,yt,style", HEADS)
def test_heads_round_once_before_the_rotation(sizes, D, xt, yt, style):
    """Tolerance: the norm's products are formed in 64 bits and rounded to fp32
    (half a step, E), 1 / sqrt to 2^-45; values that are not turned are then as they
    are, or rounded to the output's type; turned ones have two products and a sum
    in fp32: each term E of its own and E of the rounded norm, the sum E of itself, at
    most 3 E (1 + 2^-20) of |a cos| + |b sin| in all.  A 16-bit type's subnormals
    are 2^-24 (fp16), 2^-133 (bf16) apart: half of that more.
    """
    M, H, Hk = sizes
    rng = np.random.default_rng(D + len(xt) + 2 * len(yt))
    R, rest = D // 2 // 8 * 8, 4
    x = values(rng, (M, (H + Hk) * D + rest), xt, 3.0)
    angle = rng.uniform(-np.pi, np.pi, (50, R // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    table[0, :R // 2], table[0, R // 2:] = 1.0, 0.0             # position 0 turns nothing
    pos = torch.from_numpy(rng.integers(-1, 51, M).astype(np.int32)).cuda()
    pos[::3] = 0
    qw, kw = (values(rng, (D,), "f32") for _ in range(2))
    got = torch.cat(q.qmt_qk_norm_rope(x, H, Hk, D, table, pos, qw, kw, style=style, dtype=TYPES[yt]), 1).double()
    want, mag = heads64(x, H, Hk, D, table, pos, qw, kw, 1e-5, style)
    turned = torch.zeros((M, 1, D), dtype=torch.bool, device="cuda")
    turned[pos != 0, :, :R] = True
    off = torch.where(turned, 3 * E * mag, E * want.abs()) * (1 + 2.0 ** -20)
    if yt != "f32":
        off = off + HALF_STEP[yt] * (want.abs() + off) + (2.0 ** -25 if yt == "f16" else 2.0 ** -134)
    bad = (got - want).abs() > off
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[:3], ((got - want).abs() / off.clamp(min=1e-300)).max())
