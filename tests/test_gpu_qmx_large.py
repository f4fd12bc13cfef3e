"""Calls of the norm, the router and the quantizers that pass one launch's
2^20 workgroups: rows on both sides of the border against the 64-bit forms of
mx_ref.py, every other row against its twin (needs an MI355X).

The inputs repeat a few rows with a period that divides no power of two, so a
row that the second launch (or the loop's second pass) leaves out or takes
from another place differs from its twin.
"""
import numpy as np
import pytest
import torch

import bit_block_quantized_amd as q
import mx_ref as R

pytestmark = pytest.mark.gpu

PERIOD = 1009
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def rows_like(base, M):
    """M rows: the PERIOD rows of base again and again."""
    return base.repeat((M + PERIOD - 1) // PERIOD, 1)[:M].contiguous()


def all_twins(out, head):
    """Every row of out equals the row of head that its input repeats."""
    for r in range(0, out.shape[0], 64 * PERIOD):
        part = out[r:r + 64 * PERIOD]
        assert torch.equal(part, rows_like(head, part.shape[0])), r


def base(K, t, seed, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (spread * torch.randn(PERIOD, K, device="cuda", generator=g)).to(TYPES[t])


# K: one row a workgroup (16-byte accesses, single values), four rows
@pytest.mark.parametrize("K,M", [(520, (1 << 20) + 5), (257, (1 << 20) + 5), (8, (1 << 22) + 5), (5, (1 << 22) + 5)])
def test_rmsnorm_past_one_launch(K, M):
    xb, rb = base(K, "bf16", K), base(K, "f32", K + 1)
    w = base(K, "bf16", K + 2)[0].contiguous()
    y = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    h = torch.full((M, K), float("nan"), device="cuda")
    q.qmx_rmsnorm(rows_like(xb, M), w, residual=rows_like(rb, M), y=y, residual_out=h)
    want, h32 = R.rmsnorm(xb.float().cpu().numpy(), w.float().cpu().numpy(), rb.cpu().numpy())
    got = y[:PERIOD].double().cpu().numpy()
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133).all()
    assert np.array_equal(h[:PERIOD].cpu().numpy(), h32)
    all_twins(y, y[:PERIOD])
    all_twins(h, h[:PERIOD])


@pytest.mark.parametrize("fmt", ["mxfp4", "q8"])
def test_rmsnorm_blocks_past_one_launch(fmt):
    M, K = (1 << 20) + 5, 544
    xb = base(K, "bf16", 1)
    y, s, _ = q.qmx_rmsnorm(rows_like(xb, M), fmt=fmt)
    want = R.rmsnorm(xb.float().cpu().numpy())[0].astype(np.float32)
    c, cs = R.quantize_mxfp4(want) if fmt == "mxfp4" else R.quantize_q8(want)
    assert np.array_equal(y[:PERIOD].cpu().numpy(), c) and np.array_equal(s[:PERIOD].cpu().numpy(), cs)
    all_twins(y, y[:PERIOD])
    all_twins(s, s[:PERIOD])


@pytest.mark.parametrize("E,top_k", [(4, 2), (70, 8)])
def test_router_past_one_launch(E, top_k):
    M = (1 << 22) + 5
    lb = base(E, "bf16", E)
    ids = torch.full((M, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((M, top_k), float("nan"), device="cuda")
    q.qmx_router(rows_like(lb, M), top_k, ids=ids, weights=w)
    want_ids, want = R.router(lb.double().cpu().numpy(), top_k)
    assert np.array_equal(ids[:PERIOD].cpu().numpy(), want_ids)
    # |l - top| below 32: 32 roundings of the exponent's argument, and 16 more
    assert (np.abs(w[:PERIOD].double().cpu().numpy() - want) <= np.abs(want) * 64 * 2.0 ** -22).all()
    all_twins(ids, ids[:PERIOD])
    all_twins(w, w[:PERIOD])


@pytest.mark.parametrize("fmt", ["mxfp4", "q8"])
def test_quantize_and_back_past_one_pass(fmt):
    """More than 2^20 workgroups of 1024 pieces of 8 values: each loops."""
    K = 4096
    M = (1 << 33) // K + 33
    xb = base(K, "bf16", 3)
    x = rows_like(xb, M)
    c, s = q.qmx_quantize(x, fmt)
    del x
    head = xb.float().cpu().numpy()
    wc, wsc = R.quantize_mxfp4(head) if fmt == "mxfp4" else R.quantize_q8(head)
    assert np.array_equal(c[:PERIOD].cpu().numpy(), wc) and np.array_equal(s[:PERIOD].cpu().numpy(), wsc)
    all_twins(c, c[:PERIOD])
    all_twins(s, s[:PERIOD])
    y = q.qmx_dequantize(c, s, fmt)
    v = R.values(wc, wsc) if fmt == "mxfp4" else R.q8_values(wc, wsc)
    assert torch.equal(y[:PERIOD].cpu(), torch.from_numpy(v.astype(np.float32)).bfloat16())
    all_twins(y, y[:PERIOD])
