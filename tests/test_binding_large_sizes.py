"""Sizes that the C ABI's ints cannot hold are refused by the binding: cut to
32 bits, 2^32 + 5 rows would be 5 rows and the rest of the output would be left
unwritten.  Tensors without memory ("meta"); no GPU needed.
"""
import pytest
import torch

import bit_block_quantized_amd as q

BIG = (1 << 32) + 5
U8, BF16, I32 = torch.uint8, torch.bfloat16, torch.int32


def meta(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="meta")


def refused(fn, *a, **kw):
    with pytest.raises(ValueError, match=r"2\^31"):
        fn(*a, **kw)


def test_steps():
    refused(q.qmx_rmsnorm, meta(BIG, 1))
    refused(q.qmx_rmsnorm, meta(1, (1 << 32) + 32), fmt="q8")
    refused(q.qmx_rmsnorm, meta(1 << 16, 1 << 15, 1))
    refused(q.qmx_router, meta(BIG, 8), 2)
    refused(q.qmx_router, meta(2, BIG), 2)
    refused(q.qmx_quantize, meta(1, (1 << 32) + 32))
    refused(q.qmx_dequantize, meta(1, (1 << 31) + 16, dtype=U8), meta(1, (1 << 27) + 1, dtype=U8))


def test_quantizers_take_more_rows():
    """(Their row count is 64 bits wide.)"""
    with pytest.raises(ValueError, match="GPU only"):
        q.qmx_quantize(meta(BIG, 32))


@pytest.mark.parametrize("x,xs", [((1, 16), (1, 1)), ((1, 32), None)])
def test_products(x, xs):
    x = meta(*x, dtype=U8 if xs else BF16)
    xs = xs and meta(*xs, dtype=U8)
    c, s = meta(BIG, 16, dtype=U8), meta(BIG, 1, dtype=U8)
    refused(q.qmv_dense, "mxfp4", c, s, x, xs)
    ids, rw = meta(1, 2, dtype=I32), meta(1, 2, dtype=torch.float32)
    for lead in ((BIG, 1), (1, BIG)):
        c, s = meta(*lead, 16, dtype=U8), meta(*lead, 1, dtype=U8)
        refused(q.qmv_gather_moe, "mxfp4", c, s, ids, x, xs)
        refused(q.qmv_gather_moe_swiglu, "mxfp4", c, s, c, s, ids, x, xs)
        refused(q.qmv_gather_moe_combine, "mxfp4", c, s, ids, rw, x, xs)
    c, s = meta(4, 3, 16, dtype=U8), meta(4, 3, 1, dtype=U8)
    wide, rw = meta(1, BIG, dtype=I32), meta(1, BIG, dtype=torch.float32)
    refused(q.qmv_gather_moe, "mxfp4", c, s, wide, x, xs)
    refused(q.qmv_gather_moe_swiglu, "mxfp4", c, s, c, s, wide, x, xs)
    refused(q.qmv_gather_moe_combine, "mxfp4", c, s, wide, rw, x, xs)
    y = meta(1, 3, dtype=torch.float32)
    refused(q.qmv_gather_moe_combine_noalloc, "mxfp4", c, s, wide, rw, x, y, x_scales=xs)


def test_many_vectors():
    c, s = meta(3, 16, dtype=U8), meta(3, 1, dtype=U8)
    refused(q.qmv_dense, "mxfp4", c, s, meta(BIG, 16, dtype=U8), meta(BIG, 1, dtype=U8))
    refused(q.qmv_gather_moe, "mxfp4", meta(4, 3, 16, dtype=U8), meta(4, 3, 1, dtype=U8), meta(BIG, 1, dtype=I32),
            meta(BIG, 16, dtype=U8), meta(BIG, 1, dtype=U8))
