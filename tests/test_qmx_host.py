"""The C ABI and the binding of libqmx.so on the host (no GPU needed): what
the header declares is exported, every refusal of include/qmx.h is returned
before a launch (fake but aligned pointers, never dereferenced), the same
checks run clean under the host sanitizers, and the binding refuses tensors
whose sizes do not fit the call.
"""
import inspect
import os
import re
import subprocess

import pytest
import torch

import bit_block_quantized_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUP = 0, 1, 2
F = 0x10000
F32, BF16, F16 = 0, 1, 2
O_BF16, O_Q8, O_MXFP4 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    return q.qmx_lib()


def test_exports_are_what_the_header_declares(L):
    with open(os.path.join(ROOT, "include", "qmx.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(qmx_[a-z0-9_]+)\s*\(", src))
    assert declared == {"qmx_rmsnorm", "qmx_router", "qmx_quantize", "qmx_dequantize", "qmx_strerror"}
    out = os.popen(f"nm -D --defined-only {q.QMX_LIB_PATH}").read()
    assert set(re.findall(r"\bT (\S+)", out)) == declared


def rmsnorm(L, xt=F32, x=F, rt=BF16, res=F, res_out=F, wt=BF16, w=F, eps=1e-5, fmt=O_MXFP4, y=F, ys=F, M=2, K=64):
    return L.qmx_rmsnorm(xt, x, rt, res, res_out, wt, w, eps, fmt, y, ys, M, K, None)


def router(L, lt=F32, logits=F, M=2, E=32, top_k=4, scoring=0, normalize=1, scale=1.0, ids=F, weights=F):
    return L.qmx_router(lt, logits, M, E, top_k, scoring, normalize, scale, ids, weights, None)


def quantize(L, xt=F32, x=F, fmt=O_MXFP4, codes=F, scales=F, rows=2, K=64):
    return L.qmx_quantize(xt, x, fmt, codes, scales, rows, K, None)


def dequantize(L, fmt=O_Q8, codes=F, scales=F, yt=BF16, y=F, rows=2, K=64):
    return L.qmx_dequantize(fmt, codes, scales, yt, y, rows, K, None)


CASES = [
    (rmsnorm, dict(x=None), EINVAL), (rmsnorm, dict(y=None), EINVAL), (rmsnorm, dict(ys=None), EINVAL),
    (rmsnorm, dict(res=None), EINVAL), (rmsnorm, dict(res_out=None), EINVAL), (rmsnorm, dict(M=0), EINVAL),
    (rmsnorm, dict(K=0), EINVAL), (rmsnorm, dict(M=-1), EINVAL), (rmsnorm, dict(eps=-1.0), EINVAL),
    (rmsnorm, dict(eps=float("nan")), EINVAL), (rmsnorm, dict(fmt=O_BF16), EINVAL),
    (rmsnorm, dict(xt=3), EUNSUP), (rmsnorm, dict(rt=-1), EUNSUP), (rmsnorm, dict(wt=7), EUNSUP),
    (rmsnorm, dict(fmt=3), EUNSUP), (rmsnorm, dict(fmt=-1), EUNSUP), (rmsnorm, dict(K=72), EUNSUP),
    (rmsnorm, dict(fmt=O_Q8, K=33), EUNSUP), (rmsnorm, dict(K=16416), EUNSUP),
    (rmsnorm, dict(fmt=O_BF16, ys=None, K=16385), EUNSUP), (rmsnorm, dict(x=F + 8), EINVAL),
    (rmsnorm, dict(res=F + 2), EINVAL), (rmsnorm, dict(res_out=F + 4), EINVAL), (rmsnorm, dict(w=F + 2), EINVAL),
    (rmsnorm, dict(y=F + 4), EINVAL), (rmsnorm, dict(fmt=O_Q8, ys=F + 1), EINVAL),
    (rmsnorm, dict(fmt=O_BF16, ys=None, K=7, x=F + 2), EINVAL),
    (rmsnorm, dict(fmt=O_BF16, ys=None, K=7, y=F + 1), EINVAL),
    (router, dict(logits=None), EINVAL), (router, dict(ids=None), EINVAL), (router, dict(weights=None), EINVAL),
    (router, dict(M=0), EINVAL), (router, dict(E=0), EINVAL), (router, dict(top_k=0), EINVAL),
    (router, dict(lt=F16), EUNSUP), (router, dict(scoring=2), EUNSUP), (router, dict(E=1025), EUNSUP),
    (router, dict(top_k=17), EUNSUP), (router, dict(E=3), EUNSUP), (router, dict(logits=F + 2), EINVAL),
    (router, dict(lt=BF16, logits=F + 1), EINVAL), (router, dict(ids=F + 2), EINVAL),
    (router, dict(weights=F + 1), EINVAL),
    (quantize, dict(x=None), EINVAL), (quantize, dict(codes=None), EINVAL), (quantize, dict(scales=None), EINVAL),
    (quantize, dict(rows=0), EINVAL), (quantize, dict(K=-32), EINVAL), (quantize, dict(K=48), EUNSUP),
    (quantize, dict(fmt=O_BF16), EUNSUP), (quantize, dict(xt=5), EUNSUP), (quantize, dict(x=F + 4), EINVAL),
    (quantize, dict(codes=F + 8), EINVAL), (quantize, dict(fmt=O_Q8, scales=F + 1), EINVAL),
    (quantize, dict(rows=2 ** 60, K=64), EUNSUP),
    (dequantize, dict(y=None), EINVAL), (dequantize, dict(yt=3), EUNSUP), (dequantize, dict(fmt=O_BF16), EUNSUP),
    (dequantize, dict(rows=-3), EINVAL), (dequantize, dict(y=F + 2), EINVAL), (dequantize, dict(scales=F + 1), EINVAL),
]


@pytest.mark.parametrize("fn,kw,want", CASES)
def test_refusals(L, fn, kw, want):
    assert fn(L, **kw) == want


def test_strerror(L):
    assert all("unknown" not in L.qmx_strerror(s).decode() for s in range(4))
    assert L.qmx_strerror(99).decode() == "unknown status"


def test_checks_under_sanitizers(L, tmp_path):
    exe = str(tmp_path / "qmx_host_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "bit_block_quantized_amd", "csrc"),
                    os.path.join(ROOT, "tests", "qmx_host_check.cpp"), "-o", exe], check=True)
    cases = CASES + [(f, {}, OK) for f in (rmsnorm, router, quantize, dequantize)] + [
        (rmsnorm, dict(res=None, res_out=None, w=None, fmt=O_BF16, ys=None, K=7, x=F + 4, y=F + 2), OK),
        (rmsnorm, dict(ys=F + 1), OK), (quantize, dict(scales=F + 3, rows=2 ** 40), OK),
        (router, dict(lt=BF16, logits=F + 2, E=1024, top_k=16), OK)]
    lines = []
    for fn, kw, _ in cases:
        params = [p for p in inspect.signature(fn).parameters.values() if p.name != "L"]
        vals = [kw.get(p.name, p.default) for p in params]
        if any(v != v for v in vals if isinstance(v, float)):
            vals = [-1.0 if isinstance(v, float) and v != v else v for v in vals]    # (read as a number)
        lines.append(" ".join([fn.__name__] + [repr(0 if v is None else v) for v in vals]))
    r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="halt_on_error=1"))
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stderr[-2000:]
    for (fn, kw, want), got, line in zip(cases, r.stdout.split(), lines):
        assert int(got) == want, line


# ------------------------------------------------------------------ binding

def gpu_only(fn, *a, **kw):
    with pytest.raises(ValueError, match="GPU only"):
        fn(*a, **kw)


def bad(err, match, fn, *a, **kw):
    with pytest.raises(err, match=match):
        fn(*a, **kw)


def test_consistent_calls_reach_the_device_check():
    x, w = torch.zeros(3, 64), torch.zeros(64, dtype=torch.bfloat16)
    gpu_only(q.qmx_rmsnorm, x, w)
    gpu_only(q.qmx_rmsnorm, x, residual=x.half(), fmt="mxfp4")
    gpu_only(q.qmx_rmsnorm, torch.zeros(2, 3, 7))
    gpu_only(q.qmx_router, x, 16)
    gpu_only(q.qmx_quantize, x, "q8")
    gpu_only(q.qmx_dequantize, torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8))


def test_binding_refusals():
    x = torch.zeros(3, 64)
    bad(TypeError, "x must be", q.qmx_rmsnorm, [1.0])
    bad(TypeError, "dtype", q.qmx_rmsnorm, x.double())
    bad(ValueError, "contiguous", q.qmx_rmsnorm, x.t())
    bad(ValueError, "fmt", q.qmx_rmsnorm, x, fmt="fp8")
    bad(ValueError, "multiple of 32", q.qmx_rmsnorm, torch.zeros(2, 40), fmt="q8")
    bad(ValueError, "weight has shape", q.qmx_rmsnorm, x, torch.zeros(63))
    bad(ValueError, "residual has shape", q.qmx_rmsnorm, x, residual=torch.zeros(2, 64))
    bad(ValueError, "residual_out needs", q.qmx_rmsnorm, x, residual_out=x)
    bad(ValueError, "y_scales", q.qmx_rmsnorm, x, y_scales=x)
    bad(ValueError, "at least one", q.qmx_rmsnorm, torch.zeros(0, 64))
    bad(ValueError, "top_k", q.qmx_router, x, 17)
    bad(ValueError, "top_k", q.qmx_router, torch.zeros(2, 3), 4)
    bad(ValueError, "scoring", q.qmx_router, x, 2, scoring="max")
    bad(TypeError, "dtype", q.qmx_router, x.half(), 2)
    bad(ValueError, r"\[M\]\[E\]", q.qmx_router, torch.zeros(2, 3, 4), 2)
    bad(ValueError, "fmt", q.qmx_quantize, x, "bf16")
    bad(ValueError, "multiple of 32", q.qmx_quantize, torch.zeros(2, 33))
    bad(ValueError, "scales has shape", q.qmx_dequantize, torch.zeros(3, 32, dtype=torch.uint8),
        torch.zeros(3, 3, dtype=torch.uint8))
    bad(TypeError, "codes has dtype", q.qmx_dequantize, torch.zeros(3, 32, dtype=torch.uint8),
        torch.zeros(3, 1, dtype=torch.float16), "q8")
    bad(ValueError, "dtype is", q.qmx_dequantize, torch.zeros(3, 32, dtype=torch.uint8),
        torch.zeros(3, 2, dtype=torch.uint8), dtype=torch.int8)


def test_mxfp4_activation_sizes_on_the_products():
    E, N, K, M, top_k = 6, 40, 128, 3, 2
    c, s = torch.zeros(E, N, K // 2, dtype=torch.uint8), torch.zeros(E, N, K // 32, dtype=torch.uint8)
    ids = torch.zeros(M, top_k, dtype=torch.int32)
    x, xs = torch.zeros(M, K // 2, dtype=torch.uint8), torch.zeros(M, K // 32, dtype=torch.uint8)
    xp, xsp = torch.zeros(M, top_k, K // 2, dtype=torch.uint8), torch.zeros(M, top_k, K // 32, dtype=torch.uint8)
    gpu_only(q.qmv_gather_moe, "mxfp4", c, s, ids, x, xs)
    gpu_only(q.qmv_gather_moe, "mxfp4", c, s, ids, xp, xsp)
    gpu_only(q.qmv_gather_moe_swiglu, "mxfp4", c, s, c, s, ids, x, xs)
    gpu_only(q.qmv_gather_moe_combine, "mxfp4", c, s, ids, torch.zeros(M, top_k), xp, xsp)
    gpu_only(q.qmv_dense, "mxfp4", c[0], s[0], x, xs)
    bad(ValueError, "MXFP4 activations need", q.qmv_dense, "mxfp4", c[0], s[0], x)
    bad(ValueError, "x_scales has shape", q.qmv_dense, "mxfp4", c[0], s[0], x, xs[:, :-1])
    bad(ValueError, "x has shape", q.qmv_gather_moe, "mxfp4", c, s, ids, x[:-1], xs)
    bad(ValueError, "w_codes", q.qmv_gather_moe, "mxfp4", c, s, ids, torch.zeros(M, K, dtype=torch.uint8), xs)
    bad(ValueError, "x has shape", q.qmv_gather_moe, "mxfp4", c, s, ids, x, xs, x_per_slot=True)


def test_mxfp4_activation_refusals_of_the_products():
    L = q.lib()

    def dense(wfmt=0, codes=F, scales=F, x=F, xs=F, y=F, M=1, N=64, K=64):
        return L.qmv_dense(wfmt, codes, scales, 4, x, xs, y, M, N, K, None)

    for kw, want in ((dict(xs=None), EINVAL), (dict(x=None), EINVAL), (dict(x=F + 8), EINVAL), (dict(wfmt=1), EUNSUP),
                     (dict(wfmt=2), EUNSUP), (dict(K=48), EUNSUP), (dict(M=8193), EUNSUP), (dict(codes=F + 8), EINVAL),
                     (dict(y=F + 2), EINVAL), (dict(K=16416), EUNSUP)):
        assert dense(**kw) == want, kw
    assert L.qmv_gather_moe(0, F, F, 4, None, 1, 1, 4, F, F, 0, F, 64, 64, None) == EINVAL
    assert L.qmv_gather_moe(0, F, F, 1024, F, 5, 1, 4, F, F, 0, F, 64, 64, None) == EUNSUP
    assert L.qmv_gather_moe_swiglu(0, F, F, None, F, 4, F, 1, 1, 4, F, F, F, 64, 64, None) == EINVAL
    assert L.qmv_gather_moe_combine(0, F, F, 4, F, None, 1, 1, 4, F, F, 1, F, 64, 64, None) == EINVAL
    assert L.qmv_gather_moe_combine_noalloc(0, F, F, 4, F, F, 512, 8, 4, F, F, 1, F, 4097, 64, None) == 4
