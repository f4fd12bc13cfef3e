"""The C ABI and the binding of libqmt.so, and the e4m3 formats of libqmv.so and
libqmx.so, on the host (no GPU needed): what the header declares is exported,
every refusal is returned before a launch (fake but aligned pointers, never
dereferenced), the same checks run clean under the host sanitizers, and the
binding refuses tensors whose sizes do not fit the call.
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
W_F8, A_F8, O_F8 = 3, 5, 4


@pytest.fixture(scope="module")
def L():
    return q.qmt_lib()


def test_exports_are_what_the_header_declares(L):
    with open(os.path.join(ROOT, "include", "qmt.h")) as f:
        src = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(qmt_[a-z0-9_]+)\s*\(", src))
    assert declared == {"qmt_quantize_weights", "qmt_dequantize_weights", "qmt_qk_norm_rope", "qmt_logprobs",
                        "qmt_logprobs_workspace", "qmt_strerror"}
    out = os.popen(f"nm -D --defined-only {q.QMT_LIB_PATH}").read()
    assert set(re.findall(r"\bT (\S+)", out)) == declared


def quantize(L, xt=F32, x=F, codes=F, scales=F, E=2, N=40, K=64):
    return L.qmt_quantize_weights(xt, x, codes, scales, E, N, K, None)


def dequantize(L, codes=F, scales=F, yt=BF16, y=F, E=2, N=40, K=64):
    return L.qmt_dequantize_weights(codes, scales, yt, y, E, N, K, None)


def qk(L, xt=F32, x=F, row=512, heads=4, kv=2, D=64, table=F, P=9, R=64, pos=F, wt=BF16, qw=F, kw=F, eps=1e-5, style=0,
       yt=BF16, q=F, k=F, M=3):
    return L.qmt_qk_norm_rope(xt, x, row, heads, kv, D, table, P, R, pos, wt, qw, kw, eps, style, yt, q, k, M, None)


def logprobs(L, lt=F32, logits=F, M=2, V=50000, tokens=F, top_k=5, lp=F, ent=F, ids=F, top=F, ws=F):
    return L.qmt_logprobs(lt, logits, M, V, tokens, top_k, lp, ent, ids, top, ws, None)


CASES = [
    (quantize, dict(x=None), EINVAL), (quantize, dict(codes=None), EINVAL), (quantize, dict(scales=None), EINVAL),
    (quantize, dict(E=0), EINVAL), (quantize, dict(N=-1), EINVAL), (quantize, dict(K=0), EINVAL),
    (quantize, dict(K=48), EUNSUP), (quantize, dict(xt=3), EUNSUP), (quantize, dict(xt=-1), EUNSUP),
    (quantize, dict(K=1 << 24), EUNSUP), (quantize, dict(N=1 << 24), EUNSUP),
    (quantize, dict(E=2 ** 31 - 1, N=2 ** 23, K=2 ** 23), EUNSUP), (quantize, dict(x=F + 8), EINVAL),
    (quantize, dict(codes=F + 4), EINVAL), (quantize, dict(scales=F + 2), EINVAL),
    (dequantize, dict(y=None), EINVAL), (dequantize, dict(yt=4), EUNSUP), (dequantize, dict(y=F + 8), EINVAL),
    (dequantize, dict(scales=F + 1), EINVAL), (dequantize, dict(N=0), EINVAL),
    (qk, dict(x=None), EINVAL), (qk, dict(table=None), EINVAL), (qk, dict(pos=None), EINVAL), (qk, dict(q=None), EINVAL),
    (qk, dict(k=None), EINVAL), (qk, dict(kv=0), EINVAL), (qk, dict(heads=0), EINVAL), (qk, dict(kv=-1, k=None), EINVAL),
    (qk, dict(M=0), EINVAL), (qk, dict(P=0), EINVAL), (qk, dict(R=0), EINVAL), (qk, dict(R=-8), EINVAL),
    (qk, dict(eps=-1.0), EINVAL), (qk, dict(eps=float("nan")), EINVAL), (qk, dict(row=380), EINVAL),
    (qk, dict(row=514), EINVAL), (qk, dict(row=-4), EINVAL), (qk, dict(xt=3), EUNSUP), (qk, dict(yt=-1), EUNSUP),
    (qk, dict(wt=5), EUNSUP), (qk, dict(style=2), EUNSUP), (qk, dict(D=60), EUNSUP), (qk, dict(D=520, R=8), EUNSUP),
    (qk, dict(R=12), EUNSUP), (qk, dict(R=72), EUNSUP), (qk, dict(heads=4096), EUNSUP), (qk, dict(row=1 << 24), EUNSUP),
    (qk, dict(M=2 ** 29), EUNSUP), (qk, dict(x=F + 8), EINVAL), (qk, dict(xt=BF16, x=F + 4), EINVAL),
    (qk, dict(q=F + 4), EINVAL), (qk, dict(yt=F32, k=F + 8), EINVAL), (qk, dict(table=F + 8), EINVAL),
    (qk, dict(pos=F + 2), EINVAL), (qk, dict(qw=F + 4), EINVAL), (qk, dict(kw=F + 2), EINVAL),
    (logprobs, dict(logits=None), EINVAL), (logprobs, dict(tokens=None), EINVAL), (logprobs, dict(lp=None), EINVAL),
    (logprobs, dict(ids=None), EINVAL), (logprobs, dict(top=None), EINVAL), (logprobs, dict(top_k=0), EINVAL),
    (logprobs, dict(top_k=-1), EINVAL), (logprobs, dict(M=0), EINVAL), (logprobs, dict(V=0), EINVAL),
    (logprobs, dict(tokens=None, lp=None, ent=None, top_k=0, ids=None, top=None), EINVAL),
    (logprobs, dict(lt=3), EUNSUP), (logprobs, dict(top_k=33), EUNSUP), (logprobs, dict(V=1 << 30), EUNSUP),
    (logprobs, dict(M=1 << 24), EUNSUP), (logprobs, dict(logits=F + 2), EINVAL), (logprobs, dict(lt=BF16, logits=F + 1), EINVAL),
    (logprobs, dict(tokens=F + 2), EINVAL), (logprobs, dict(lp=F + 1), EINVAL), (logprobs, dict(ent=F + 2), EINVAL),
    (logprobs, dict(ids=F + 2), EINVAL), (logprobs, dict(top=F + 1), EINVAL),
]


@pytest.mark.parametrize("fn,kw,want", CASES)
def test_refusals(L, fn, kw, want):
    assert fn(L, **kw) == want


def test_logprobs_workspace_is_checked(L):
    assert L.qmt_logprobs_workspace(2, 50000, 5) > 0
    assert logprobs(L, ws=None) == EINVAL and logprobs(L, ws=F + 8) == EINVAL
    assert L.qmt_logprobs_workspace(4096, 50000, 5) == 0
    for bad in ((0, 5, 1), (1, 0, 1), (1, 5, -1), (1, 5, 33), (1, 1 << 30, 1), (1 << 24, 5, 1)):
        assert L.qmt_logprobs_workspace(*bad) == 0


def test_strerror(L):
    assert all("unknown" not in L.qmt_strerror(s).decode() for s in range(4))
    assert L.qmt_strerror(99).decode() == "unknown status"


def test_checks_under_sanitizers(L, tmp_path):
    exe = str(tmp_path / "qmt_host_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "bit_block_quantized_amd", "csrc"),
                    os.path.join(ROOT, "tests", "qmt_host_check.cpp"), "-o", exe], check=True)
    cases = CASES + [(f, {}, OK) for f in (quantize, dequantize, qk, logprobs)] + [
        (quantize, dict(E=2 ** 20, N=2 ** 20, K=2 ** 20), OK), (qk, dict(kv=0, k=None, qw=None, kw=None, wt=9), OK),
        (qk, dict(xt=BF16, x=F + 8, q=F + 8, k=F + 8, qw=F + 8, R=8, D=512, row=4096), OK),
        (qk, dict(heads=4094, row=4096 * 64, M=2 ** 19 - 1), OK),
        (logprobs, dict(lt=F16, logits=F + 2, V=2 ** 30 - 1, top_k=32), OK),
        (logprobs, dict(tokens=None, lp=None, top_k=0, ids=None, top=None), OK), (logprobs, dict(ent=None), OK)]
    lines = []
    for fn, kw, _ in cases:
        params = [p for p in inspect.signature(fn).parameters.values() if p.name != "L"]
        vals = [kw.get(p.name, p.default) for p in params]
        vals = [-1.0 if isinstance(v, float) and v != v else v for v in vals]          # (read as a number)
        lines.append(" ".join([fn.__name__] + [repr(0 if v is None else v) for v in vals]))
    sizes = [(M, V) for M in (1, 2, 3, 100, 1023, 1024, 1025, 70000)
             for V in (1, 2, 7, 8, 2040, 2041, 2042, 2047, 2048, 2049, 4090, 131071, 201088, 2 ** 30 - 1)]
    lines += [f"covered {M} {V}" for M, V in sizes] + [f"workspace {M} {V} 32" for M, V in sizes]
    r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="halt_on_error=1"))
    assert r.returncode == 0 and "runtime error" not in r.stderr, r.stderr[-2000:]
    out = [int(v) for v in r.stdout.split()]
    for (fn, kw, want), got, line in zip(cases, out, lines):
        assert got == want, line
    rest = out[len(cases):]
    assert rest[:len(sizes)] == [1] * len(sizes)
    assert rest[len(sizes):] == [L.qmt_logprobs_workspace(M, V, 32) for M, V in sizes]


# ------------------------------------------------------ e4m3 elsewhere, host

def test_refusals_of_the_products():
    P = q.lib()

    def dense(wfmt=W_F8, codes=F, scales=F, afmt=A_F8, x=F, xs=F, y=F, M=1, N=64, K=64):
        return P.qmv_dense(wfmt, codes, scales, afmt, x, xs, y, M, N, K, None)

    for kw, want in ((dict(xs=None), EINVAL), (dict(x=None), EINVAL), (dict(scales=None), EINVAL), (dict(x=F + 8), EINVAL),
                     (dict(codes=F + 8), EINVAL), (dict(scales=F + 2), EINVAL), (dict(xs=F + 2), EINVAL),
                     (dict(y=F + 2), EINVAL), (dict(K=48), EUNSUP), (dict(K=16416), EUNSUP), (dict(M=8193), EUNSUP),
                     (dict(wfmt=4), EUNSUP), (dict(afmt=0), EUNSUP), (dict(afmt=1), EUNSUP), (dict(afmt=2), EUNSUP),
                     (dict(afmt=4), EUNSUP), (dict(wfmt=0), EUNSUP), (dict(wfmt=1), EUNSUP), (dict(wfmt=2), EUNSUP),
                     (dict(N=1 << 24), EUNSUP), (dict(N=131072, K=16384), EUNSUP), (dict(N=0), EINVAL)):
        assert dense(**kw) == want, kw
    assert P.qmv_gather_moe(W_F8, F, F, 4, None, 1, 1, A_F8, F, F, 0, F, 64, 64, None) == EINVAL
    assert P.qmv_gather_moe(W_F8, F, F, 1024, F, 5, 1, A_F8, F, F, 0, F, 64, 64, None) == EUNSUP
    assert P.qmv_gather_moe(W_F8, F, F, 4, F, 2049, 4, A_F8, F, F, 0, F, 64, 64, None) == EUNSUP
    assert P.qmv_gather_moe_swiglu(W_F8, F, F, None, F, 4, F, 1, 1, A_F8, F, F, F, 64, 64, None) == EINVAL
    assert P.qmv_gather_moe_combine(W_F8, F, F, 4, F, None, 1, 1, A_F8, F, F, 1, F, 64, 64, None) == EINVAL
    assert P.qmv_gather_moe_combine_noalloc(W_F8, F, F, 4, F, F, 512, 8, A_F8, F, F, 1, F, 4097, 64, None) == 4


def test_refusals_of_the_block_formats():
    X = q.qmx_lib()
    assert X.qmx_rmsnorm(F32, F, 0, None, None, 0, None, 1e-5, O_F8, F, F + 2, 2, 64, None) == EINVAL
    assert X.qmx_rmsnorm(F32, F, 0, None, None, 0, None, 1e-5, O_F8, F, None, 2, 64, None) == EINVAL
    assert X.qmx_rmsnorm(F32, F, 0, None, None, 0, None, 1e-5, O_F8, F, F, 2, 72, None) == EUNSUP
    assert X.qmx_rmsnorm(F32, F, 0, None, None, 0, None, 1e-5, 5, F, F, 2, 64, None) == EUNSUP
    assert X.qmx_quantize(F32, F, O_F8, F, F + 2, 2, 64, None) == EINVAL
    assert X.qmx_quantize(F32, F, O_F8, F, F, 2, 48, None) == EUNSUP
    assert X.qmx_quantize(F32, F, 3, F, F, 2, 64, None) == EUNSUP
    assert X.qmx_dequantize(O_F8, F + 8, F, F32, F, 2, 64, None) == EINVAL


# ------------------------------------------------------------------ binding

def gpu_only(fn, *a, **kw):
    with pytest.raises(ValueError, match="GPU only"):
        fn(*a, **kw)


def bad(err, match, fn, *a, **kw):
    with pytest.raises(err, match=match):
        fn(*a, **kw)


F8 = torch.float8_e4m3fn


def test_consistent_calls_reach_the_device_check():
    x = torch.zeros(3, 288)
    for dt in (torch.uint8, F8):
        c, s = torch.zeros(3, 288, dtype=torch.uint8).view(dt), torch.zeros(3, 3)
        gpu_only(q.qmx_dequantize, c, s, "f8")
        gpu_only(q.qmt_dequantize_weights, c, torch.zeros(1, 3))
        w, ws = torch.zeros(4, 130, 288, dtype=torch.uint8).view(dt), torch.zeros(4, 2, 3)
        ids = torch.zeros(3, 2, dtype=torch.int32)
        gpu_only(q.qmv_dense, "f8", w[0], ws[0], c, s)
        gpu_only(q.qmv_gather_moe, "f8", w, ws, ids, c, s)
        gpu_only(q.qmv_gather_moe_swiglu, "f8", w, ws, w, ws, ids, c, s)
        cp, sp = torch.zeros(3, 2, 288, dtype=torch.uint8).view(dt), torch.zeros(3, 2, 3)
        gpu_only(q.qmv_gather_moe_combine, "f8", w, ws, ids, torch.zeros(3, 2), cp, sp)
        gpu_only(q.qmv_gather_moe, "f8", w, ws, ids, cp.view(6, 288), sp.view(6, 3), x_per_slot=True)
    gpu_only(q.qmx_quantize, x, "f8")
    gpu_only(q.qmx_rmsnorm, x, fmt="f8")
    gpu_only(q.qmt_quantize_weights, x)
    gpu_only(q.qmt_logprobs, x)
    gpu_only(q.qmt_logprobs, x.half(), torch.zeros(3, dtype=torch.int32), 32)
    gpu_only(q.qmt_qk_norm_rope, x, 3, 1, 64, torch.zeros(9, 64), torch.zeros(3, dtype=torch.int32))
    gpu_only(q.qmt_qk_norm_rope, x, 3, 0, 64, torch.zeros(9, 8), torch.zeros(3, dtype=torch.int32), torch.zeros(64))


def test_binding_refusals_of_the_products():
    w, ws = torch.zeros(4, 130, 288, dtype=torch.uint8), torch.zeros(4, 2, 3)
    x, xs, ids = torch.zeros(3, 288, dtype=torch.uint8), torch.zeros(3, 3), torch.zeros(3, 2, dtype=torch.int32)
    bad(ValueError, "need x_scales", q.qmv_dense, "f8", w[0], ws[0], x)
    bad(ValueError, "x_scales has shape", q.qmv_dense, "f8", w[0], ws[0], x, xs[:, :2])
    bad(ValueError, "x_scales has shape", q.qmv_dense, "f8", w[0], ws[0], x, xs.t().contiguous()[:2])
    bad(ValueError, "w_scales has shape", q.qmv_dense, "f8", w[0], ws[0, :1], x, xs)
    bad(ValueError, "w_scales has shape", q.qmv_gather_moe, "f8", w, ws[:3], ids, x, xs)
    bad(ValueError, "w_codes has shape", q.qmv_gather_moe, "f8", w[..., :256], ws, ids, x, xs)
    bad(ValueError, "up_scales has shape", q.qmv_gather_moe_swiglu, "f8", w, ws, w, ws[..., :2], ids, x, xs)
    bad(ValueError, "x has shape", q.qmv_gather_moe, "f8", w, ws, ids, x[:2], xs[:2])
    c = w.contiguous()
    # (types are looked at after the device)
    with pytest.raises(TypeError, match="x has dtype"):
        q._dev_ptr(torch.zeros(3, 288, dtype=torch.bfloat16), "x", q._afmt(q.W_F8B128, x)[1], x.device)
    with pytest.raises(TypeError, match="w_scales has dtype"):
        q._dev_ptr(ws.half(), "w_scales", q._scale_dt(q.W_F8B128), ws.device)
    with pytest.raises(TypeError, match="w_codes has dtype"):
        q._dev_ptr(c.view(torch.int8), "w_codes", q._code_dt(q.W_F8B128), c.device)


def test_binding_refusals_of_the_steps():
    x, i3 = torch.zeros(3, 288), torch.zeros(3, dtype=torch.int32)
    bad(ValueError, "multiple of 32", q.qmt_quantize_weights, torch.zeros(3, 40))
    bad(ValueError, r"\[N\]\[K\]", q.qmt_quantize_weights, torch.zeros(64))
    bad(TypeError, "dtype", q.qmt_quantize_weights, x.double())
    bad(ValueError, "contiguous", q.qmt_quantize_weights, torch.zeros(64, 32).t())
    bad(ValueError, "scales has shape", q.qmt_dequantize_weights, torch.zeros(3, 288, dtype=torch.uint8), torch.zeros(3, 3))
    bad(TypeError, "codes has dtype", q.qmt_dequantize_weights, torch.zeros(3, 288, dtype=torch.int8), torch.zeros(1, 3))
    bad(ValueError, "dtype is", q.qmt_dequantize_weights, torch.zeros(3, 288, dtype=torch.uint8), torch.zeros(1, 3), torch.int8)
    bad(ValueError, "scales has shape", q.qmx_dequantize, torch.zeros(3, 288, dtype=torch.uint8), torch.zeros(3, 9), "f8")
    qk = q.qmt_qk_norm_rope
    tb = torch.zeros(9, 64)
    bad(ValueError, "style", qk, x, 3, 1, 64, tb, i3, style="neox")
    bad(ValueError, "rows of 288", qk, x, 4, 1, 64, tb, i3)
    bad(ValueError, "multiple of 4", qk, torch.zeros(3, 290), 3, 1, 64, tb, i3)
    bad(ValueError, "heads", qk, x, 0, 1, 64, tb, i3)
    bad(ValueError, "heads", qk, x, 1, 1, 60, tb, i3)
    bad(ValueError, "heads", qk, x, 1, -1, 64, tb, i3)
    bad(ValueError, "table has shape", qk, x, 1, 1, 32, tb, i3)
    bad(ValueError, "table has shape", qk, x, 1, 1, 64, tb[:, :12].contiguous(), i3)
    bad(ValueError, "table has shape", qk, x, 1, 1, 64, tb[:, :0].contiguous(), i3)
    bad(TypeError, "table has dtype", qk, x, 1, 1, 64, tb.half(), i3)
    bad(ValueError, "positions has shape", qk, x, 1, 1, 64, tb, i3[:2])
    bad(TypeError, "positions has dtype", qk, x, 1, 1, 64, tb, i3.long())
    bad(ValueError, "q_weight has shape", qk, x, 1, 1, 64, tb, i3, torch.zeros(63))
    bad(TypeError, "one type", qk, x, 1, 1, 64, tb, i3, torch.zeros(64), torch.zeros(64).half())
    bad(ValueError, "k needs key heads", qk, x, 1, 0, 64, tb, i3, k=torch.zeros(1))
    bad(ValueError, "dtype is", qk, x, 1, 1, 64, tb, i3, dtype=torch.float64)
    lp = q.qmt_logprobs
    bad(ValueError, r"\[M\]\[V\]", lp, torch.zeros(3))
    bad(TypeError, "dtype", lp, x.double())
    bad(ValueError, "top_k is 33", lp, x, None, 33)
    bad(ValueError, "top_k is -1", lp, x, None, -1)
    bad(ValueError, "tokens has shape", lp, x, i3[:2])
    bad(TypeError, "tokens has dtype", lp, x, i3.long())
    bad(ValueError, "logprobs needs tokens", lp, x, logprobs=torch.zeros(3))
    bad(ValueError, "need top_k", lp, x, top_ids=i3)
    bad(TypeError, "workspace has dtype", lp, x, workspace=torch.zeros(9))
