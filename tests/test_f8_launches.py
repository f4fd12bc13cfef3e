"""On the host (no GPU needed): every case of test_gpu_f8_kernels.py reaches the
kernel that it names, the kernels of libqmt.so that calls reach, and LDS beyond
64 KB is granted on every device before it is used.
"""
import os
import re
import subprocess
import sys

import pytest

import launches
import test_gpu_f8 as D
import test_gpu_f8_kernels as G
import test_gpu_qmt_edges as Q
from launches import P, HERE, ROOT, SERVER

W, A = 3, 5


class Launches(launches.Launches):
    """With libqmt.so beside the other two."""

    def __init__(self, tmp_path):
        so = str(tmp_path / "hip_recorder.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        os.path.join(HERE, "hip_recorder.cpp"), "-o", so], check=True)
        libs = [os.path.join(ROOT, "bit_block_quantized_amd", f"lib{n}.so") for n in ("qmv", "qmx", "qmt")]
        self.p = subprocess.Popen([sys.executable, "-c", SERVER, so, *libs], stdin=subprocess.PIPE, stdout=subprocess.PIPE,
                                  text=True)


def name(mangled):
    """qmt_qk_norm_rope_kernel<16, 4, 1, 1, 0> of a launch's kernel."""
    m = re.search(r"\d(qm[vxt]_[a-z0-9_]*?_kernel)(?:I((?:L[a-z]n?\d+E)*))?", mangled)
    args = re.findall(r"L[a-z](n?)(\d+)E", m.group(2) or "")
    return m.group(1) + (f"<{', '.join(('-' if n else '') + v for n, v in args)}>" if args else "")


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    with Launches(tmp_path_factory.mktemp("recorder")) as l:
        yield l


def dense(M, N, K):
    return "qmv_dense", (W, P(), P(), A, P(), P(), P(), M, N, K, None)


def gather(M, E, top_k, N, K):
    return "qmv_gather_moe", (W, P(), P(), E, P(), M, top_k, A, P(), P(), 0, P(), N, K, None)


def swiglu(M, E, top_k, N, K):
    return "qmv_gather_moe_swiglu", (W, P(), P(), P(), P(), E, P(), M, top_k, A, P(), P(), P(), N, K, None)


def combine(M, E, top_k, N, K):
    return "qmv_gather_moe_combine", (W, P(), P(), E, P(), P(), M, top_k, A, P(), P(), 1, P(), N, K, None)


def kernels(L, call):
    return [l.kernel for l in L.call(call[0], *call[1])]


def test_products(L):
    for kernel, M, N, K in G.DENSE:
        assert kernels(L, dense(M, N, K)) == [kernel], (M, N, K)
    pairs, E = sum(G.COUNTS) + 12, len(G.COUNTS)
    for kernel, N, K in G.ROUTED:
        for top_k in (1, 5):
            M = -(-pairs // top_k)
            assert kernels(L, gather(M, E, top_k, N, K)) == [kernel], (N, K)
            assert kernels(L, combine(M, E, top_k, N, K))[0] == kernel, (N, K)
        assert kernels(L, swiglu(-(-pairs // 3), E, 3, N, K)) == [G.GU[kernel]], (N, K)
    assert kernels(L, combine(4, 64, 8, 300, 2880)) == [G.FEW_COMB]
    assert kernels(L, swiglu(1, 64, 8, 300, 2880)) == [G.FEW_GU]
    # more experts than the tile kernel counts, and rows longer than one launch's vectors fit LDS
    assert kernels(L, gather(4, 5000, 16, 20000, 16384)) == [G.FEW]


def test_workgroups(L):
    """A workgroup for each tile that the call can have, and 512 threads for two halves."""
    (l,) = L.call(*gather_args(600, 8, 2, 5500, 160))
    assert l.kernel == G.TILE and l.threads == 256 and l.grid[0] >= (8 + 1200 // 96) * 43
    (l,) = L.call(*gather_args(600, 8, 2, 300, 160))
    assert l.kernel == G.HALVES and l.threads == 512 and l.grid[0] >= (8 + 1200 // 96) * 3


def gather_args(*case):
    fn, args = gather(*case)
    return (fn, *args)


def test_every_device_has_its_own_lds_limits(tmp_path):
    with Launches(tmp_path) as L:                               # (limits are set once in a process)
        lds_limits(L)


def lds_limits(L):
    calls = [dense(8, 100, 16384), dense(8192, 7168, 7168), dense(64, 32897, 96), dense(97, 8193, 544),
             gather(200, 8, 2, 5500, 160), gather(200, 8, 2, 300, 160), swiglu(200, 8, 2, 5500, 160),
             swiglu(200, 8, 2, 300, 160), combine(4, 8, 4, 100, 16384), swiglu(1, 8, 8, 100, 16384)]
    limit, seen = {}, set()
    for device in (0, 1, 0):
        for fn, args in calls:
            status, lines = L.lines(fn, *args, device=device)
            assert status == 0
            for kind, dev, kernel, *v in lines:
                if kind == "attr":
                    limit[int(dev), kernel] = int(v[0])
                elif int(v[4]) > 64 * 1024:
                    seen.add(name(kernel))
                    assert limit.get((int(dev), kernel), 0) >= int(v[4]), (fn, args, device)
    assert {G.FEW, G.FEW_GU, G.FEW_COMB, G.TILE, G.TILE_GU, G.HALVES, G.HALVES_GU, G.WIDE} <= seen | {G.FEW_COMB}, seen


def test_combine_has_its_lds_limit_on_every_device(tmp_path):
    """Slots staged beyond 64 KB."""
    with Launches(tmp_path) as L:                               # (limits are set once in a process)
        combine_limit(L)


def combine_limit(L):
    limit = {}
    for device in (0, 1, 0):
        for case in D.BIG_COMBINE:
            fn, args = combine(*case)
            status, lines = L.lines(fn, *args, device=device)
            assert status == 0
            limit.update({(int(l[1]), l[2]): int(l[3]) for l in lines if l[0] == "attr"})
            ((dev, kernel, lds),) = [(int(l[1]), l[2], int(l[7])) for l in lines if l[0] == "launch"]
            assert name(kernel) == G.FEW_COMB and dev == device
            assert 64 * 1024 < lds <= limit.get((dev, kernel), 0) <= 160 * 1024, (case, device, lds)


def steps(L, fn, *args):
    status, lines = L.lines(fn, *args)
    assert status == 0
    return [(name(l[2]), int(l[3])) for l in lines if l[0] == "launch"]


def qk(M, H, Hk, D, xt=1, yt=1, style=0):
    row = (H + Hk) * D
    return ("qmt_qk_norm_rope", xt, P(), row, H, Hk, D, P(), 9, 8, P(), 1, P(), P(), 1e-5, style, yt, P(), P() if Hk else None,
            M, None)


def test_steps(L):
    for t in range(3):
        assert steps(L, "qmt_quantize_weights", t, P(), P(), P(), 2, 130, 160, None) == [(f"qmt_quantize_weights_kernel<{t}>", 8)]
    assert steps(L, "qmt_quantize_weights", 1, P(), P(), P(), (1 << 20) + 100, 1, 32, None) == \
        [("qmt_quantize_weights_kernel<1>", 1 << 20)]
    for D, G_ in ((32, 4), (40, 8), (128, 16), (256, 32), (264, 64)):
        assert steps(L, *qk(1, 8, 2, D))[0][0] == f"qmt_qk_norm_rope_kernel<{G_}, 1, -1, -1, -1>"
        for xt, yt, style in ((0, 1, 0), (1, 1, 1), (2, 0, 0), (1, 2, 1)):
            assert steps(L, *qk(4000, 8, 2, D, xt, yt, style)) == \
                [(f"qmt_qk_norm_rope_kernel<{G_}, 4, {xt}, {yt}, {style}>", -(-4000 * 3 * G_ // 256))]
    assert [n for _, n in steps(L, *qk(4100, 4096, 0, 264))] == [1 << 20, 1024]

    def logprobs(M, V, top_k):
        return ("qmt_logprobs", 1, P(), M, V, P(), top_k, P(), P(), P() if top_k else None, P() if top_k else None, P(), None)

    assert [n for _, n in steps(L, *logprobs((1 << 20) + 77, 9, 2))] == [1 << 20, 77]
    assert [k.split("<")[0] for k, _ in steps(L, *logprobs(1, 200000, 20))] == ["qmt_logprobs_part_kernel", "qmt_logprobs_join_kernel"]
    assert [k.split("<")[0] for k, _ in steps(L, *logprobs(2000, 131071, 5))] == ["qmt_logprobs_kernel"]


def test_edges_of_log_probabilities(L):
    """The rows of test_gpu_qmt_edges.py reach the kernels that they are meant for."""
    for M, want in zip(Q.PLANS, (["qmt_logprobs_part_kernel", "qmt_logprobs_join_kernel"], ["qmt_logprobs_kernel"])):
        assert [k.split("<")[0] for k, _ in steps(L, "qmt_logprobs", 0, P(), M, 5003, P(), 2, P(), P(), P(), P(), P(), None)] == want
    for M, V, parts in Q.LONG:
        got = steps(L, "qmt_logprobs", 0, P(), M, V, P(), 2, P(), P(), P(), P(), P(), None)
        assert got[0][0].split("<")[0] == "qmt_logprobs_kernel" and got[0][1] == M * parts and len(got) == 1 + (parts > 1)


def test_many_heads(L):
    """Every kernel that takes four heads a group, and only those, in the cases of test_gpu_qmt_edges.py with many."""
    t, seen = {"f32": 0, "bf16": 1, "f16": 2}, set()
    for (M, H, Hk), D, xt, yt, style in Q.HEADS:
        ((kernel, _),) = steps(L, *qk(M, H, Hk, D, t[xt], t[yt], Q.STYLES.index(style)))
        if M == Q.MANY[0]:
            seen.add(kernel)
        else:
            assert kernel.endswith(", 1, -1, -1, -1>")
    assert seen == {f"qmt_qk_norm_rope_kernel<{g}, 4, {x}, {y}, {s}>" for g in (4, 8, 16, 32, 64) for x in range(3) for y in range(3)
                    for s in range(2)}
