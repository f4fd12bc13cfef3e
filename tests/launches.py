"""Which kernels a library call launches, on the host: the library runs in a
process of its own against the stand-in runtime of hip_recorder.cpp (256
compute units), with pointers that nothing dereferences.

    with Launches(tmp_path) as L:
        L.call("qmv_dense", 0, P(), P(), 4, P(), P(), P(), M, N, K, None)
        -> [Launch(device, kernel, grid, threads, lds)]
"""
import collections
import json
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
F = 0x10000                                                    # an aligned address

Launch = collections.namedtuple("Launch", "device kernel grid threads lds")

SERVER = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
rec.rec_lines.restype = ctypes.c_char_p
libs = [ctypes.CDLL(p) for p in sys.argv[2:]]
for line in sys.stdin:
    device, name, args = json.loads(line)
    rec.hipSetDevice(device)
    rec.rec_clear()
    fn = next(getattr(l, name) for l in libs if hasattr(l, name))
    put = [ctypes.c_void_p(None) if a is None else ctypes.c_void_p(int(a[1:])) if isinstance(a, str) else
           ctypes.c_float(a) if isinstance(a, float) else ctypes.c_longlong(a) for a in args]
    print(json.dumps([fn(*put), rec.rec_lines().decode()]), flush=True)
"""


def short(mangled):
    """qmv_mx4_tile_kernel<0, 64> of its mangled name."""
    m = re.search(r"\d(qm[vx]_[a-z0-9_]*?_kernel)(?:I((?:L[a-z]\d+E)*))?", mangled)
    if not m:
        return mangled
    args = re.findall(r"L[a-z](\d+)E", m.group(2) or "")
    return m.group(1) + (f"<{', '.join(args)}>" if args else "")


class Launches:
    def __init__(self, tmp_path):
        so = str(tmp_path / "hip_recorder.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        os.path.join(HERE, "hip_recorder.cpp"), "-o", so], check=True)
        pkg = os.path.join(ROOT, "bit_block_quantized_amd")
        self.p = subprocess.Popen([sys.executable, "-c", SERVER, so, os.path.join(pkg, "libqmv.so"),
                                   os.path.join(pkg, "libqmx.so")], stdin=subprocess.PIPE, stdout=subprocess.PIPE, text=True)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.p.stdin.close()
        self.p.wait(30)

    def lines(self, name, *args, device=0):
        """(status, recorded lines) of a call; addresses are given as P(int)."""
        self.p.stdin.write(json.dumps([device, name, list(args)]) + "\n")
        self.p.stdin.flush()
        out = self.p.stdout.readline()
        assert out, "the process with the stand-in runtime ended"
        status, text = json.loads(out)
        return status, [l.split() for l in text.splitlines()]

    def call(self, name, *args, device=0):
        status, lines = self.lines(name, *args, device=device)
        assert status == 0, (name, args, status)
        return [Launch(int(l[1]), short(l[2]), tuple(int(v) for v in l[3:6]), int(l[6]), int(l[7]))
                for l in lines if l[0] == "launch"]


def P(address=F):
    """An address as an argument (a plain number is an int)."""
    return f"@{address}"


MXFP4, A_MXFP4 = 0, 4


def mx4_dense(L, M, N, K, **kw):
    return L.call("qmv_dense", MXFP4, P(), P(), A_MXFP4, P(), P(), P(), M, N, K, None, **kw)


def mx4_gather(L, M, E, top_k, N, K, per_slot=False, **kw):
    return L.call("qmv_gather_moe", MXFP4, P(), P(), E, P(), M, top_k, A_MXFP4, P(), P(), int(per_slot), P(), N, K, None,
                  **kw)


def mx4_swiglu(L, M, E, top_k, N, K, **kw):
    return L.call("qmv_gather_moe_swiglu", MXFP4, P(), P(), P(), P(), E, P(), M, top_k, A_MXFP4, P(), P(), P(), N, K, None,
                  **kw)


def mx4_combine(L, M, E, top_k, N, K, per_slot=True, entry="qmv_gather_moe_combine", **kw):
    return L.call(entry, MXFP4, P(), P(), E, P(), P(), M, top_k, A_MXFP4, P(), P(), int(per_slot), P(), N, K, None, **kw)
