"""On the host (no GPU needed): a kernel that is launched with more than 64 KB
of LDS has been given as much on the device of the launch, whichever device
the process used first.
"""
import pytest

import launches
from launches import P

DEFAULT = 64 * 1024                                            # dynamic LDS that needs no attribute


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    with launches.Launches(tmp_path_factory.mktemp("recorder")) as l:
        yield l


def calls():
    """(name, entry, arguments) that reach every kernel family with its largest LDS."""
    yield from ((f"mx4 dense {M} {N} {K}", "qmv_dense", (0, P(), P(), 4, P(), P(), P(), M, N, K, None))
                for M, N, K in ((16, 100, 16384), (64, 13000, 16384), (600, 7000, 544)))
    for M, E, top_k, N, K in ((4, 8, 4, 100, 16384), (60, 40, 2, 300, 16384), (150, 4, 4, 96, 3584), (40, 8, 2, 100, 16384)):
        yield f"mx4 gather {M} {K}", "qmv_gather_moe", (0, P(), P(), E, P(), M, top_k, 4, P(), P(), 0, P(), N, K, None)
        yield (f"mx4 swiglu {M} {K}", "qmv_gather_moe_swiglu",
               (0, P(), P(), P(), P(), E, P(), M, top_k, 4, P(), P(), P(), N, K, None))
        yield (f"mx4 combine {M} {K}", "qmv_gather_moe_combine",
               (0, P(), P(), E, P(), P(), M, top_k, 4, P(), P(), 1, P(), N, K, None))
    for wfmt in (0, 1, 2):
        for afmt in ((0, 1) if wfmt == 0 else (1, 2)):
            xs = P() if afmt == 1 else None
            for M in (1, 4, 8, 16, 64, 200):
                for N in (1000, 8192):
                    yield f"dense {wfmt} {afmt} {M} {N}", "qmv_dense", (wfmt, P(), P(), afmt, P(), xs, P(), M, N, 16384, None)
            for M, E in ((1, 64), (4, 64), (20, 1000), (200, 64), (500, 8)):
                for K in (16384, 2880):
                    a = (M, 4, afmt, P(), xs)
                    yield f"gather {wfmt} {afmt} {M} {K}", "qmv_gather_moe", (wfmt, P(), P(), E, P(), *a, 0, P(), 2880, K, None)
                    yield (f"swiglu {wfmt} {afmt} {M} {K}", "qmv_gather_moe_swiglu",
                           (wfmt, P(), P(), P(), P(), E, P(), *a, P(), 2880, K, None))
                    yield (f"combine {wfmt} {afmt} {M} {K}", "qmv_gather_moe_combine",
                           (wfmt, P(), P(), E, P(), P(), *a, 1, P(), 2880, K, None))


def test_every_device_has_its_own_lds_limits(L):
    limit, large = {}, set()
    for device in (0, 1, 0):
        for what, entry, args in calls():
            status, lines = L.lines(entry, *args, device=device)
            assert status == 0, (what, status)
            for kind, dev, kernel, *v in lines:
                if kind == "attr":
                    limit[int(dev), kernel] = int(v[0])
                elif int(v[4]) > DEFAULT:
                    large.add(launches.short(kernel).split("<")[0])
                    assert limit.get((int(dev), kernel), 0) >= int(v[4]), (what, dev, launches.short(kernel), v)
    assert {"qmv_mx4_few_kernel", "qmv_mx4_tile_kernel", "qmv_mx4_wide_kernel", "qmv_gmma_kernel"} <= large, large


def test_limits_are_set_once(L):
    for what, entry, args in calls():
        assert not [l for l in L.lines(entry, *args, device=1)[1] if l[0] == "attr"], what
