"""The planner prices every candidate by the tiles its units sweep, the first keys'
tiles among them (CPU only)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32P, F64P = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rowcost") / "row_plan_cost.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I/usr/local/cuda/include",
                    os.path.join(ROOT, "tests", "row_plan_cost.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so).row_plan_cost


def price(shim, S, T, P, hq, hkv, page, window, sinks, sms=152, row_bytes=512, chunk=4):
    S, T = np.asarray(S, np.int32), np.asarray(T, np.int32)
    out = [np.zeros(3) for _ in range(3)] + [np.zeros(1)]
    rc = shim(*(a.ctypes.data_as(I32P) for a in (S, T)), len(S), P, hq, hkv, page, 1, window, sinks,
              sms, row_bytes, chunk, *(a.ctypes.data_as(F64P) for a in out))
    assert rc == 0
    return out


CASES = [  # S, T, P, window, sinks
    ([512] * 24, [16] * 24, 16384, 1024, 1024), ([1] * 8, [1] * 8, 32768, 4096, 2048),
    ([4096], [4096], 4096, 1024, 4), ([4096], [4096], 4096, 1024, 900),
    ([300, 2000, 50], [3, 1, 30], 900, 256, 130), ([700] * 5, [700] * 5, 0, 100, 300),
    ([512] * 8, [1] * 8, 32768, 4096, 4), ([512] * 8, [1] * 8, 32768, 0, 0),
    (list(range(64, 4096, 130)), [1 + i % 32 for i in range(32)], 16384, 2048, 16),
]


@pytest.mark.parametrize("S,T,P,window,sinks", CASES)
@pytest.mark.parametrize("page,sms,chunk", [(64, 152, 4), (16, 152, 10), (64, 20, 2)])
def test_cost_is_the_busiest_cta_and_the_merge(shim, S, T, P, window, sinks, page, sms, chunk):
    cost, load, merge, _ = price(shim, S, T, P, 64, 8, page, window, sinks, sms=sms, chunk=chunk)
    assert np.allclose(cost, load + merge, rtol=1e-12), (cost, load + merge)


@pytest.mark.parametrize("S,T,P,window,sinks", CASES)
def test_chosen_plan_is_no_worse_than_equal_chunks(shim, S, T, P, window, sinks):
    """By the same account: no candidate of equal chunks may have a busiest CTA so much
    shorter that its whole cost would have been the smaller one by the planner's margin."""
    for row_bytes in (144, 512):
        best = np.inf
        for chunk in (0, 2, 3, 4, 6, 8, 10, 12, 16, 24, 32):
            cost, load, merge, chosen = price(shim, S, T, P, 64, 8, 64, window, sinks, chunk=chunk,
                                              row_bytes=row_bytes)
            best = min(best, load[0] + merge[0])
        assert chosen[0] <= best / 0.97
