"""K and V rows that a call reads out of a cache: outputs that share bytes are refused, rows
of one array between those of the other are not (CPU only)."""
import ctypes
import os
import random
import subprocess

import pytest

from shared_prefix_fan_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from shared_prefix_fan_gb300 import build
    build.build()
    return binding.load()


# 4 rows of 2 heads (512 bytes) into made-up addresses; each call is refused
READ = dict(kp=0x100000, vp=0x200000, slots=0x3000, n=4, pages=9, hkv=2, d=128, ps=16, kscale=1.0,
            vscale=1.0, k=0x10000, v=0x20000, ks=256, vs=256, stream=None)


@pytest.mark.parametrize("name", ["q4", "q8"])
@pytest.mark.parametrize("kw", [
    dict(v=0x10000), dict(v=0x10000 + 0x7f0), dict(v=0x10000 - 0x7f0), dict(v=0x10200),
    dict(ks=512, vs=512, v=0x10000 + 0x1f0), dict(ks=512, vs=512, v=0x10000 - 0x1f0),
    dict(ks=512, vs=520, v=0x10200),  # between each other, but for the last rows
    dict(ks=2 ** 40, vs=2 ** 40), dict(n=1, ks=2 ** 60, vs=2 ** 60, v=0x101f0)])
def test_outputs_over_each_other_are_refused(lib, name, kw):
    a = {**READ, **kw}
    if "v" not in kw:
        a["v"] = a["k"] + 16
    assert getattr(lib, f"fanout_kv_read_{name}")(*a.values()) == binding.EINVAL


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rows") / "rows_overlap.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I/usr/local/cuda/include",
                    os.path.join(ROOT, "tests", "rows_overlap.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).rows_share
    u64, i64 = ctypes.c_uint64, ctypes.c_int64
    f.argtypes, f.restype = [u64, i64, u64, i64, i64, i64], ctypes.c_int
    return f


@pytest.mark.parametrize("seed", range(8))
def test_against_the_bytes_themselves(share, seed):
    r = random.Random(seed)
    found = [0, 0]
    for _ in range(4000):
        row, n = r.randint(1, 12), r.randint(1, 9)
        s, t = (row + r.choice([0, 1, row, row + 1, 3 * row, r.randint(0, 40)]) for _ in range(2))
        if r.random() < 0.5:
            t = s
        a, b = 1000, 1000 + r.randint(-300, 300)
        of = lambda at, step: {at + 2 * step * i + x for i in range(n) for x in range(2 * row)}  # noqa: E731
        want = not of(a, s).isdisjoint(of(b, t))
        assert share(a, s, b, t, n, row) == want, (a, s, b, t, n, row)
        found[want] += 1
    assert min(found) > 500


def test_large_arrays(share):
    far = (1 << 40, 2 ** 60, (1 << 40) + 256, 2 ** 60, 2 ** 30, 128)
    assert share(*far) == 0 and share(*far[:5], 129) == 1
    assert share(0, 256, 2 * 128, 256, 2 ** 20, 128) == 0  # every second half row
    assert share(0, 256, 2 * 127, 256, 2 ** 20, 128) == 1
    assert share(0, 384, 256, 392, 2 ** 20, 128) == 1  # drifts into it
