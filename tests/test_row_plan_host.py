"""Row plans (windowed and 4-bit attention) on the host: every visible (row, key)
pair is swept by exactly one unit, and no page is read that no row of the call
sees (CPU only)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32P = ctypes.POINTER(ctypes.c_int32)


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rowplan") / "row_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I/usr/local/cuda/include",
                    os.path.join(ROOT, "tests", "row_plan.cpp"),
                    os.path.join(ROOT, "shared_prefix_fan_gb300", "csrc", "plan.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so).row_plan


def make(shim, S, T, P, hq, hkv, page, causal=1, window=0, sinks=0, prev=None, splits=0, sms=152,
         row_bytes=512):
    S, T = np.asarray(S, np.int32), np.asarray(T, np.int32)
    prev = None if prev is None else np.asarray(prev, np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(I32P)  # noqa: E731
    cap = 200000
    units = np.zeros((cap, 8), np.int32)
    pos, info = np.zeros(max(int(T.sum()), 1), np.int32), np.zeros(8, np.int32)
    cnt = np.zeros(max(int(T.sum()) * hkv, 1), np.int32)
    n = shim(ptr(prev), ptr(S), ptr(T), len(S), P, hq, hkv, page, causal, window, sinks, sms,
             splits, row_bytes, ptr(units), cap, ptr(pos), ptr(info), ptr(cnt))
    assert 0 <= n <= cap
    return units[:n], pos[:int(T.sum())], info, cnt


def visible(S, T, P, causal, window, sinks):
    """Per row: (branch, mask of visible keys)."""
    rows = []
    for b, (s, t) in enumerate(zip(S, T)):
        j = np.arange(P + s)
        for i in range(t):
            pos = P + s - t + i
            see = j <= pos if causal else j >= 0
            if window:
                see = see & ((j > pos - window) | (j < sinks))
            rows.append((b, see))
    return rows


def check(shim, S, T, P, hq, hkv, page, causal=1, window=0, sinks=0, **kw):
    units, pos, info, cnt = make(shim, S, T, P, hq, hkv, page, causal, window, sinks, **kw)
    split_at = int(info[0])
    rows = visible(S, T, P, causal, window, sinks)
    seen = {(r, h): np.zeros(len(m), np.int32) for r, (_, m) in enumerate(rows) for h in range(hkv)}
    pages_ok = {}
    for r, (b, m) in enumerate(rows):
        keys = np.nonzero(m)[0]
        pages_ok.setdefault(b, set()).update((keys // page).tolist())
    shared_ok = set().union(*pages_ok.values()) if pages_ok else set()
    parts = np.zeros(len(rows) * hkv, np.int32)
    for h, b, t0, nt, kb, ke, first_end, part in units.tolist():
        assert nt >= 1 and nt <= int(info[1]) * int(info[2])
        base = split_at if kb >= split_at else 0
        begin = kb // page * page
        assert base <= begin <= kb < ke
        runs = [(begin, ke, True)]
        if first_end:
            assert base < first_end <= begin + page
            runs.insert(0, (base, first_end, False))
        for lo, hi, main in runs:
            allowed = shared_ok if (split_at and lo < split_at) else pages_ok[b]
            assert set(range(lo // page, (hi - 1) // page + 1)) <= allowed
            for r in range(t0, t0 + nt):
                rb, m = rows[r]
                assert rb == b or (split_at and hi <= split_at)
                j = np.arange(lo, hi)
                p = int(pos[r])
                use = j <= p
                if window:
                    use &= (j > p - window) | ((j < sinks) & (not main or first_end == 0))
                use &= j >= (kb if main else lo)  # keys before are zeroed and hidden
                hidden_front = (j < kb) & (j > p - window) if (main and window) else j < lo
                assert not hidden_front.any()
                seen[(r, h)][j[use]] += 1
        if part >= 0:
            for r in range(t0, t0 + nt):
                parts[r * hkv + h] += 1
    for r, (_, m) in enumerate(rows):
        for h in range(hkv):
            assert np.array_equal(seen[(r, h)], m.astype(np.int32)), (r, h)
    if int(info[3]):
        assert np.array_equal(parts, cnt[:len(parts)])
    return units, info


@pytest.mark.parametrize("seed", range(40))
def test_every_visible_pair_once(shim, seed):
    rng = np.random.default_rng(seed)
    page = int(rng.choice([16, 32, 64, 128]))
    hkv = int(rng.choice([1, 2]))
    hq = hkv * int(rng.choice([1, 4, 7, 8]))
    B = int(rng.integers(1, 7))
    P = int(rng.integers(0, 900))
    T = rng.integers(0, 40, size=B)
    S = T + rng.integers(0, 300, size=B)
    if int(T.sum()) == 0:
        T[0], S[0] = 1, S[0] + 1
    window = int(rng.choice([0, 1, 2, 15, 64, 200, 700, 5000]))
    sinks = int(rng.choice([0, 1, 4, 130, 1000])) if window else 0
    check(shim, S, T, P, hq, hkv, page, 1, window, sinks, splits=int(rng.choice([0, 0, 1, 3])),
          sms=int(rng.choice([8, 152])), row_bytes=int(rng.choice([144, 512])))


@pytest.mark.parametrize("T,S", [([3, 2], [0, 5]), ([1], [0]), ([0, 4], [7, 1])])
def test_not_causal(shim, T, S):
    check(shim, S, T, 100, 8, 2, 16, causal=0)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (300, 0), (40, 20)])
def test_patched_plans_stay_right(shim, window, sinks):
    """A decode loop: each step's plan carried over from the step before when it can be."""
    S, T = np.array([70, 33, 120]), np.array([1, 1, 1])
    kept = 0
    for _ in range(40):
        units, info = check(shim, S + 1, T, 256, 8, 2, 16, 1, window, sinks, prev=S)
        kept += int(info[4])
        S = S + 1
    assert kept > 20


def test_window_that_stays_private_is_one_unit(shim):
    """No window reaches the prefix: the first keys ride in the same unit, written directly."""
    units, info = check(shim, [500, 600], [1, 1], 4096, 8, 1, 64, 1, 256, 4, splits=1)
    assert int(info[0]) == 0 and int(info[3]) == 0 and len(units) == 2
    assert (units[:, 6] == 4).all()


def test_short_contexts_need_no_merge(shim):
    """A few tiles of keys: every branch sweeps its own; a long prefix stays shared.
    Steps carry either plan over."""
    for prev in (None, [20, 30, 10]):
        S = [21, 31, 11]
        units, info = check(shim, S, [1, 1, 1], 256, 16, 2, 16, prev=prev, row_bytes=144)
        assert int(info[0]) == 0 and int(info[3]) == 0 and len(units) == 6
        assert prev is None or int(info[4]) == 1
        units, info = check(shim, S, [1, 1, 1], 2048, 16, 2, 16, prev=prev, row_bytes=144)
        assert int(info[0]) == 2048 and int(info[3]) > 0
    units, info = check(shim, [500, 20], [40, 3], 200, 8, 1, 16, window=90, sinks=5)
    assert int(info[0]) in (0, 192)
