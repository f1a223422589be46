"""The plain forms that the GPU tests of drafted trees and of 8-bit rows compare with,
against written-out cases and torch, and the row plans of drafted trees (CPU only)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from . import tree_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
I32P = ctypes.POINTER(ctypes.c_int32)


def test_rows_of_a_written_out_tree():
    #        0   1  2  3  4  5
    tree = [-1, 0, 0, 1, 3, -1]
    table = np.array([[7, 3, -1]], np.int32)
    masks, positions, slots = tree_ref.tree_rows([tree], table, 5, [9], 16, 8, 2)
    assert masks[:, 0].tolist() == [1, 0b11, 0b101, 0b1011, 0b11011, 0b100000, 0, 0]
    assert not masks[:, 1].any()
    assert positions.tolist() == [14, 15, 15, 16, 17, 14, 0, 0]
    assert slots.tolist() == [7 * 16 + 14, 7 * 16 + 15, 3 * 16, 3 * 16 + 1, 3 * 16 + 2, 3 * 16 + 3,
                              -1, -1]
    near, _, _ = tree_ref.tree_rows([tree], table, 5, [9], 16, 6, 1, window=2)
    assert near[:, 0].tolist() == [1, 0b11, 0b101, 0b1010, 0b11000, 0b100000]


def test_path_of_a_written_out_tree():
    tree, draft = [-1, 0, 0, 2, 2, -1], [5, 6, 7, 9, 9, 5]
    # 0 (lowest of two drafted as 5), then 2, then 3 (lowest of two drafted as 9), then none
    path, counts, after = tree_ref.accept([tree], draft, [7, 0, 9, 1, 2, 3], [5], 7)
    assert path.tolist() == [0, 2, 3, -1, -1, -1, -1] and counts.tolist() == [3] and after.tolist() == [1]
    path, counts, after = tree_ref.accept([tree], draft, [7, 0, 9, 1, 2, 3], [4], 6)
    assert path.tolist() == [-1] * 6 and counts.tolist() == [0] and after.tolist() == [4]


@pytest.mark.parametrize("gs", [1.0, 0.25, 0.07, 3.0])
def test_8_bit_values_are_torchs(gs):
    """Every bf16 number, against torch's own conversion of the saturated quotient."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    want = (x / torch.tensor(gs)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    got = tree_ref.encode8(x.numpy(), gs)
    assert np.array_equal(got, want.view(torch.uint8).numpy())
    assert np.array_equal(tree_ref.decode8(got, gs),
                          want.double().numpy() * float(np.float32(gs)))


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("treeplan") / "tree_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I/usr/local/cuda/include",
                    os.path.join(ROOT, "tests", "tree_plan.cpp"),
                    os.path.join(ROOT, "shared_prefix_fan_gb300", "csrc", "plan.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so).tree_plan


def plan(shim, S, T, P, hq, hkv, page, window=0, sinks=0, prev=None, splits=0, row_bytes=256,
         tree=1):
    """S counts the drafted tokens, as the attention calls do."""
    S, T = np.asarray(S, np.int32), np.asarray(T, np.int32)
    prev = None if prev is None else np.asarray(prev, np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(I32P)  # noqa: E731
    units, R = np.zeros((50000, 8), np.int32), int(T.sum())
    pos, info = np.zeros(max(2 * R, 1), np.int32), np.zeros(6, np.int32)
    n = shim(ptr(prev), ptr(S), ptr(T), len(S), P, hq, hkv, page, window, sinks, splits, row_bytes,
             tree, ptr(units), len(units), ptr(pos), ptr(info))
    assert 0 <= n <= len(units)
    return units[:n], pos[:R], pos[R:2 * R], info


def check_plan(shim, S, T, P, hq, hkv, page, window=0, sinks=0, **kw):
    """Every key that a row may see is swept once: the keys before the draft by window and
    first keys, at every depth a tree can have, and all drafted ones."""
    units, base, own, info = plan(shim, S, T, P, hq, hkv, page, window, sinks, **kw)
    split_at, rows = int(info[0]), [(b, i) for b, t in enumerate(T) for i in range(t)]
    for r, (b, i) in enumerate(rows):
        assert base[r] == P + S[b] - T[b] and own[r] == base[r] + i
    swept = {(r, h): np.zeros(P + max(S), np.int32) for r in range(len(rows)) for h in range(hkv)}
    for h, b, t0, nt, kb, ke, first_end, _ in units.tolist():
        runs = [(kb, ke)]
        if first_end:
            runs.append((split_at if kb >= split_at else 0, first_end))
        for lo, hi in runs:
            assert lo < hi
            for r in range(t0, t0 + nt):
                assert rows[r][0] == b or (split_at and hi <= split_at)
                swept[(r, h)][lo:hi] += 1
    for r, (b, i) in enumerate(rows):
        j = np.arange(P + S[b])
        may = j < base[r]
        if window:  # position base .. : the oldest key is that of a token without a parent
            may = may & ((j > base[r] - window) | (j < sinks))
        may = may | (j >= base[r])
        for h in range(hkv):
            n = swept[(r, h)][:P + S[b]]
            assert (n[may] == 1).all() and (n <= 1).all() and not swept[(r, h)][P + S[b]:].any()
    return units, info


@pytest.mark.parametrize("seed", range(30))
def test_tree_plans_sweep_every_key_once(shim, seed):
    rng = np.random.default_rng(seed)
    page, hkv = int(rng.choice([16, 32, 64, 128])), int(rng.choice([1, 2]))
    hq = hkv * int(rng.choice([1, 4, 7, 8]))
    B, P = int(rng.integers(1, 6)), int(rng.integers(0, 900))
    T = rng.integers(0, 40, size=B)
    if seed % 5 == 0:
        T[0] = 300  # more than a unit of rows, more than two tiles of drafted keys
    if not T.any():
        T[0] = 3
    S = T + rng.integers(0, 500, size=B)
    window, sinks = (0, 0) if seed % 3 == 0 else (int(rng.integers(1, 400)), int(rng.integers(0, 40)))
    check_plan(shim, S.tolist(), T.tolist(), P, hq, hkv, page, window, sinks,
               splits=int(rng.choice([0, 0, 1, 3])))


CUT = [  # (S, T, P, H_q, H_kv, page, window, sinks): row blocks that hold one branch only
    ([100 + 40 * b for b in range(8)], [32] * 8, 16384, 64, 8, 64, 0, 0),
    ([700, 90, 333], [64, 32, 31], 5000, 16, 2, 16, 0, 0),
    ([100 + 40 * b for b in range(8)], [32] * 8, 16384, 64, 8, 64, 8192, 4),
    ([40, 900], [96, 160], 9000, 32, 4, 128, 3000, 300)]


@pytest.mark.parametrize("case", CUT)
def test_branches_that_sweep_the_prefix_themselves_are_cut(shim, case):
    units, info = check_plan(shim, [s + t for s, t in zip(case[0], case[1])], *case[1:])
    assert info[0] == 0 and info[3] > 0  # no shared range, and partials
    moved = [s + t + 1 for s, t in zip(case[0], case[1])]
    check_plan(shim, moved, *case[1:], prev=[s - 1 for s in moved])


@pytest.mark.parametrize("case", CUT)
def test_cut_causal_plans_sweep_every_key_once(shim, case):
    S, T, P, hq, hkv, page, window, sinks = case
    S = [s + t for s, t in zip(S, T)]
    kept = 0
    for prev in [None] + [[s - i for s in S] for i in (1, 2, 3, 5, 8)]:
        units, pos, _, info = plan(shim, S, T, P, hq, hkv, page, window, sinks, prev=prev, tree=0)
        kept += int(info[4])
        assert info[0] == 0 and info[3] > 0
        swept = np.zeros((sum(T), hkv, P + max(S)), np.int32)
        rows = [(b, i) for b, t in enumerate(T) for i in range(t)]
        for h, b, t0, nt, kb, ke, first_end, _ in units.tolist():
            assert all(rows[r][0] == b for r in range(t0, t0 + nt))
            swept[t0:t0 + nt, h, kb:ke] += 1
            swept[t0:t0 + nt, h, :first_end] += 1
        for r, (b, i) in enumerate(rows):
            assert pos[r] == P + S[b] - T[b] + i
            j = np.arange(P + max(S))
            may = (j <= pos[r]) & ((j > pos[r] - window) | (j < sinks) if window else True)
            assert (swept[r, :, may] == 1).all() and (swept[r] <= 1).all()
            assert not swept[r, :, P + S[b]:].any()
    assert kept > 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 4)])
def test_tree_plans_move_with_the_suffixes(shim, window, sinks):
    """A plan carried over to longer suffixes sweeps what a new one does."""
    kept = 0
    for step in range(1, 40):
        prev = [40 + 8, 60 + 20]
        S = [prev[0] + step, prev[1] + 2 * step]
        _, info = check_plan(shim, S, [8, 20], 256, 8, 1, 16, window, sinks, prev=prev)
        kept += int(info[4])
    assert kept > 0


def test_ragged_windows_are_swept_whole(shim):
    """Windows that reach little of the prefix: no shared range, and no partials."""
    rng = np.random.default_rng(2)
    T = rng.integers(1, 33, size=32).tolist()
    S = [int(t + s) for t, s in zip(T, rng.integers(64, 4096, size=32))]
    units, info = check_plan(shim, S, T, 16384, 64, 8, 16, 2048, 16)
    assert info[0] == 0 and info[3] == 0
