"""Positions of drafted tokens that no forest has: every token levels behind its context, and
values past the deepest tree. Which cached keys may then hold anything."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import tree_ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "q4", "q8"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def problem(kind, levels, P=300, S=(300, 20), T=(6, 40), window=150, sinks=5, page=16):
    """Every drafted token `levels` further behind its context than its depth. Keys that a
    token right behind the context would not see hold NaN, their pages are no pages."""
    rng = np.random.default_rng(levels + page)
    prob = tree_ref.Problem(list(S), list(T), P, 16, 2, page, kind=kind, window=window, sinks=sinks,
                            trees=[tree_ref.random_tree(rng, t) for t in T], seed=levels)
    prob.positions = prob.positions + np.int32(levels)
    see = []
    for r, (b, m) in enumerate(prob.see):
        n = P + S[b]
        j, m = np.arange(n), m.copy()
        m[:n] = (j > prob.positions[r] - window) | (j < sinks)
        see.append((b, m))
    assert any((a[1] != b[1]).any() for a, b in zip(see, prob.see))
    prob.see = see
    return prob


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("levels,page", [(1, 16), (40, 64), (149, 16), (700, 32)])
def test_keys_in_front_of_the_window_at_the_context_may_hold_anything(kind, levels, page):
    """(A window of which nothing but the drafted tokens is left, too.)"""
    prob = problem(kind, levels, page=page)
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    prob.check(out, lse)


def test_keys_behind_it_are_read_whatever_the_positions_say():
    """What the header asks of the caller: here a page in a window that no position leaves
    visible is none."""
    prob = problem("bf16", 149, sinks=0)
    page = (300 + 300 - 100) // 16  # of the first branch: hidden from all of its rows
    assert not any(m[page * 16:page * 16 + 16].any() for b, m in prob.see if b == 0)
    prob.args()[3][0, page] = -1
    prob.run()
    assert binding.last_error() == binding.EINVAL


@pytest.mark.parametrize("kind", KINDS)
def test_positions_past_the_deepest_tree_count_as_its_end(kind):
    rng = np.random.default_rng(4)
    prob = tree_ref.Problem([300, 200], [6, 9], 1500, 16, 2, 16, kind=kind, window=1200, sinks=2, seed=4,
                            trees=[tree_ref.random_tree(rng, t) for t in (6, 9)])
    base = np.repeat([1800, 1700], [6, 9])
    got = []
    for positions in (base + 1023, np.full(15, 2 ** 31 - 1), base + 1024, base + 1022):
        prob.args()[5].copy_(torch.from_numpy(positions.astype(np.int32)))
        got.append(prob.run())
        assert binding.last_error() == binding.OK
    for out, lse in got[1:3]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert not torch.equal(got[3][0], got[0][0])  # (a key more)
    prob.see = [(b, np.concatenate([(np.arange(n) > n + 1023 - 1200) | (np.arange(n) < 2), m[n:]]))
                for (b, m), n in zip(prob.see, base)]
    prob.check(*got[0])
