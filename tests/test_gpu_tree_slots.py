"""Slots of drafted rows against those of the extension that gave them their pages."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import tree_ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("B,t_hi,P,page", [(1, 1, 0, 16), (9, 20, 37, 16), (5, 300, 64, 32), (64, 40, 100, 128)])
def test_slots_are_those_of_the_extension(B, t_hi, P, page):
    """Pages for the drafted tokens from a shuffled free list: page and place of every row."""
    rng = np.random.default_rng(B + t_hi)
    T = rng.integers(0, t_hi + 1, size=B)
    T[0] = t_hi
    S = rng.integers(0, 60, size=B)
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    held = [-(-(P + int(s)) // page) for s in S]
    width = max(-(-(P + int(s + t)) // page) for s, t in zip(S, T)) + 1
    ids = rng.permutation(int(sum(held)) + B * (t_hi // page + 2))
    table, at = np.full((B, width), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    table, R = dev(table), int(T.sum())
    want, used = binding.extend_device(table, P, dev(S), dev(T), page, dev(ids[at:]), R)
    parents = dev([p for t in T for p in tree_ref.random_tree(rng, int(t))])
    _, _, slots = binding.tree_rows(parents, table, P, dev(S), dev(T), page, t_hi)
    assert binding.last_error() == binding.OK
    assert torch.equal(slots, want)
    assert int(used) == sum(-(-(P + int(s + t)) // page) for s, t in zip(S, T)) - sum(held)
    assert (slots >= 0).all() and slots.unique().numel() == R
