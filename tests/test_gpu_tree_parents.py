"""Parents out of range mean the same to every call of a drafting step."""
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


def dev(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


@pytest.mark.parametrize("first,want", [(7, [1]), (5, [0, 4]), (9, [2, 3]), (4, [])])
def test_bad_parents_are_roots_to_both_calls(first, want):
    """Tokens 1 (its own parent), 2 (a later one) and 3 (below -1) count as roots."""
    parents = dev([-1, 1, 5, 2, 0, -7], torch.int32)
    draft, target = [5, 7, 9, 3, 8, 6], [8, 1, 3, 0, 2, 0]
    lens, table = dev([6], torch.int32), dev(np.arange(8)[None], torch.int32)
    masks, positions, _ = binding.tree_rows(parents, table, 0, dev([10], torch.int32), lens, 16, 6)
    assert binding.last_error() == binding.EINVAL
    assert masks[:, 0].tolist() == [1, 2, 4, 12, 17, 32] and positions.tolist() == [10, 10, 10, 11, 11, 10]
    path, counts, after = binding.tree_accept(parents, dev(draft, torch.int64), dev(target, torch.int64),
                                              dev([first], torch.int64), lens)
    assert binding.last_error() == binding.EINVAL
    assert path.tolist() == want + [-1] * (6 - len(want)) and counts.tolist() == [len(want)]
    assert after.tolist() == [target[want[-1]] if want else first]


@pytest.mark.parametrize("seed", range(6))
def test_random_bad_parents(seed):
    rng = np.random.default_rng(seed)
    trees = [tree_ref.random_tree(rng, int(t)) for t in rng.integers(0, 200, size=5)]
    bad = [[p if rng.random() < 0.7 else int(rng.choice([t, t + 1, 5000, -2, -2 ** 31])) for t, p in enumerate(x)]
           for x in trees]
    good = [[p if -1 <= p < t else -1 for t, p in enumerate(x)] for x in bad]
    assert bad != good
    R = sum(len(x) for x in trees)
    draft, target, first = (rng.integers(0, 3, size=n) for n in (R, R, 5))
    tok = [dev(x, torch.int64) for x in (draft, target, first)]
    path, counts, after = binding.tree_accept(dev([p for x in bad for p in x], torch.int32), *tok,
                                              dev([len(x) for x in trees], torch.int32))
    assert binding.last_error() == binding.EINVAL
    p, c, n = tree_ref.accept(good, draft, target, first, R)
    assert np.array_equal(path.cpu().numpy(), p) and np.array_equal(counts.cpu().numpy(), c)
    assert np.array_equal(after.cpu().numpy(), n)
