"""First keys that stay visible among the drafted tokens: masks against a plain form, and
chains of drafts against what decoding their tokens one by one sees."""
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def deep(rng, T):
    return [-1] + [max(0, t - 1 - int(rng.integers(0, 3))) for t in range(1, T)] if T else []


@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 7), (2, 4), (5, 40), (31, 33), (32, 64), (33, 100),
                                          (70, 2 ** 31 - 1), (2 ** 31 - 1, 9), (3, 0), (1, 1100)])
def test_masks(window, sinks):
    """Contexts shorter and longer than `sinks`, ancestors over many words of 32 tokens."""
    rng = np.random.default_rng(window % 1000 + sinks % 1000)
    trees = [list(range(-1, 1023)), deep(rng, 700), [-1] * 40, [-1] + [0] * 99, list(range(-1, 63)), [],
             tree_ref.random_tree(rng, 300), [-1]]
    S, T, P = [0, 3, 17, 0, 40, 5, 1, 200], [len(t) for t in trees], 2
    table = np.arange(len(T) * 80).reshape(len(T), 80)
    masks, positions, slots = binding.tree_rows(i32(np.concatenate(trees)), i32(table), P, i32(S), i32(T),
                                                16, 1024, window, sinks=sinks)
    assert binding.last_error() == binding.OK
    bits = np.unpackbits(masks.cpu().numpy().view(np.uint8), axis=1, bitorder="little").astype(bool)
    row = 0
    for b, (tree, s) in enumerate(zip(trees, S)):
        for t in range(len(tree)):
            line, depth = tree_ref.lineage(tree, t)
            want = np.zeros(1024, bool)
            for levels, u in enumerate(line):
                want[u] = levels < window or P + s + depth - levels < sinks
            assert np.array_equal(bits[row], want), (b, t)
            assert int(positions[row]) == P + s + depth
            key = P + s + t
            assert int(slots[row]) == table[b][key // 16] * 16 + key % 16
            row += 1


def test_captured_masks():
    rng = np.random.default_rng(3)
    trees = [deep(rng, 50), deep(rng, 9)]
    a = (i32(np.concatenate(trees)), i32(np.arange(20).reshape(2, 10)), 3)
    S, T = i32([0, 4]), i32([50, 9])
    binding.tree_rows(*a, S, T, 16, 50, 4, sinks=12)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m = binding.tree_rows(*a, S, T, 16, 50, 4, sinks=12)
    for s in ([0, 4], [9, 0], [40, 7]):
        S.copy_(i32(s))
        g.replay()
        want = binding.tree_rows(*a, S, T, 16, 50, 4, sinks=12)
        assert all(torch.equal(x, y) for x, y in zip(m, want))


CHAINS = [  # suffixes without the drafts, drafts, prefix, window, sinks
    ([0], [4], 2, 2, 4), ([0], [40], 1, 1, 8), ([0, 3], [12, 9], 5, 3, 10), ([5, 0], [33, 64], 0, 16, 40),
    ([30, 90], [20, 30], 40, 7, 60), ([0], [300], 3, 20, 200), ([300, 20], [9, 30], 200, 16, 4)]


@pytest.mark.parametrize("kind", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("case", CHAINS)
def test_a_chain_sees_what_decoding_sees(kind, case):
    """Drafted tokens in order, whose context may be shorter than the first keys."""
    S, T, P, window, sinks = case
    prob = tree_ref.Problem([s + t for s, t in zip(S, T)], T, P, 16, 2, 16, kind=kind, window=window,
                            sinks=sinks, seed=sum(T))
    q, k, v, table = prob.args()
    parents = np.concatenate([np.arange(-1, t - 1) for t in T])
    masks, positions, _ = binding.tree_rows(i32(parents), i32(prob.table), P, i32(S), i32(T), 16, max(T),
                                            window, sinks=sinks)
    out, lse = binding.attn_tree(q, k, v, table, P, prob.S, prob.T, 16, 2, 16, prob.scale, masks, positions,
                                 window, sinks, prob.gs, prob.gs)
    assert binding.last_error() == binding.OK
    prob.check(out, lse, str(case))
