"""Attention for trees of drafted tokens, over pools of every kind, against a plain 64-bit
form. Keys before the drafts that no row sees hold NaN."""
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


def run(S, trees, P, hq, hkv, page, out_dtype="f32", **kw):
    prob = tree_ref.Problem(S, [len(t) for t in trees], P, hq, hkv, page, trees=trees, **kw)
    out, lse = prob.run(out_dtype)
    rc = binding.last_error_detail()
    assert rc[0] == binding.OK, rc
    prob.check(out, lse, str(kw))
    return prob, out, lse


def trees_of(T, shape="random", seed=0):
    rng = np.random.default_rng(seed)
    return [tree_ref.random_tree(rng, t, shape) for t in T]


CASES = [
    # S without the drafts, T, P, hq, hkv, page, shape, options
    ([0], [1], 0, 1, 1, 16, "random", {}),                   # a lone token sees itself
    ([0], [5], 0, 8, 1, 16, "flat", {}),                     # nothing but themselves
    ([0, 3], [8, 8], 40, 8, 2, 16, "random", {}),            # prefix ending inside a page
    ([127], [2], 0, 8, 1, 32, "chain", {}),                  # drafts over a tile's end
    ([100, 5, 9], [33, 0, 64], 256, 16, 2, 32, "random", {}),
    ([20, 30], [32, 31], 300, 28, 4, 64, "star", {}),
    ([60], [300], 130, 8, 1, 128, "random", {}),             # drafts over three tiles
    ([9], [1024], 20, 4, 1, 16, "random", {}),               # the most
    ([100, 90], [40, 7], 2000, 64, 8, 16, "random", {}),     # split over CTAs
    ([5, 5], [3, 3], 333, 128, 1, 32, "random", {}),         # G = 128
    ([300, 200], [20, 30], 400, 16, 2, 16, "random", dict(window=1)),
    ([300, 200], [20, 30], 400, 16, 2, 16, "chain", dict(window=7, sinks=3)),
    ([300, 200], [20, 30], 400, 16, 2, 64, "random", dict(window=100, sinks=150)),
    ([30, 20], [20, 30], 900, 16, 2, 64, "random", dict(window=500, sinks=4)),
    ([30, 20], [20, 30], 900, 16, 2, 128, "random", dict(window=1 << 30)),
    ([30, 2], [20, 50], 90, 16, 2, 32, "random", dict(masks="random", extra_words=2)),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_cases(kind, case):
    S, T, P, hq, hkv, page, shape, kw = case
    run(S, trees_of(T, shape), P, hq, hkv, page, kind=kind, **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(12))
def test_random_problems(kind, seed):
    rng = np.random.default_rng(77 + seed)
    hkv, B = int(rng.choice([1, 2, 3])), int(rng.integers(1, 6))
    T = rng.integers(0, 70, size=B)
    T[0] = max(1, T[0])
    window, sinks = (0, 0) if seed % 2 else (int(rng.integers(1, 300)), int(rng.integers(0, 40)))
    run(rng.integers(0, 300, size=B).tolist(), trees_of(T.tolist(), seed=seed),
        int(rng.integers(0, 900)), hkv * int(rng.choice([1, 4, 7, 8])), hkv,
        int(rng.choice([16, 32, 64, 128])), kind=kind, out_dtype=str(rng.choice(["f32", "bf16"])),
        window=window, sinks=sinks, gs=1.0 if kind == "bf16" else float(rng.choice([1.0, 0.25, 0.07])),
        masks="random" if seed % 3 == 0 else "tree", seed=seed)


@pytest.mark.parametrize("kind", KINDS)
def test_a_chain_is_causal_attention(kind):
    """Tokens in order: the causal calls are held to the same reference."""
    prob, out, lse = run([40, 61], trees_of([5, 9], "chain"), 512, 16, 2, 64, kind=kind, seed=3)
    q, k, v, table, *_ = prob.args()
    a = (q, k, v, table, prob.P, prob.S, prob.T, 16, 2, 64, prob.scale)
    if kind == "q4":
        o, l = binding.attn_q4(*a, True, prob.gs, prob.gs)
    elif kind == "q8":
        o, l = binding.attn_q8(*a, True, prob.gs, prob.gs)
    else:
        o, l = binding.attn_window(*a, 1 << 30)
    prob.check(o, l)


@pytest.mark.parametrize("kind", KINDS)
def test_own_bit_is_not_needed(kind):
    """A mask without any bit: the row sees its context and itself."""
    prob = tree_ref.Problem([40, 0], [6, 9], 70, 8, 2, 16, kind=kind, trees=trees_of([6, 9], "flat"))
    prob.args()[4].zero_()
    out, lse = prob.run()
    prob.check(out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_splits_and_many_rounds(kind):
    prob = tree_ref.Problem([70, 90], [30, 200], 3000, 16, 2, 16, kind=kind,
                            trees=trees_of([30, 200]), seed=8)
    ref = prob.reference()
    prob.reference = lambda: ref
    for option, value in ((binding.OPT_SPLITS, 1), (binding.OPT_SPLITS, 7), (binding.OPT_NUM_SMS, 1)):
        binding.set_option(option, value)
        try:
            out, lse = prob.run()
            assert binding.last_error() == binding.OK
        finally:
            binding.set_option(option, 0)
        prob.check(out, lse, f"option {option} {value}")


def test_layers_with_and_without_window_alternate():
    """Each keeps its own plan on the stream, beside the causal calls'."""
    probs = [tree_ref.Problem([40, 61], [5, 9], 512, 16, 2, 64, kind=kind, trees=trees_of([5, 9]),
                              window=w, sinks=s, seed=i)
             for i, (kind, w, s) in enumerate([("q8", 0, 0), ("q8", 64, 4), ("bf16", 0, 0)])]
    probs.append(tree_ref.Problem([40, 61], [5, 9], 512, 16, 2, 64, seed=9))
    refs = [p.run() for p in probs]
    for _ in range(3):
        for p, (o, l) in zip(probs, refs):
            a, b = p.run()
            assert torch.equal(a, o) and torch.equal(b, l)
    for p, (o, l) in zip(probs, refs):
        p.check(o, l)


def test_growing_contexts():
    for s in range(100, 130, 4):
        prob = tree_ref.Problem([s, 2 * s], [8, 8], 256, 8, 1, 16, kind="q8", trees=trees_of([8, 8]),
                                seed=s)
        out, lse = prob.run()
        prob.check(out, lse, str(s))


def test_positions_out_of_range_count_as_the_nearest():
    trees = trees_of([6, 9])
    prob = tree_ref.Problem([300, 200], [6, 9], 70, 8, 2, 16, trees=trees, window=50, sinks=2, seed=4)
    low = prob.positions.copy()
    for r in range(15):
        base = 70 + (300 if r < 6 else 200)
        low[r] = base  # what -5 and the like count as
    junk = np.where(np.arange(15) % 2 == 0, -5, -2 ** 31).astype(np.int32)
    prob.args()[5].copy_(torch.from_numpy(junk))
    a, la = prob.run()
    prob.args()[5].copy_(torch.from_numpy(low))
    b, lb = prob.run()
    assert torch.equal(a, b) and torch.equal(la, lb)
    prob.args()[5].fill_(2 ** 31 - 1)  # as far behind as a tree is deep
    a, _ = prob.run()
    assert torch.isfinite(a).all() and binding.last_error() == binding.OK


def test_validated_tables():
    prob = tree_ref.Problem([300, 200], [6, 9], 70, 8, 2, 16, kind="q8", trees=trees_of([6, 9]),
                            window=50, sinks=2, seed=5)
    binding.set_option(binding.OPT_VALIDATE_TABLE, 1)
    try:
        out, lse = prob.run()
        prob.check(out, lse)
    finally:
        binding.set_option(binding.OPT_VALIDATE_TABLE, 0)


def test_capture_is_refused():
    prob = tree_ref.Problem([30], [5], 100, 8, 1, 16, trees=trees_of([5]), seed=10)
    out, _ = prob.run()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        with pytest.raises(binding.FanoutError) as e:
            prob.run(out=out)
        out.add_(0.0)
    assert e.value.code == binding.EUNSUPPORTED


@pytest.mark.parametrize("kind", KINDS)
def test_pools_past_32_bit_offsets(kind):
    trees = trees_of([9, 5])
    prob = tree_ref.Problem([300, 40], [9, 5], 100, 8, 8, 128, kind=kind, trees=trees, seed=12, spare=0)
    q, k, v, table, *rest = prob.args()
    n = {"bf16": 17000, "q4": 62000, "q8": 34000}[kind]
    big = [torch.empty((n, *x.shape[1:]), dtype=x.dtype, device="cuda") for x in (k, v)]
    assert big[0].numel() * big[0].element_size() > 2 ** 32
    for x, y in zip(big, (k, v)):
        x.view(torch.uint8)[-y.shape[0]:] = y.view(torch.uint8)
    prob.dev[1:4] = [*big, table + (n - k.shape[0])]
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    prob.check(out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_on_another_stream_and_into_given_outputs(kind):
    prob = tree_ref.Problem([30, 28], [5, 9], 1024, 32, 4, 16, kind=kind, trees=trees_of([5, 9]), seed=9)
    here, lse = prob.run("bf16")
    prob.check(here, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # an output that starts on 16 bytes only
    flat = torch.zeros(14 * 32 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    out = flat[8:].view(14, 32, 128)
    got, none = prob.run("bf16", stream=s, out=out, want_lse=False)
    torch.cuda.current_stream().wait_stream(s)
    assert none is None and got is out and torch.equal(out, here) and not flat[:8].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 200)])
def test_branches_that_sweep_the_prefix_themselves(kind, window, sinks):
    """Branches of a unit's rows and more: their own sweeps are cut, and the plan moves with
    the suffixes."""
    for more in (0, 1, 2, 130):
        run([300 + more, 20 + more, 133], trees_of([64, 32, 31], seed=more), 3000, 16, 2, 16, kind=kind,
            window=window, sinks=sinks, out_dtype="bf16", seed=more)
