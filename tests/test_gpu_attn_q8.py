"""Attention over 8-bit pools against a plain 64-bit form. Slots that no row sees hold NaN
bytes, and with a window the table entries of pages that nobody sees are no page."""
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


def run(S, T, P, hq, hkv, page, out_dtype="f32", **kw):
    prob = tree_ref.Problem(S, T, P, hq, hkv, page, **kw)
    out, lse = prob.run(out_dtype)
    rc = binding.last_error_detail()
    assert rc[0] == binding.OK, rc
    prob.check(out, lse, str(kw))
    return prob, out, lse


CASES = [
    # S, T, P, hq, hkv, page, options
    ([1], [1], 0, 1, 1, 16, {}),                                  # one token, one key
    ([1], [1], 1, 8, 1, 16, {}),
    ([5, 3], [1, 1], 40, 8, 2, 16, {}),                           # prefix ending inside a page
    ([16, 16, 16], [4, 4, 4], 256, 8, 1, 16, {}),
    ([17, 1, 0, 90], [1, 1, 0, 1], 300, 16, 2, 32, {}),           # a branch without rows
    ([129], [129], 0, 8, 8, 64, {}),                              # G = 1, a tile and one key
    ([40, 33], [40, 33], 128, 28, 4, 128, {}),                    # G = 7
    ([200, 260], [150, 7], 1000, 40, 8, 64, {}),                  # G = 5, two query tiles
    ([300], [3], 5000, 64, 8, 16, {}),                            # long, split over CTAs
    ([64, 64], [16, 16], 700, 128, 1, 32, {}),                    # G = 128
    ([70, 9], [9, 70], 333, 8, 2, 64, dict(causal=False)),        # all keys, more rows than suffix
    ([600, 41], [5, 41], 500, 16, 2, 16, dict(window=1)),
    ([600, 41], [5, 41], 500, 16, 2, 16, dict(window=100, sinks=5)),
    ([300, 300], [300, 20], 900, 16, 2, 64, dict(window=130, sinks=129)),
    ([80, 90], [1, 1], 2000, 8, 1, 128, dict(window=1 << 30, sinks=3)),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_cases(case):
    S, T, P, hq, hkv, page, kw = case
    run(S, T, P, hq, hkv, page, **kw)


@pytest.mark.parametrize("seed", range(24))
def test_random_problems(seed):
    rng = np.random.default_rng(1000 + seed)
    hkv = int(rng.choice([1, 2, 3]))
    B = int(rng.integers(1, 6))
    T = rng.integers(0, 30, size=B)
    if seed % 4 == 0:
        T[:] = 1
    if seed % 7 == 0:
        T[0] = int(rng.integers(100, 280))
    T[0] = max(T[0], 1)
    S = T + rng.integers(0, 400, size=B)
    window, sinks = (0, 0) if seed % 2 else (int(rng.integers(1, 300)), int(rng.integers(0, 40)))
    run(S.tolist(), T.tolist(), int(rng.integers(0, 1500)), hkv * int(rng.choice([1, 4, 7, 8])), hkv,
        int(rng.choice([16, 32, 64, 128])), out_dtype=str(rng.choice(["f32", "bf16"])),
        window=window, sinks=sinks, gs=float(rng.choice([1.0, 0.25, 0.07, 8.0])), seed=seed)


@pytest.mark.parametrize("T", [1, 40])
def test_long_sweeps(T):
    """Rings go round many times in one unit."""
    prob = tree_ref.Problem([T + 3], [T], 20000, 8, 1, 16, seed=3)
    binding.set_option(binding.OPT_NUM_SMS, 2)
    try:
        out, lse = prob.run()
        assert binding.last_error() == binding.OK
        prob.check(out, lse)
    finally:
        binding.set_option(binding.OPT_NUM_SMS, 0)


def test_large_and_small_scores():
    """Rows whose scores spread over hundreds of units, and rows of tiny and mixed q."""
    run([60, 70], [6, 7], 500, 8, 2, 32, q_amp=40.0, k_amp=4.0, seed=1)
    prob = tree_ref.Problem([60, 70], [6, 7], 500, 8, 2, 32, seed=2)
    prob.q[0] *= 2.0 ** -60
    prob.q[1] = 0
    prob.q[2, :, 5] *= 2.0 ** 12  # one channel far above the others
    prob.q[3] *= 2.0 ** 40
    prob.q[3] *= torch.sign(prob.q[3]) * 0  # a row of signed zeros
    out, lse = prob.run()
    prob.check(out, lse)


def test_rows_that_are_no_numbers_stay_alone():
    prob = tree_ref.Problem([60, 70], [6, 7], 500, 8, 2, 32, seed=4)
    clean, clean_lse = prob.run()
    bad = prob.q.clone()
    bad[2, 1, 7] = float("inf")
    bad[9, 6, 100] = float("nan")
    prob.dev[0] = bad.cuda()
    out, lse = prob.run()
    hit = torch.zeros(13, 8, dtype=torch.bool)
    hit[2, 1] = hit[9, 6] = True
    assert torch.isnan(out[hit.cuda()]).all()
    assert torch.equal(out[~hit.cuda()], clean[~hit.cuda()])
    assert torch.equal(lse[~hit.cuda()], clean_lse[~hit.cuda()])


def test_bf16_pools_of_the_same_values_agree():
    """fanout_attn over bf16 pools that hold what the bytes stand for."""
    prob, out, lse = run([300, 280], [5, 9], 1024, 32, 4, 64, seed=5)
    q, k, v, table = prob.args()
    o2, l2 = binding.attn(q, k.to(torch.bfloat16).nan_to_num(), v.to(torch.bfloat16).nan_to_num(),
                          table, prob.P, prob.S, prob.T, 32, 4, 64, prob.scale, True)
    prob.kind = "bf16"
    prob.check(o2, l2)  # the same reference, with the steps of bf16


def test_results_do_not_depend_on_the_call():
    prob, out, lse = run([300, 28, 77], [5, 9, 1], 1024, 32, 4, 16, seed=6)
    for _ in range(3):
        o, l = prob.run()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_decode_steps_move_the_plan():
    """Lengths that grow from call to call on one stream, past tiles and pages."""
    for s in range(120, 140, 3):
        prob = tree_ref.Problem([s, 2 * s], [1, 1], 256, 8, 1, 16, seed=s)
        out, lse = prob.run()
        prob.check(out, lse, str(s))


def test_splits_and_merges():
    prob = tree_ref.Problem([700, 900], [3, 40], 1500, 16, 2, 64, seed=8, window=1700, sinks=30)
    ref = prob.reference()
    prob.reference = lambda: ref
    for n in (1, 2, 5, 16):
        binding.set_option(binding.OPT_SPLITS, n)
        try:
            out, lse = prob.run()
            assert binding.last_error() == binding.OK
        finally:
            binding.set_option(binding.OPT_SPLITS, 0)
        prob.check(out, lse, f"splits {n}")


def test_on_another_stream_and_without_lse():
    prob = tree_ref.Problem([300, 28], [5, 9], 1024, 32, 4, 16, seed=9)
    prob.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = prob.run(stream=s, want_lse=False)
    assert lse is None
    torch.cuda.current_stream().wait_stream(s)
    again, lse = prob.run()
    prob.check(again, lse)
    assert torch.equal(out, again)


def test_capture_is_refused():
    prob = tree_ref.Problem([30], [5], 100, 8, 1, 16, seed=10)
    out, _ = prob.run()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        with pytest.raises(binding.FanoutError) as e:
            prob.run(out=out)
        out.add_(0.0)
    assert e.value.code == binding.EUNSUPPORTED


def test_a_page_outside_the_pool_is_reported():
    prob = tree_ref.Problem([30], [5], 100, 8, 1, 16, seed=11)
    args = prob.args()
    args[3][0, 2] = 1 << 20
    prob.run()
    assert binding.last_error() == binding.EINVAL


def test_pools_past_32_bit_offsets():
    prob = tree_ref.Problem([30, 40], [5, 1], 100, 8, 8, 128, seed=12, spare=0)
    q, k, v, table = prob.args()
    n = 34000
    big = [torch.empty((n, 8, 128, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip(big, (k, v)):
        x[-y.shape[0]:] = y.view(torch.uint8)
    prob.dev[1:] = [big[0].view(k.dtype), big[1].view(k.dtype), table + (n - k.shape[0])]
    assert big[0].numel() > 2 ** 32
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    prob.check(out, lse)


@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (True, 2500, 200), (False, 0, 0)])
def test_branches_that_sweep_the_prefix_themselves(causal, window, sinks):
    """Branches of a unit's rows and more: their own sweeps are cut, and the plan moves with
    the suffixes."""
    for more in (0, 1, 2, 130):
        run([364 + more, 52 + more, 164], [64, 32, 31], 3000, 16, 2, 16, causal=causal, window=window,
            sinks=sinks, seed=more)
