"""The shortest wait limit: attention calls give the results of the default one."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import DevWorkload, ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_shortest_wait_limit():
    """A limit of 1 ns is taken as the shortest that copies in flight leave: no wait of
    these calls runs out, and none ends a block before its copies have landed."""
    from shared_prefix_fan_gb300.workloads import draw, small_spec
    probs = [ref.Problem([300, 200], [20, 31], 4000, 16, 2, 32, window=w, sinks=s, q4=q4)
             for w, s, q4 in ((900, 4, False), (0, 0, True), (900, 4, True))]
    probs += [ref.Problem([300, 200], [1, 1], 4000, 16, 2, 32, window=900, q4=q4)
              for q4 in (False, True)]
    w = DevWorkload(draw(small_spec(h_q=8, h_kv=2, prefix_len=1024, q_rows=[6, 3],
                                    suffix_lens=[100, 20])))
    runs = [p.run for p in probs] + [w.run]
    want = [run() for run in runs]
    binding.set_option(binding.OPT_WAIT_LIMIT_NS, 1)
    try:
        for run, (out, lse) in zip(runs, want):
            got = run()
            assert binding.last_error_detail() == (binding.OK, 0, 0)
            assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    finally:
        binding.set_option(binding.OPT_WAIT_LIMIT_NS, 1_000_000_000)
