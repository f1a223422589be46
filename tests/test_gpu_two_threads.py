"""Serving calls made at once: from threads that share a stream, and from threads with a
stream each. Every result equals the one of the call made alone."""
import threading

import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def steps(q4, seed):
    """A few decode steps (their plans are patched) and a change of shape between them."""
    probs = []
    for i in range(4):
        probs.append(ref.Problem([90 + i, 200 + i, 40 + i], [1, 1, 1], 700, 16, 2, 32, window=300,
                                 sinks=4, q4=q4, seed=seed + i))
    probs.append(ref.Problem([60, 9], [20, 3], 130 + seed, 16, 2, 16, window=0 if q4 else 77, q4=q4,
                             seed=seed))
    return probs


@pytest.mark.parametrize("shared_stream", [True, False])
def test_threads_at_once(shared_stream):
    jobs = [steps(q4, seed) for q4, seed in ((True, 1), (True, 20), (False, 40), (False, 60))]
    want = [[p.run() for p in job] for job in jobs]
    assert binding.last_error() == binding.OK
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    streams = [one if shared_stream else torch.cuda.Stream() for _ in jobs]
    start, bad = threading.Barrier(len(jobs)), []

    def work(job, expect, stream):
        try:
            start.wait(30)
            got = [p.run(stream=stream) for _ in range(10) for p in job]
            stream.synchronize()
            for (out, lse), (o, l) in zip(got, expect * 10):
                if not (torch.equal(out, o) and torch.equal(lse, l)):
                    bad.append("differs")
        except Exception as e:  # shown by the main thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
        assert not t.is_alive()
    assert not bad, bad[:3]
    assert binding.last_error() == binding.OK
