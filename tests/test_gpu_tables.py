"""Page tables and slot maps built on the device, against the plain host form:
equal, entry for entry."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def dev(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def draw(seed, B, page, P, s_hi, a_hi):
    rng = np.random.default_rng(seed)
    S, A = rng.integers(0, s_hi + 1, B), rng.integers(0, a_hi + 1, B)
    n_pre = -(-P // page)
    width = max([n_pre] + [-(-(P + s + a) // page) for s, a in zip(S, A)]) + int(rng.integers(0, 4))
    own = sum(max(-(-(P + s + a) // page), n_pre) - P // page for s, a in zip(S, A))
    ids = rng.permutation(n_pre + own + 40).astype(np.int32)
    return S, A, width, ids[:n_pre], ids[n_pre:]


CASES = [(1, 16, 0, 0, 1), (1, 64, 1, 0, 0), (3, 16, 250, 40, 1), (8, 64, 1000, 512, 1),
         (7, 128, 128, 5, 300), (33, 32, 77, 100, 40), (255, 16, 4096, 64, 3),
         (257, 24, 50, 64, 3), (1024, 16, 160, 300, 2), (4096, 16, 32, 20, 2), (2, 16, 70000, 9, 5000),
         (1, 16, 40, 0, 70000)]


@pytest.mark.parametrize("B,page,P,s_hi,a_hi", CASES)
@pytest.mark.parametrize("used", [None, 7])
def test_fork_then_extend(B, page, P, s_hi, a_hi, used):
    S, A, width, prefix, free = draw(B * page + P, B, page, P, s_hi, a_hi)
    start = used or 0
    t_ref, cow_ref, u_ref = ref.fork(prefix, P, S, page, free, start, width)
    u_dev = None if used is None else dev([used])
    table, cow, u1 = binding.fork_device(dev(prefix), P, dev(S), page, dev(free), width, u_dev)
    assert np.array_equal(table.cpu().numpy(), t_ref) and int(u1) == u_ref
    assert (cow is None) == (P % page == 0)
    if cow is not None:
        assert np.array_equal(cow.cpu().numpy(), cow_ref)
    n = int(A.sum()) + 5
    t2, s_ref, u2 = ref.extend(t_ref, P, S, A, page, free, u_ref, n)
    slots, u3 = binding.extend_device(table, P, dev(S), dev(A), page, dev(free), n, u1)
    assert np.array_equal(table.cpu().numpy(), t2)
    assert np.array_equal(slots.cpu().numpy(), s_ref) and int(u3) == u2
    again, u4 = binding.extend_device(table, P, dev(S), dev(A), page, dev(free), n, u1)
    assert torch.equal(again, slots) and int(u4) == u2 and np.array_equal(table.cpu().numpy(), t2)
    assert binding.last_error() == binding.OK


def test_no_branches_and_no_rows():
    table, cow, used = binding.fork_device(dev([]), 0, dev([]), 16, dev([]), 4, dev([3]))
    assert tuple(table.shape) == (0, 4) and int(used) == 3
    slots, used = binding.extend_device(table, 0, dev([]), dev([]), 16, dev([]), 6, dev([3]))
    assert int(used) == 3 and (slots == -1).all()
    table, _, _ = binding.fork_device(dev([5]), 16, dev([0, 0]), 16, dev([1]), 1)
    assert table.cpu().tolist() == [[5], [5]]
    slots, used = binding.extend_device(table, 16, dev([0, 0]), dev([0, 0]), 16, dev([1]), 0)
    assert slots.numel() == 0 and int(used) == 0
    assert binding.last_error() == binding.OK


@pytest.mark.parametrize("what", ["suffix", "narrow", "list", "used", "tokens"])
def test_fork_refused_on_the_device(what):
    S, width, free, used = [20, 30], 8, list(range(10, 20)), 0
    if what == "suffix":
        S = [20, -1]
    if what == "narrow":
        width = 3
    if what == "list":
        free = free[:3]
    if what == "used":
        used = -1
    if what == "tokens":
        S = [20, 2 ** 31 - 10]
    out = torch.full((2, width), 77, dtype=torch.int32, device="cuda")
    table, cow, after = binding.fork_device(dev([1, 2]), 20, dev(S), 16, dev(free), width,
                                            dev([used]), out=out)
    assert binding.last_error() == binding.EINVAL and binding.last_error() == binding.OK
    assert (table == 77).all() and int(after) == used


@pytest.mark.parametrize("what", ["add", "narrow", "list", "slots", "page"])
def test_extend_refused_on_the_device(what):
    table = dev([[4, -1, -1], [5, -1, -1]])
    S, A, free, n = [10, 3], [20, 4], [8, 9], 30
    if what == "add":
        A = [20, -4]
    if what == "narrow":
        A = [60, 4]
        free = list(range(10, 30))
        n = 80
    if what == "list":
        free = [8]
        A = [30, 4]
    if what == "slots":
        n = 23
    if what == "page":
        table[1, 0] = -3
    before = table.clone()
    slots, used = binding.extend_device(table, 0, dev(S), dev(A), 16, dev(free), n)
    assert binding.last_error() == binding.EINVAL
    if what == "page":  # only the rows that the bad entry holds
        assert (slots[20:] == -1).all() and int(slots[0]) == 4 * 16 + 10
        return
    assert torch.equal(table, before) and int(used) == 0 and (slots == -1).all()


def test_captured_steps_follow_device_lengths():
    """One captured step replayed: lengths, table and list move on the device only."""
    P, page, free = 40, 16, np.arange(100, 160, dtype=np.int32)
    S = np.array([3, 9, 0])
    t_ref, _, u_ref = ref.fork([50, 51, 52], P, S, page, free, 0, 8)
    S_d, A_d, free_d, used = dev(S), dev([1, 1, 1]), dev(free), dev([u_ref])
    table = torch.as_tensor(t_ref).cuda()
    slots = torch.empty(4, dtype=torch.int64, device="cuda")
    probe = table.clone()  # the first call on a device is made outside a capture
    binding.extend_device(probe, P, S_d, A_d, page, free_d, 4, used)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, after = binding.extend_device(table, P, S_d, A_d, page, free_d, 4, used, slots=slots)
        S_d += A_d
        used.copy_(after)
    for _ in range(40):
        t_ref, s_ref, u_ref = ref.extend(t_ref, P, S, [1, 1, 1], page, free, u_ref, 4)
        S = S + 1
        graph.replay()
        assert np.array_equal(slots.cpu().numpy(), s_ref)
        assert np.array_equal(table.cpu().numpy(), t_ref) and int(used) == u_ref
    assert binding.last_error() == binding.OK


def test_two_streams():
    """Two builds at once, each on a stream of its own."""
    jobs = [draw(s, 300, 16, 500, 200, 10) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in jobs]
    held = [[dev(prefix), dev(S), dev(free)] for S, A, width, prefix, free in jobs]
    torch.cuda.synchronize()
    outs = []
    for (S, A, width, _, _), (prefix, S_d, free), st in zip(jobs, held, streams):
        with torch.cuda.stream(st):
            outs.append(binding.fork_device(prefix, 500, S_d, 16, free, width))
    torch.cuda.synchronize()
    for (S, A, width, prefix, free), (table, cow, used) in zip(jobs, outs):
        t_ref, cow_ref, u_ref = ref.fork(prefix, 500, S, 16, free, 0, width)
        assert np.array_equal(table.cpu().numpy(), t_ref) and int(used) == u_ref
        assert np.array_equal(cow.cpu().numpy(), cow_ref)
