"""A fork that only the device can refuse hands out no page ids."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def dev(a):
    return torch.as_tensor(a, dtype=torch.int32).cuda()


@pytest.mark.parametrize("B,width", [(2, 8), (5, 7), (40, 4100)])
@pytest.mark.parametrize("what", ["suffix", "list", "used", "tokens"])
def test_refused_fork_copies_no_pages(B, width, what):
    """After a fork of the same shape has left its ids in the allocator's blocks: the
    refused one's tables and pairs are -1 throughout, and what a caller does with them
    before looking at the error changes no page."""
    n, page, P = 200, 16, 20
    prefix, S, free = dev([0, 1]), [20] * B, list(range(2, 2 + 3 * B))
    pools = torch.randint(0, 120, (2, n, 2, page * 72), device="cuda").to(torch.uint8)
    table, cow, _ = binding.fork_device(prefix, P, dev(S), page, dev(free), width)
    assert int(cow.min()) >= 1 and binding.last_error() == binding.OK
    del table, cow
    used = 0
    if what == "suffix":
        S[-1] = -1
    if what == "list":
        free = free[:2 * B - 1]
    if what == "used":
        used = -1
    if what == "tokens":
        S[-1] = 2 ** 31 - 10
    S_dev, free_dev, used_dev = dev(S), dev(free), dev([used])
    before = pools.clone()
    table, cow, after = binding.fork_device(prefix, P, S_dev, page, free_dev, width, used_dev)
    binding.copy_pages_q4(pools[0], pools[1], cow, page)
    assert torch.equal(pools, before)
    assert (table == -1).all() and (cow == -1).all() and int(after) == used
    assert binding.last_error() == binding.EINVAL and binding.last_error() == binding.OK


def test_refused_fork_into_a_given_table():
    """The caller's table stays as it was; the pairs are -1."""
    out = torch.full((2, 8), 77, dtype=torch.int32, device="cuda")
    stale = torch.full((2, 2), 3, dtype=torch.int32, device="cuda")
    del stale
    _, cow, _ = binding.fork_device(dev([1, 2]), 20, dev([20, -1]), 16, dev(list(range(10, 20))), 8,
                                    out=out)
    assert (out == 77).all() and (cow == -1).all()
    assert binding.last_error() == binding.EINVAL


def test_refused_fork_without_pairs():
    """A prefix of whole pages, and one of which the caller wants no pairs."""
    for P, want in ((32, True), (20, False)):
        binding.fork_device(dev([1, 2]), P, dev([20, 1]), 16, dev(list(range(10, 20))), 8)
        table, cow, _ = binding.fork_device(dev([1, 2]), P, dev([20, -1]), 16,
                                            dev(list(range(10, 20))), 8, want_cow=want)
        assert cow is None and (table == -1).all()
        assert binding.last_error() == binding.EINVAL


def test_prefix_from_a_row_of_the_table():
    """The whole prefix pages of a branch as the prefix of a new fork into the same table;
    a page that the fork replaces in that row is not taken from it."""
    table = torch.full((3, 9), 5, dtype=torch.int32, device="cuda")
    table[1, :2] = dev([8, 9])
    S, free = dev([20, 0, 33]), dev(list(range(20, 40)))
    want, _, used = binding.fork_device(dev([8, 9]), 32, S, 16, free, 9)
    out, cow, after = binding.fork_device(table[1, :2], 32, S, 16, free, 9, out=table)
    assert cow is None and torch.equal(out, want) and int(after) == int(used)
    before = table.clone()
    with pytest.raises(binding.FanoutError) as e:
        binding.fork_device(table[1, :3], 40, S, 16, free, 9, out=table)
    assert e.value.code == binding.EINVAL and torch.equal(table, before)
    assert binding.last_error() == binding.OK
