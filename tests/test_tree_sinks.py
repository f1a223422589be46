"""Masks of drafted rows with first keys: which calls are refused on the host (CPU only)."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from .test_tree_arguments import ROWS

E_, U_, OK = binding.EINVAL, binding.EUNSUPPORTED, binding.OK


@pytest.fixture(scope="module")
def lib():
    from shared_prefix_fan_gb300 import build
    build.build()
    return binding.load()


@pytest.mark.parametrize("kw,rc", [
    (dict(sinks=-1, window=4), E_), (dict(sinks=4), E_), (dict(window=-1), E_), (dict(R=-1), E_),
    (dict(words=33, window=4, sinks=4), U_), (dict(masks=0x10000, window=4, sinks=4), E_),
    (dict(slots=None, window=4, sinks=4), E_), (dict(R=0, window=4, sinks=4), OK), (dict(R=0), OK)])
def test_refusals(lib, kw, rc):
    a = {**ROWS, "sinks": 0, **kw}
    order = list(ROWS)
    order.insert(order.index("window") + 1, "sinks")
    assert lib.fanout_tree_rows_sinks(*[a[x] for x in order]) == rc


def test_sinks_reach_the_library(monkeypatch):
    """In front of the outputs, and clamped to 32 bits with their sign; without any, the call
    that has none."""
    calls = []
    monkeypatch.setattr(binding, "_host", type("Host", (), {
        "tree_rows": lambda self, *a: calls.append(("tree_rows", a)),
        "tree_rows_sinks": lambda self, *a: calls.append(("tree_rows_sinks", a))})())
    i, table = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    for sinks, want in ((5, 5), (1 << 40, 2 ** 31 - 1), (-1 << 40, -1)):
        binding.tree_rows(i, table, 0, i, i, 16, 4, 7, sinks=sinks)
        name, a = calls.pop()
        assert name == "tree_rows_sinks" and len(a) == 13 and a[7:9] == (7, want)
    binding.tree_rows(i, table, 0, i, i, 16, 4, 7)
    assert calls[0][0] == "tree_rows" and len(calls[0][1]) == 12


def test_arguments_of_the_extension(lib):
    from . import test_host_calls as t
    module, fake = binding._host_calls(), t.Torch()
    module.setup(t.TYPES, fake.empty, fake.raw_stream, fake.get_device, fake.guard, fake.empty_on,
                 fake.handle_of, binding._check)
    try:
        a = list(t.rows(window=4).values())
        masks, positions, slots = module.tree_rows_sinks(*a[:8], 4, *a[8:])
        assert masks.shape == (0, 2) and positions.shape == slots.shape == (0,)
        for bad in (1 << 31, -(1 << 40)):
            with pytest.raises(ValueError, match="32 bits"):
                module.tree_rows_sinks(*a[:8], bad, *a[8:])
        with pytest.raises(binding.FanoutError):
            module.tree_rows_sinks(*a[:8], -1, *a[8:])
        for args in (a, [*a, 0, 0], [*a[:8], object(), *a[8:]]):
            with pytest.raises(TypeError):
                module.tree_rows_sinks(*args)
    finally:
        binding._host = None  # the next call sets it up with torch's own
