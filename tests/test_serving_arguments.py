"""Arguments that the serving calls of the binding refuse before anything reaches the
library (CPU only)."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding


@pytest.mark.parametrize("page", [1, 17])
def test_copy_pages_q4_refuses_pages_it_would_copy_in_part(page):
    """A page is copied as pairs of 72-byte rows: with an odd size its last row, or all of a
    page of one, would stay behind."""
    pool = torch.zeros((2, 1, page * 72), dtype=torch.uint8)
    with pytest.raises(ValueError, match="page_size"):
        binding.copy_pages_q4(pool, pool, torch.zeros((1, 2), dtype=torch.int32), page)


class Pointer:
    """What a call would have handed to the library."""

    def __init__(self, monkeypatch):
        self.calls = []
        monkeypatch.setattr(binding, "_device_call", lambda *a: self.calls.append(a))
        monkeypatch.setattr(binding, "_need", lambda *a, **k: None)
        monkeypatch.setattr(binding, "_q4_pools", lambda k, v, page, dev: (4, 1))


BIG = (2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1)


@pytest.mark.parametrize("big", BIG)
def test_integers_past_32_bits_are_refused(monkeypatch, big):
    """ctypes hands their low 32 bits over: 2^32 + 16 would be 16 tokens."""
    p = Pointer(monkeypatch)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    pool = torch.zeros((4, 1, 16, 128), dtype=torch.bfloat16)
    table = torch.zeros((1, 4), dtype=torch.int32)
    long = torch.zeros(1, dtype=torch.int32).expand(2 ** 33)  # a prefix list of any length
    for f in (lambda: binding.fork_device(long, big, i, 16, i, 4),
              lambda: binding.fork_device(long, 16, i, big if big > 0 else 2 ** 31, i, 4),
              lambda: binding.fork_device(long, 0, i[:0], 16, i, abs(big), out=table),
              lambda: binding.extend_device(table, big, i[:1], i[:1], 16, i, 2),
              lambda: binding.extend_device(table, 16, i[:1], i[:1], big, i, 2),
              lambda: binding.attn_window(q, pool, pool, table, big, [4], [2], 1, 1, 16, 1.0, 4),
              lambda: binding.attn_q4(q, pool, pool, table, big, [4], [2], 1, 1, 16, 1.0, True)):
        with pytest.raises((ValueError, OverflowError), match="32 bits"):
            f()
    assert not p.calls


@pytest.mark.parametrize("kind", ["numpy", "tensor", "list"])
def test_lengths_past_32_bits_are_refused(kind):
    import numpy as np
    wrap = {"numpy": lambda x: np.array(x, dtype=np.int64), "tensor": torch.tensor,
            "list": list}[kind]
    for S, T in (([2 ** 32 + 5], [1]), ([5], [2 ** 32 + 1]), ([-2 ** 31 - 1], [1])):
        with pytest.raises((ValueError, OverflowError)):
            binding._lens(wrap(S), wrap(T))
    held, at, B, R = binding._lens(wrap([5, 6]), wrap([1, 2]))
    assert (B, R) == (2, 3) and list(np.frombuffer(held, np.int32)) == [5, 6, 1, 2] and at


@pytest.mark.parametrize("window,sinks", [(-2 ** 32 + 5, 0), (-1, 0), (4, -2 ** 32 + 1)])
def test_negative_windows_stay_negative(monkeypatch, window, sinks):
    """The library refuses them: they must reach it as what they are."""
    p = Pointer(monkeypatch)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    pool = torch.zeros((4, 1, 16, 128), dtype=torch.bfloat16)
    table = torch.zeros((1, 4), dtype=torch.int32)
    binding.attn_window(q, pool, pool, table, 16, [4], [2], 1, 1, 16, 1.0, window, sinks)
    binding.attn_q4(q, pool, pool, table, 16, [4], [2], 1, 1, 16, 1.0, True, 1.0, 1.0, window, sinks)
    for args in p.calls:
        ints = [a for a in args if isinstance(a, int) and a < 0]
        assert len(ints) == (window < 0) + (sinks < 0) and all(a >= -2 ** 31 for a in ints)


@pytest.fixture(scope="module")
def lib():
    from shared_prefix_fan_gb300 import build
    build.build()
    return binding.load()


# made-up addresses, every array apart from the others
FORK = dict(prefix=0x10000, P=40, B=2, S=0x20000, ps=16, free=0x30000, n_free=9, used=0x40000,
            after=0x50000, table=0x60000, width=8, cow=0x70000, stream=None)
EXTEND = dict(table=0x10000, B=2, width=8, P=40, S=0x20000, A=0x30000, ps=16, free=0x40000, n_free=9,
              used=0x50000, after=0x60000, slots=0x70000, n_slots=4, stream=None)


@pytest.mark.parametrize("kw", [
    dict(prefix=0x60000 + 4), dict(prefix=0x60000 + 24),  # into a row, and over its last entries
    dict(prefix=0x60000), dict(prefix=0x60000 + 32),      # a row, whose partial page is replaced
    dict(S=0x60000 + 60), dict(S=0x70000 + 12), dict(S=0x50000 - 4), dict(free=0x60000 - 32),
    dict(free=0x70000), dict(used=0x60000 + 8), dict(prefix=0x70000 - 8), dict(prefix=0x50000 - 8)])
@pytest.mark.parametrize("name", ["fanout_fork_device", "fanout_fork_device_new"])
def test_fork_refuses_arrays_that_share_memory(lib, name, kw):
    assert getattr(lib, name)(*{**FORK, **kw}.values()) == binding.EINVAL


@pytest.mark.parametrize("kw", [
    dict(S=0x10000), dict(A=0x10000 + 60), dict(free=0x10000 - 32), dict(used=0x10000 + 4),
    dict(slots=0x10000 + 56), dict(slots=0x10000 - 24), dict(S=0x70000 + 28), dict(A=0x60000),
    dict(free=0x60000 - 32), dict(S=0x60000 - 4)])
def test_extend_refuses_arrays_that_share_memory(lib, kw):
    assert lib.fanout_extend_device(*{**EXTEND, **kw}.values()) == binding.EINVAL


E_, U_ = binding.EINVAL, binding.EUNSUPPORTED


@pytest.mark.parametrize("kw,rc", [
    (dict(P=-1), E_), (dict(B=-1), E_), (dict(ps=0), E_), (dict(n_free=-1), E_), (dict(width=-1), E_),
    (dict(B=4097), U_), (dict(width=(1 << 24) + 1), U_), (dict(width=2), E_), (dict(S=None), E_),
    (dict(prefix=None), E_), (dict(table=None), E_), (dict(free=None), E_), (dict(used=0x50000), E_),
    (dict(table=0x60002), E_), (dict(cow=0x70001), E_), (dict(after=0x50003), E_)])
def test_fork_refusals_with_arrays_apart(lib, kw, rc):
    assert lib.fanout_fork_device(*{**FORK, **kw}.values()) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(P=-1), E_), (dict(B=-1), E_), (dict(ps=0), E_), (dict(n_free=-1), E_), (dict(width=-1), E_),
    (dict(B=4097), U_), (dict(S=None), E_), (dict(A=None), E_), (dict(table=None), E_),
    (dict(free=None), E_), (dict(slots=None), E_), (dict(n_slots=-1), E_), (dict(n_slots=1 << 31), E_),
    (dict(used=0x60000), E_), (dict(slots=0x70004), E_), (dict(A=0x30002), E_)])
def test_extend_refusals_with_arrays_apart(lib, kw, rc):
    assert lib.fanout_extend_device(*{**EXTEND, **kw}.values()) == rc


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
@pytest.mark.parametrize("kw", [
    {}, dict(prefix=0x60000 + 32, P=48), dict(prefix=0x60000, P=48, cow=None),
    dict(prefix=0x60000, cow=None), dict(S=0x50000 + 4), dict(used=None), dict(n_free=0, free=None),
    dict(table=0x70000 - 64)])
def test_arrays_apart_are_not_refused(lib, kw):
    """(They fail later, for want of a device.)"""
    assert lib.fanout_fork_device(*{**FORK, **kw}.values()) == binding.ECUDA


@pytest.mark.parametrize("name", ["fanout_attn", "fanout_attn_noalloc", "fanout_attn_window",
                                  "fanout_attn_q4"])
@pytest.mark.parametrize("kw", [dict(pt=1026), dict(pt=1025), dict(lse=4098), dict(lse=4097)])
def test_attention_refuses_words_off_their_boundary(lib, name, kw):
    """Read or written as 32-bit words on the device, where that would be a fault."""
    import ctypes

    import numpy as np
    a = dict(q=1024, k=1024, v=1024, pt=1024, P=64, S=[32, 32], T=[2, 2], B=2, maxp=8, npages=16,
             hq=8, hkv=2, d=128, ps=16, scale=0.088, causal=1, kg=1.0, vg=1.0, window=9, sinks=0,
             out=1024, od=0, lse=None, stream=None)
    a.update(kw)
    held = [np.asarray(a[n], np.int32) for n in "ST"]
    a["S"], a["T"] = (h.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)) for h in held)
    drop = {"fanout_attn_q4": (), "fanout_attn_window": ("causal", "kg", "vg")}.get(
        name, ("kg", "vg", "window", "sinks"))
    args = [v for n, v in a.items() if n not in drop]
    assert getattr(lib, name)(*args) == binding.EINVAL


def test_append_refuses_a_table_off_its_boundary(lib):
    import ctypes

    import numpy as np
    n = np.array([3, 2], np.int32)
    at = n.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    assert lib.fanout_kv_append(1024, 1024, 1024, 1024, 1026, 0, at, at, 2, 4, 8, 2, 128, 16,
                                None) == binding.EINVAL
