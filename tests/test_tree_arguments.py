"""Calls of the 8-bit cache and of drafted trees that are refused on the host (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

E_, U_, OK = binding.EINVAL, binding.EUNSUPPORTED, binding.OK


@pytest.fixture(scope="module")
def lib():
    from shared_prefix_fan_gb300 import build
    build.build()
    return binding.load()


# made-up addresses, every array apart from the others; each call below is refused (or has
# nothing to do) before anything is launched
ROWS = dict(parents=0x10000, table=0x20000, B=2, width=8, P=40, S=0x30000, A=0x40000, ps=16, R=6,
            words=2, window=0, masks=0x50000, positions=0x60000, slots=0x70000, stream=None)
ACCEPT = dict(parents=0x10000, draft=0x20000, target=0x30000, first=0x40000, A=0x50000, B=2, R=6,
              path=0x60000, counts=0x70000, after=0x80000, stream=None)
KEEP = dict(k=0x100000, v=0x200000, kv=2, table=0x20000, B=2, width=8, P=40, S=0x30000, A=0x40000,
            path=0x50000, counts=0x60000, R=6, pages=9, hkv=2, d=128, ps=16, stream=None)
ROW8 = dict(k=0x1000, v=0x2000, ks=256, vs=256, kp=0x100000, vp=0x200000, slots=0x3000, n=4,
            pages=9, hkv=2, d=128, ps=16, kscale=1.0, vscale=1.0, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), E_), (dict(width=-1), E_), (dict(P=-1), E_), (dict(ps=0), E_), (dict(R=-1), E_),
    (dict(words=0), E_), (dict(window=-1), E_), (dict(B=4097), U_), (dict(words=33), U_),
    (dict(R=1 << 31), U_), (dict(parents=None), E_), (dict(table=None), E_), (dict(S=None), E_),
    (dict(A=None), E_), (dict(masks=None), E_), (dict(positions=None), E_), (dict(slots=None), E_),
    (dict(parents=0x10002), E_), (dict(masks=0x50001), E_), (dict(slots=0x70004), E_),
    (dict(masks=0x10000), E_), (dict(positions=0x20000 + 60), E_), (dict(slots=0x40000), E_),
    (dict(positions=0x50000 + 44), E_), (dict(slots=0x60000 + 16), E_), (dict(R=0), OK)])
def test_tree_rows_refusals(lib, kw, rc):
    assert lib.fanout_tree_rows(*{**ROWS, **kw}.values()) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), E_), (dict(R=-1), E_), (dict(B=4097), U_), (dict(R=1 << 31), U_),
    (dict(parents=None), E_), (dict(draft=None), E_), (dict(target=None), E_),
    (dict(first=None), E_), (dict(A=None), E_), (dict(path=None), E_), (dict(counts=None), E_),
    (dict(after=None), E_), (dict(draft=0x20004), E_), (dict(path=0x60001), E_),
    (dict(after=0x80004), E_), (dict(path=0x10000 + 20), E_), (dict(after=0x40000), E_),
    (dict(counts=0x60000 + 20), E_), (dict(B=0, R=0), OK)])
def test_tree_accept_refusals(lib, kw, rc):
    assert lib.fanout_tree_accept(*{**ACCEPT, **kw}.values()) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(kv=3), E_), (dict(kv=-1), E_), (dict(B=-1), E_), (dict(width=-1), E_), (dict(P=-1), E_),
    (dict(R=-1), E_), (dict(pages=0), E_), (dict(hkv=0), E_), (dict(d=0), E_), (dict(ps=0), E_),
    (dict(d=64), U_), (dict(ps=24), U_), (dict(B=4097), U_), (dict(R=1 << 31), U_),
    (dict(hkv=1 << 30), U_), (dict(k=None), E_), (dict(v=None), E_), (dict(k=0x100008), E_),
    (dict(table=None), E_), (dict(S=None), E_), (dict(A=None), E_), (dict(path=None), E_),
    (dict(counts=None), E_), (dict(path=0x50002), E_), (dict(R=0), OK), (dict(B=0), OK),
    # arrays inside the pools (9 pages of 2 heads x 16 rows of 128 bytes), pools over each other
    (dict(table=0x108ffc), E_), (dict(S=0x200000), E_), (dict(A=0x200004), E_),
    (dict(path=0x100000 - 20), E_), (dict(counts=0x208ff8), E_), (dict(v=0x108ff0), E_),
    (dict(k=0x200000), E_), (dict(kv=0, path=0x111ffc), E_), (dict(kv=1, path=0x1050fc), E_),
    (dict(pages=2 ** 31 - 1, hkv=2 ** 29), E_)])
def test_kv_keep_refusals(lib, kw, rc):
    assert lib.fanout_kv_keep(*{**KEEP, **kw}.values()) == rc


@pytest.mark.parametrize("name", ["append", "read"])
@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), E_), (dict(pages=0), E_), (dict(hkv=0), E_), (dict(d=64), U_), (dict(ps=8), U_),
    (dict(kscale=0.0), E_), (dict(vscale=float("nan")), E_), (dict(kscale=1e31), E_),
    (dict(vscale=-1.0), E_), (dict(n=1 << 30), U_), (dict(ks=255), E_), (dict(vs=128), E_),
    (dict(ks=260), E_), (dict(k=None), E_), (dict(kp=0x100008), E_), (dict(slots=0x3004), E_),
    (dict(v=0x2008), E_), (dict(n=0), OK)])
def test_8_bit_row_refusals(lib, name, kw, rc):
    a = {**ROW8, **kw}
    if name == "read":
        a = {k: a[k] for k in ("kp", "vp", "slots", "n", "pages", "hkv", "d", "ps", "kscale",
                               "vscale", "k", "v", "ks", "vs", "stream")}
    assert getattr(lib, f"fanout_kv_{name}_q8")(*a.values()) == rc


@pytest.mark.parametrize("name,kw", [
    ("append", dict(vp=0x108ff0)), ("append", dict(kp=0x200000)),
    ("append", dict(k=0x108ff0)), ("append", dict(v=0x200000 - 0x710)),
    ("append", dict(slots=0x208ff8)), ("append", dict(slots=0x100000 - 24)),
    ("read", dict(k=0x108ff0)), ("read", dict(v=0x200000 - 0x7f0)), ("read", dict(slots=0x1000)),
    ("read", dict(slots=0x27f8)), ("read", dict(ks=1 << 40)),
    ("append", dict(pages=2 ** 31 - 1, hkv=2 ** 28, ks=2 ** 60, vs=2 ** 60))])
def test_8_bit_rows_over_pools_are_refused(lib, name, kw):
    test_8_bit_row_refusals(lib, name, kw, E_)


def attn(lib, tree, **kw):
    a = dict(q=0x1000, k=0x100000, v=0x200000, kv=2, table=0x2000, P=32, S=[9, 7], T=[4, 2], B=2, width=8,
             pages=9, hq=8, hkv=2, d=128, ps=16, scale=0.1, causal=1, masks=0x3000, words=1,
             positions=0x4000, window=0, sinks=0, ks=1.0, vs=1.0, out=0x5000, dt=0, lse=None)
    a.update(kw)
    S, T = (np.asarray(a[x], np.int32) for x in ("S", "T"))
    s, t = (x.ctypes.data_as(ctypes.c_void_p) for x in (S, T))
    if tree:
        return lib.fanout_attn_tree(a["q"], a["k"], a["v"], a["kv"], a["table"], a["P"], s, t, a["B"],
                                    a["width"], a["pages"], a["hq"], a["hkv"], a["d"], a["ps"],
                                    a["scale"], a["masks"], a["words"], a["positions"], a["window"],
                                    a["sinks"], a["ks"], a["vs"], a["out"], a["dt"], a["lse"], None)
    return lib.fanout_attn_q8(a["q"], a["k"], a["v"], a["table"], a["P"], s, t, a["B"], a["width"],
                              a["pages"], a["hq"], a["hkv"], a["d"], a["ps"], a["scale"],
                              a["causal"], a["ks"], a["vs"], a["window"], a["sinks"], a["out"],
                              a["dt"], a["lse"], None)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(d=64), U_), (dict(ps=8), U_), (dict(hq=6, hkv=4), E_), (dict(hq=256, hkv=1), U_),
    (dict(T=[10, 2]), E_), (dict(S=[-1, 7]), E_), (dict(q=None), E_), (dict(k=0x100008), E_),
    (dict(width=2), E_), (dict(dt=5), E_), (dict(scale=0.0), E_), (dict(scale=float("inf")), E_),
    (dict(window=-1), E_), (dict(sinks=-1), E_), (dict(sinks=1), E_), (dict(ks=0.0), E_),
    (dict(vs=float("nan")), E_), (dict(ks=1e-30, scale=1e-10), E_), (dict(lse=0x6002), E_),
    (dict(table=0x2002), E_), (dict(T=[0, 0], q=None, out=None), OK)])
def test_attention_refusals(lib, tree, kw, rc):
    assert attn(lib, tree, **kw) == rc


def test_windows_over_all_keys_are_refused(lib):
    assert attn(lib, False, causal=0, window=4) == E_


@pytest.mark.parametrize("kw,rc", [
    (dict(kv=3), E_), (dict(kv=-1), E_), (dict(masks=None), E_), (dict(masks=0x3001), E_),
    (dict(words=0), E_), (dict(positions=0x4002), E_), (dict(window=4, positions=None), E_),
    (dict(S=[90, 7], T=[33, 2], width=16), E_),        # more tokens than the mask has bits
    (dict(S=[1100, 7], T=[1025, 2], words=64, width=99), U_)])
def test_tree_attention_refusals(lib, kw, rc):
    assert attn(lib, True, **kw) == rc


class Calls:
    def __init__(self, monkeypatch):
        self.calls = []
        monkeypatch.setattr(binding, "_device_call", lambda *a: self.calls.append(a))
        monkeypatch.setattr(binding, "_need", lambda *a, **k: None)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1])
def test_integers_past_32_bits_are_refused(monkeypatch, big):
    c = Calls(monkeypatch)
    i, table = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    pool = torch.zeros((4, 1, 16, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    masks = torch.zeros((2, 1), dtype=torch.int32)
    for f in (lambda: binding.tree_rows(i, table, big, i, i, 16, 4),
              lambda: binding.tree_rows(i, table, 0, i, i, big, 4),
              lambda: binding.kv_keep(pool, pool, table, big, i, i, i, i, 16),
              lambda: binding.attn_q8(q, pool, pool, table, big, [4], [2], 1, 1, 16, 1.0, True),
              lambda: binding.attn_tree(q, pool, pool, table, big, [4], [2], 1, 1, 16, 1.0, masks)):
        with pytest.raises((ValueError, OverflowError), match="32 bits"):
            f()
    assert not c.calls


@pytest.mark.parametrize("window,sinks", [(-2 ** 32 + 5, 0), (4, -2 ** 32 + 1)])
def test_negative_windows_stay_negative(monkeypatch, window, sinks):
    calls = []
    record = lambda self, *a: calls.append(a)  # noqa: E731
    monkeypatch.setattr(binding, "_host", type("Host", (), {
        "tree_rows": record, "attn_q8": record, "attn_tree": record})())
    i, table = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 4), dtype=torch.int32)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    pool = torch.zeros((4, 1, 16, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    masks = torch.zeros((2, 1), dtype=torch.int32)
    binding.attn_q8(q, pool, pool, table, 16, [4], [2], 1, 1, 16, 1.0, True, 1.0, 1.0, window, sinks)
    binding.attn_tree(q, pool, pool, table, 16, [4], [2], 1, 1, 16, 1.0, masks, None, window, sinks)
    if not sinks:
        binding.tree_rows(i, table, 0, i, i, 16, 4, window)
    assert len(calls) == (2 if sinks else 3)
    for args in calls:
        ints = [a for a in args if isinstance(a, int) and a < 0]
        assert ints and all(a >= -2 ** 31 for a in ints)


def test_wrong_tensors_are_refused():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q4 = torch.zeros((4, 1, 16 * 72), dtype=torch.uint8)
    q8 = torch.zeros((4, 1, 16, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    q = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    for f in (lambda: binding.tree_rows(i32(3), i32(1, 4), 0, i32(1), i32(1), 16, 0),
              lambda: binding.tree_rows(i32(3), i32(1, 4), 0, i32(1), i32(1), 16, 1025),
              lambda: binding.tree_rows(i32(3).long(), i32(1, 4), 0, i32(1), i32(1), 16, 4),
              lambda: binding.kv_append_q8(q, q, q4, q4, torch.zeros(2, dtype=torch.int64)),
              lambda: binding.kv_read_q8(q8, q4, torch.zeros(2, dtype=torch.int64)),
              lambda: binding.copy_pages_q8(q4, q4, i32(1, 2), 4),
              lambda: binding.attn_q8(q, q4, q4, i32(1, 4), 0, [4], [2], 1, 1, 16, 1.0, True),
              lambda: binding.attn_tree(q, q8, q8, i32(1, 4), 0, [4], [2], 1, 1, 16, 1.0, i32(3, 1)),
              lambda: binding.kv_keep(q8, q8, i32(1, 4), 0, i32(1), i32(1), i32(3), i32(1), 32)):
        with pytest.raises(ValueError):
            f()
