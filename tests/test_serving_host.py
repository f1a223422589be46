"""Host-side refusals of the serving operators, before anything is launched
(CPU only: the addresses are made up)."""
import ctypes

import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding, build

E, U, OK = binding.EINVAL, binding.EUNSUPPORTED, binding.OK
P32 = ctypes.POINTER(ctypes.c_int32)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


FORK = dict(prefix=1024, P=40, B=2, S=1024, ps=16, free=1024, n_free=9, used=None, after=2048,
            table=1024, width=8, cow=None, stream=None)
EXTEND = dict(table=1024, B=2, width=8, P=40, S=1024, A=1024, ps=16, free=1024, n_free=9,
              used=None, after=2048, slots=1024, n_slots=4, stream=None)
APPEND = dict(k=1024, v=1024, ks=256, vs=256, kp=1024, vp=1024, slots=1024, n=4, pages=8, hkv=2,
              d=128, ps=16, kg=1.0, vg=1.0, stream=None)
READ = dict(kp=1024, vp=1024, slots=1024, n=4, pages=8, hkv=2, d=128, ps=16, kg=1.0, vg=1.0,
            k=1024, v=1024, ks=256, vs=256, stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(P=-1), E), (dict(B=-1), E), (dict(ps=0), E), (dict(n_free=-1), E), (dict(width=-1), E),
    (dict(B=4097), U), (dict(width=(1 << 24) + 1), U), (dict(width=2), E), (dict(S=None), E),
    (dict(prefix=None), E),
    (dict(table=None), E), (dict(free=None), E), (dict(used=2048), E), (dict(table=1026), E),
    (dict(cow=1025), E), (dict(after=2046 + 1), E)])
def test_fork_device_refuses(lib, kw, rc):
    assert call(lib.fanout_fork_device, FORK, **kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(P=-1), E), (dict(B=-1), E), (dict(ps=0), E), (dict(n_free=-1), E), (dict(width=-1), E),
    (dict(B=4097), U), (dict(S=None), E), (dict(A=None), E), (dict(table=None), E),
    (dict(free=None), E), (dict(slots=None), E), (dict(n_slots=-1), E), (dict(n_slots=1 << 31), E),
    (dict(used=2048), E), (dict(slots=1028), E), (dict(A=1026), E)])
def test_extend_device_refuses(lib, kw, rc):
    assert call(lib.fanout_extend_device, EXTEND, **kw) == rc


@pytest.mark.parametrize("name,base", [("fanout_kv_append_q4", APPEND),
                                       ("fanout_kv_read_q4", READ)])
@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), E), (dict(pages=0), E), (dict(hkv=0), E), (dict(d=64), U), (dict(ps=24), U),
    (dict(kg=0.0), E), (dict(vg=float("nan")), E), (dict(vg=float("inf")), E), (dict(kg=-1.0), E),
    (dict(ks=255), E), (dict(vs=260), E), (dict(ks=128), E), (dict(k=None), E), (dict(v=1032), E),
    (dict(kp=None), E), (dict(vp=1028), E), (dict(slots=None), E), (dict(slots=1028), E),
    (dict(n=1 << 30, hkv=2), U), (dict(n=0, k=None, slots=None), OK)])
def test_rows_refuse(lib, name, base, kw, rc):
    assert call(getattr(lib, name), base, **kw) == rc


def attn_args(q4, **kw):
    a = dict(q=1024, k=1024, v=1024, pt=1024, P=64, S=[32, 32], T=[2, 2], B=2, maxp=8, npages=16,
             hq=8, hkv=2, d=128, ps=16, scale=0.088, causal=1, kg=1.0, vg=1.0, window=0 if q4 else 9,
             sinks=0, out=1024, od=0, lse=None, stream=None)
    a.update(kw)
    held = [np.asarray(a[n], np.int32) for n in "ST"]
    a["S"], a["T"] = (h.ctypes.data_as(P32) for h in held)
    if not q4:
        for n in ("causal", "kg", "vg"):
            a.pop(n)
    return held, list(a.values())


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(window=-1), E), (dict(sinks=-1), E), (dict(d=64), U), (dict(ps=24), U),
    (dict(hq=7), E), (dict(hq=258), U), (dict(T=[33, 2]), E), (dict(q=None), E), (dict(k=1032), E),
    (dict(maxp=5), E), (dict(npages=0), E), (dict(scale=0.0), E), (dict(scale=float("nan")), E),
    (dict(od=2), E), (dict(out=1028), E), (dict(S=[1 << 29, 2]), U), (dict(pt=None), E),
    (dict(T=[0, 0], q=None, out=None), OK)])
def test_attention_refuses(lib, q4, kw, rc):
    held, args = attn_args(q4, **kw)
    assert (lib.fanout_attn_q4 if q4 else lib.fanout_attn_window)(*args) == rc and held


def test_window_rules(lib):
    assert lib.fanout_attn_window(*attn_args(False, window=0)[1]) == E
    assert lib.fanout_attn_q4(*attn_args(True, window=4, causal=0)[1]) == E
    assert lib.fanout_attn_q4(*attn_args(True, sinks=4)[1]) == E
    assert lib.fanout_attn_q4(*attn_args(True, kg=0.0)[1]) == E


@pytest.mark.parametrize("scale,kg", [(1e-20, 1e-18), (1e30, 1e8), (3e38, 1.0), (1e-38, 1.0)])
def test_softmax_scale_of_the_held_values(lib, scale, kg):
    assert lib.fanout_attn_q4(*attn_args(True, scale=scale, kg=kg)[1]) == E


def test_binding_refuses_host_tensors():
    i, pool = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1, 16 * 72), dtype=torch.uint8)
    x = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int64)
    for f in (lambda: binding.fork_device(i, 16, i, 16, i, 4),
              lambda: binding.extend_device(i.reshape(1, 2), 16, i[:1], i[:1], 16, i, 4),
              lambda: binding.kv_append_q4(x, x, pool, pool, slots, 16),
              lambda: binding.kv_read_q4(pool, pool, slots, 16),
              lambda: binding.copy_pages_q4(pool, pool, i.reshape(1, 2), 16),
              lambda: binding.attn_q4(x, pool, pool, i.reshape(1, 2), 0, [4], [2], 1, 1, 16, 1.0,
                                      True),
              lambda: binding.attn_window(x, x, x, i.reshape(1, 2), 0, [4], [2], 1, 1, 16, 1.0, 4)):
        with pytest.raises(ValueError):
            f()
