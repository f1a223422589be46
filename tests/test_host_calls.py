"""The extension module behind the calls of the 8-bit cache and of drafts, on the CPU: which arguments it refuses,
what it hands to the library, which device and stream it uses, and that no object is kept.

Its tensors here are stand-ins with the attributes that it reads; their addresses are made up,
and every call is refused or has no rows, so nothing is launched."""
import sys

import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

BF16, F8, U8, I32, I64, F32 = TYPES = (torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32,
                                       torch.int64, torch.float32)
DEV, OTHER = torch.device("cuda", 0), torch.device("cuda", 1)


class Fake:
    """A tensor of this type and shape at a made-up address."""
    places = iter(range(1 << 20, 1 << 40, 1 << 20))

    def __init__(self, dtype, *shape, device=DEV, stride=None, contiguous=True):
        self.dtype, self.shape, self.device, self.address = dtype, shape, device, next(Fake.places)
        self.is_cuda, self.contiguous = device.type == "cuda", contiguous
        self.steps = stride or tuple(torch.empty(shape, device="meta").stride())

    def is_contiguous(self):
        return self.contiguous

    def stride(self):
        return self.steps

    def data_ptr(self):
        return self.address


class Torch:
    """What setup() is given in place of torch's functions, and what was done with it."""

    def __init__(self):
        self.device, self.log, self.made = 0, [], []

    def empty(self, size, dtype, device):
        self.made.append((size, dtype, device))
        return Fake(dtype, *size, device=device)

    def raw_stream(self, index):
        self.log.append(("raw", index))
        return 64

    def get_device(self):
        return self.device

    def guard(self, index):
        outer = self

        class Guard:
            def __enter__(self):
                outer.log.append(("enter", index))

            def __exit__(self, *exc):
                outer.log.append(("exit", index))
        return Guard()

    def empty_on(self, dev, stream):
        self.log.append(("empty_on", stream))
        return self.empty

    def handle_of(self, stream):
        return 4096 + stream


@pytest.fixture(scope="module")
def built():
    from shared_prefix_fan_gb300 import build
    build.build()


@pytest.fixture
def host(built):
    module, fake = binding._host_calls(), Torch()
    module.setup(TYPES, fake.empty, fake.raw_stream, fake.get_device, fake.guard,
                 fake.empty_on, fake.handle_of, binding._check)
    yield module, fake
    binding._host = None  # the next call sets it up with torch's own


def append(n=0, **kw):
    d = dict(k_new=Fake(BF16, n, 2, 128), v_new=Fake(BF16, n, 2, 128), k_pages=Fake(F8, 9, 2, 16, 128),
             v_pages=Fake(F8, 9, 2, 16, 128), slots=Fake(I64, n), k_scale=1.0, v_scale=1.0, stream=None)
    return {**d, **kw}


def read(n=0, **kw):
    d = dict(k_pages=Fake(F8, 9, 2, 16, 128), v_pages=Fake(F8, 9, 2, 16, 128), slots=Fake(I64, n),
             k_scale=1.0, v_scale=1.0, k_out=None, v_out=None, stream=None)
    return {**d, **kw}


def rows(n=0, B=2, **kw):
    d = dict(parents=Fake(I32, n), page_table=Fake(I32, B, 8), prefix_len=40, suffix_lens=Fake(I32, B),
             add_lens=Fake(I32, B), page_size=16, words=2, window=0, masks=None, positions=None,
             slots=None, stream=None)
    return {**d, **kw}


def accept(n=0, B=0, **kw):
    d = dict(parents=Fake(I32, n), draft=Fake(I64, n), target=Fake(I64, n), first=Fake(I64, B),
             add_lens=Fake(I32, B), stream=None)
    return {**d, **kw}


def keep(n=0, B=2, dtype=BF16, **kw):
    shape = (9, 2, 16 * 72) if dtype is U8 else (9, 2, 16, 128)
    d = dict(k_pages=Fake(dtype, *shape), v_pages=Fake(dtype, *shape), page_table=Fake(I32, B, 8),
             prefix_len=40, suffix_lens=Fake(I32, B), add_lens=Fake(I32, B), path=Fake(I32, n),
             counts=Fake(I32, B), page_size=16, stream=None)
    return {**d, **kw}


LENS = np.zeros((2, 3), dtype=np.int32)  # three branches of no rows


def attn(R=0, **kw):
    d = dict(q=Fake(BF16, R, 4, 128), k_pages=Fake(F8, 9, 2, 16, 128), v_pages=Fake(F8, 9, 2, 16, 128),
             page_table=Fake(I32, 3, 8), prefix_len=0, lens=LENS.ctypes.data, B=3, R=R, h_q=4, h_kv=2,
             page_size=16, scale=1.0, causal=True, window=0, sinks=0, k_scale=1.0, v_scale=1.0, out=None,
             lse=None, bf16=False, want_lse=True, stream=None)
    return {**d, **kw}


def tree(R=0, dtype=BF16, **kw):
    shape = (9, 2, 16 * 72) if dtype is U8 else (9, 2, 16, 128)
    d = attn(R, k_pages=Fake(dtype, *shape), v_pages=Fake(dtype, *shape))
    tail = {k: d.pop(k) for k in list(d)[list(d).index("causal"):]}
    del tail["causal"]
    return {**d, "masks": Fake(I32, R, 1), "positions": Fake(I32, R), **tail, **kw}


CALLS = {"attn_q8": attn, "attn_tree": tree, "kv_append_q8": append, "kv_read_q8": read, "tree_rows": rows, "tree_accept": accept,
         "kv_keep": keep}


def test_no_rows_is_no_work(host):
    module, fake = host
    assert module.kv_append_q8(*append().values()) is None
    k, v = module.kv_read_q8(*read().values())
    assert k.shape == v.shape == (0, 2, 128) and k.dtype == v.dtype == BF16
    to = read(k_out=Fake(BF16, 0, 2, 128), v_out=Fake(BF16, 0, 2, 128))
    assert module.kv_read_q8(*to.values()) == (to["k_out"], to["v_out"])
    masks, positions, slots = module.tree_rows(*rows().values())
    assert masks.shape == (0, 2) and positions.shape == slots.shape == (0,)
    assert (masks.dtype, positions.dtype, slots.dtype) == (I32, I32, I64)
    path, counts, after = module.tree_accept(*accept().values())
    assert path.shape == counts.shape == after.shape == (0,)
    assert (path.dtype, counts.dtype, after.dtype) == (I32, I32, I64)
    for dtype in (BF16, F8, U8):
        assert module.kv_keep(*keep(dtype=dtype).values()) is None
        out, lse = module.attn_tree(*tree(dtype=dtype).values())
        assert (out.shape, out.dtype, lse.shape, lse.dtype) == ((0, 4, 128), F32, (0, 4), F32)
    out, lse = module.attn_q8(*attn(bf16=True).values())
    assert (out.shape, out.dtype, lse.shape, lse.dtype) == ((0, 4, 128), BF16, (0, 4), F32)
    to = attn(out=Fake(F32, 0, 4, 128), lse=Fake(F32, 0, 4), want_lse=False)
    assert module.attn_q8(*to.values()) == (to["out"], to["lse"])
    assert module.attn_tree(*tree(want_lse=False, positions=None).values())[1] is None


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current,stream", [(0, None), (0, 5), (1, None), (1, 5)])
def test_device_and_stream(host, name, current, stream):
    """The call's device is made current when another one is; results of a call on a given
    stream come from that stream's memory."""
    module, fake = host
    fake.device = current
    getattr(module, name)(*CALLS[name](stream=stream).values())
    want = [("raw", 0)] if stream is None else [("empty_on", 5)]
    assert fake.log == want + ([("enter", 0), ("exit", 0)] if current else [])
    assert all(d == DEV for _, _, d in fake.made)


def test_refused_by_the_library(host):
    """An error code of the library is raised, and the device that was current is so again."""
    module, fake = host
    fake.device = 1
    for name, args in (("kv_append_q8", append(k_scale=0.0)), ("kv_read_q8", read(v_scale=-1.0)),
                       ("tree_rows", rows(page_size=0)), ("tree_accept", accept(B=5000)),
                       ("kv_keep", keep(prefix_len=-1)), ("attn_q8", attn(scale=0.0)),
                       ("attn_q8", attn(window=4, causal=False)), ("attn_tree", tree(sinks=1)),
                       ("attn_tree", tree(scale=float("inf")))):
        fake.log.clear()
        with pytest.raises(binding.FanoutError):
            getattr(module, name)(*args.values())
        assert fake.log[-1] == ("exit", 0)


REFUSED = [
    ("kv_append_q8", append(k_pages=Fake(F8, 9, 2, 16, 128, device=torch.device("cpu")))),
    ("kv_append_q8", append(k_pages=Fake(BF16, 9, 2, 16, 128))),
    ("kv_append_q8", append(k_pages=Fake(F8, 9, 2, 16 * 128))),
    ("kv_append_q8", append(k_pages=Fake(F8, 1 << 31, 2, 16, 128), v_pages=Fake(F8, 1 << 31, 2, 16, 128))),
    ("kv_append_q8", append(v_pages=Fake(F8, 9, 2, 32, 128))),
    ("kv_append_q8", append(v_pages=Fake(F8, 9, 2, 16, 128, device=OTHER))),
    ("kv_append_q8", append(v_pages=Fake(F8, 9, 2, 16, 128, contiguous=False))),
    ("kv_append_q8", append(slots=Fake(I32, 0))), ("kv_append_q8", append(slots=Fake(I64, 0, 1))),
    ("kv_append_q8", append(4, slots=Fake(I64, 5))),
    ("kv_append_q8", append(slots=Fake(I64, 1 << 31))),
    ("kv_append_q8", append(4, k_new=Fake(torch.float16, 4, 2, 128))),
    ("kv_append_q8", append(4, k_new=Fake(BF16, 4, 3, 128))),
    ("kv_append_q8", append(4, v_new=Fake(BF16, 4, 2, 64))),
    ("kv_append_q8", append(4, v_new=Fake(BF16, 4, 256))),
    ("kv_append_q8", append(4, v_new=Fake(BF16, 4, 2, 128, device=OTHER))),
    ("kv_append_q8", append(4, k_new=Fake(BF16, 4, 2, 128, stride=(256, 128, 2)))),
    ("kv_append_q8", append(4, k_new=Fake(BF16, 4, 2, 128, stride=(512, 256, 1)))),
    ("kv_read_q8", read(4, k_out=Fake(BF16, 3, 2, 128))),
    ("kv_read_q8", read(4, v_out=Fake(I32, 4, 2, 128))),
    ("kv_read_q8", read(4, v_out=Fake(BF16, 4, 2, 128, stride=(256, 1, 2)))),
    ("tree_rows", rows(prefix_len=1 << 31)), ("tree_rows", rows(page_size=-(1 << 40))),
    ("tree_rows", rows(window=1 << 70)), ("tree_rows", rows(parents=Fake(I64, 0))),
    ("tree_rows", rows(suffix_lens=Fake(I32, 3))), ("tree_rows", rows(add_lens=Fake(I32, 1))),
    ("tree_rows", rows(page_table=Fake(I32, 16))), ("tree_rows", rows(masks=Fake(I32, 0, 3))),
    ("tree_rows", rows(positions=Fake(I64, 0))), ("tree_rows", rows(slots=Fake(I64, 1))),
    ("tree_accept", accept(4, draft=Fake(I64, 5))), ("tree_accept", accept(4, target=Fake(I32, 4))),
    ("tree_accept", accept(4, B=2, first=Fake(I64, 3))),
    ("tree_accept", accept(4, B=2, add_lens=Fake(I32, 2, 1))),
    ("kv_keep", keep(k_pages=Fake(I32, 9, 2, 16, 128))), ("kv_keep", keep(page_size=32)),
    ("kv_keep", keep(dtype=U8, page_size=32)), ("kv_keep", keep(v_pages=Fake(F8, 9, 2, 16, 128))),
    ("kv_keep", keep(v_pages=Fake(BF16, 9, 4, 16, 128))), ("kv_keep", keep(counts=Fake(I32, 3))),
    ("kv_keep", keep(path=Fake(I64, 0))), ("kv_keep", keep(prefix_len=1 << 32)),
    ("attn_q8", attn(q=Fake(F32, 0, 4, 128))), ("attn_q8", attn(q=Fake(BF16, 4, 128))),
    ("attn_q8", attn(R=2, q=Fake(BF16, 1, 4, 128))), ("attn_q8", attn(h_q=8)),
    ("attn_q8", {**attn(), "R": -1}), ("attn_q8", attn(h_kv=-1)), ("attn_q8", attn(h_kv=4)),
    ("attn_q8", attn(page_size=32)), ("attn_q8", attn(page_size=-1)), ("attn_q8", attn(B=2)),
    ("attn_q8", attn(page_table=Fake(I32, 24))), ("attn_q8", attn(window=1 << 31)),
    ("attn_q8", attn(k_pages=Fake(BF16, 9, 2, 16, 128))), ("attn_q8", attn(out=Fake(BF16, 0, 4, 128))),
    ("attn_q8", attn(bf16=True, out=Fake(F32, 0, 4, 128))), ("attn_q8", attn(lse=Fake(F32, 1, 4))),
    ("attn_q8", attn(v_pages=Fake(F8, 8, 2, 16, 128))), ("attn_q8", attn(prefix_len=1 << 31)),
    ("attn_tree", tree(masks=Fake(I32, 1, 1))), ("attn_tree", tree(masks=Fake(I64, 0, 1))),
    ("attn_tree", tree(masks=Fake(I32, 0))), ("attn_tree", tree(positions=Fake(I32, 1))),
    ("attn_tree", tree(positions=Fake(I32, 0, device=OTHER))), ("attn_tree", tree(h_kv=1)),
    ("attn_tree", tree(dtype=U8, page_size=32)), ("attn_tree", tree(v_pages=Fake(F8, 9, 2, 16, 128))),
    ("attn_tree", tree(out=Fake(F32, 0, 4, 64))), ("attn_tree", tree(sinks=-(1 << 40))),
    ("kv_keep", keep(dtype=F8, k_pages=Fake(F8, 9, 2, 16, 64), v_pages=Fake(F8, 9, 2, 16, 64))),
]


@pytest.mark.parametrize("name,args", REFUSED)
def test_refusals(host, name, args):
    module, fake = host
    with pytest.raises(ValueError) as e:
        getattr(module, name)(*args.values())
    assert not isinstance(e.value, binding.FanoutError) and fake.log == []


@pytest.mark.parametrize("name", CALLS)
def test_wrong_kinds_of_objects(host, name):
    module, fake = host
    names, args = list(CALLS[name]()), list(CALLS[name]().values())
    for bad in (args[:-1], args + [None], [None] + args[1:]):
        with pytest.raises((TypeError, AttributeError)):
            getattr(module, name)(*bad)
    for i in range(len(args)):  # any one argument of a type it cannot be
        if names[i] in ("causal", "bf16", "want_lse"):  # (truth values: anything has one)
            continue
        with pytest.raises((TypeError, AttributeError, ValueError)):
            getattr(module, name)(*args[:i], object(), *args[i + 1:])


@pytest.mark.parametrize("name", CALLS)
def test_nothing_is_kept(host, name):
    """Neither a call that succeeds nor one that is refused changes a reference count."""
    module, fake = host
    call = getattr(module, name)
    good = list(CALLS[name](stream=1 << 20).values())
    bad = [a for n, a in REFUSED if n == name]
    held = good + [x for a in bad for x in a.values()] + [
        DEV, OTHER, *TYPES, fake.empty.__func__, ()]

    def run(times):
        for _ in range(times):
            call(*good)
            for a in bad:
                try:
                    call(*a.values())
                except ValueError:
                    pass
            try:
                call(*good[:-1])
            except TypeError:
                pass
        fake.log.clear()
        fake.made.clear()
    run(3)
    before = [sys.getrefcount(x) for x in held]
    run(200)
    after = [sys.getrefcount(x) for x in held]
    assert all(b - a < 100 for a, b in zip(before, after)), (before, after)
