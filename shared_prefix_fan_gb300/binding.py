"""Python binding of libfanout.so: argument marshalling only (ctypes, and for the calls of
the 8-bit cache and of drafted trees the extension module _host_calls).

Every step of the attention path runs in the library's CUDA kernels; this
module turns torch tensors into pointers, checks dtypes/devices/shapes, calls
the C ABI and raises on a non-zero status. There is no fallback: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import sysconfig
from array import array
from typing import Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libfanout.so")
HOST_PATH = os.path.join(_HERE, "lib", "_host_calls" + sysconfig.get_config_var("EXT_SUFFIX"))

OK, EINVAL, EUNSUPPORTED, ECUDA, ENOMEM, ETIMEOUT = range(6)
OUT_F32, OUT_BF16 = 0, 1
OPT_SPLITS, OPT_VALIDATE_TABLE, OPT_WAIT_LIMIT_NS, OPT_NUM_SMS, OPT_FUSED_MERGE = 1, 2, 3, 4, 5

# The C ABI (include/fanout.h): name -> (restype, argtypes)
_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int32)
ABI = {
    "fanout_fork": (ctypes.c_int, [_i32p, _i32, _i32, _i32p, _i32, _i32p, _i32, _i32p, _i32]),
    "fanout_fork_cow": (ctypes.c_int, [_i32p, _i32, _i32, _i32p, _i32, _i32p, _i32, _i32p, _i32,
                                       _i32p, _i32p]),
    "fanout_copy_pages": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp]),
    "fanout_extend": (ctypes.c_int, [_i32p, _i32, _i32, _i32, _i32p, _i32p, _i32, _i32p, _i32,
                                     _i32p]),
    "fanout_kv_append": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32p, _i32p, _i32, _i32,
                                        _i32, _i32, _i32, _i32, _vp]),
    "fanout_attn": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32p, _i32p, _i32, _i32, _i32, _i32,
                                   _i32, _i32, _i32, _f32, _i32, _vp, _i32, _vp, _vp]),
    "fanout_attn_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32p, _i32p, _i32, _i32,
                                           _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp, _i32,
                                           _vp, _vp]),
    "fanout_fork_device": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _vp,
                                          _i32, _vp, _vp]),
    "fanout_fork_device_new": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp,
                                              _vp, _i32, _vp, _vp]),
    "fanout_extend_device": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _vp,
                                            _vp, _vp, _i64, _vp]),
    "fanout_kv_append_q4": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32, _i32,
                                           _i32, _i32, _f32, _f32, _vp]),
    "fanout_kv_read_q4": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _f32,
                                         _vp, _vp, _i64, _i64, _vp]),
    "fanout_attn_window": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32,
                                          _i32, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp,
                                          _i32, _vp, _vp]),
    "fanout_attn_q4": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                      _i32, _i32, _i32, _i32, _f32, _i32, _f32, _f32, _i32, _i32,
                                      _vp, _i32, _vp, _vp]),
    "fanout_kv_append_q8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _i32, _i32,
                                           _i32, _i32, _f32, _f32, _vp]),
    "fanout_kv_read_q8": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _f32,
                                         _vp, _vp, _i64, _i64, _vp]),
    "fanout_attn_q8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                      _i32, _i32, _i32, _i32, _f32, _i32, _f32, _f32, _i32, _i32,
                                      _vp, _i32, _vp, _vp]),
    "fanout_tree_rows": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32, _i64, _i32,
                                        _i32, _vp, _vp, _vp, _vp]),
    "fanout_tree_rows_sinks": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32, _i64,
                                              _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "fanout_tree_accept": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp,
                                          _vp]),
    "fanout_kv_keep": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                      _i64, _i32, _i32, _i32, _i32, _vp]),
    "fanout_attn_tree": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32,
                                        _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp, _i32, _i32,
                                        _f32, _f32, _vp, _i32, _vp, _vp]),
    "fanout_lse_merge": (ctypes.c_int, [_vp, _vp, _i32, _i64, _i32, _vp, _i32, _vp, _vp]),
    "fanout_last_error": (ctypes.c_int, [_vp]),
    "fanout_last_error_detail": (ctypes.c_int, [_vp, _i32p, _i32p]),
    "fanout_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "fanout_set_option": (ctypes.c_int, [_i32, _i64]),
    "fanout_set_profile_events": (ctypes.c_int, [_vp, _vp]),
    "fanout_plan": (ctypes.c_int, [_i32p, _i32p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32p,
                                   _i32, _i32p, _i32p, _i32, _i32p, _i32p]),
    "fanout_plan_step": (ctypes.c_int, [_i32p, _i32p, _i32p, _i32, _i32, _i32, _i32, _i32, _i32,
                                        _i32, _i32p, _i32, _i32p, _i32p, _i32, _i32p, _i32p,
                                        _i32p]),
    "fanout_selftest_wait_timeout": (ctypes.c_int, [_i64, _vp]),
    "fanout_read_floor": (ctypes.c_int, [_vp, _i64, _vp, _vp]),
    "fanout_release": (ctypes.c_int, []),
    "fanout_version": (ctypes.c_char_p, []),
}

_lib = None


class FanoutError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


def load(path: Optional[str] = None):
    """Load libfanout.so (built by shared_prefix_fan_gb300.build). Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libfanout.so not built ({p}); run shared_prefix_fan_gb300.build.build()")
    lib = ctypes.CDLL(p)
    for name, (res, args) in ABI.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    if path is None:
        _lib = lib
    return lib


_host = None


def _host_calls():
    """The extension module behind those calls (csrc/host_calls.c), set up with torch's
    functions. Raises if it has not been built."""
    global _host
    if _host is None:
        import importlib.machinery
        import importlib.util

        import torch
        load()
        if not os.path.exists(HOST_PATH):
            raise RuntimeError(f"_host_calls not built ({HOST_PATH}); run "
                               "shared_prefix_fan_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_host_calls", HOST_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_host_calls", loader))
        loader.exec_module(module)
        types = (torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32, torch.int64,
                 torch.float32)
        module.setup(types, torch.empty, torch._C._cuda_getCurrentRawStream,
                     torch._C._cuda_getDevice, torch.cuda.device, _empty_on, _stream_handle, _check)
        _host = module
    return _host


def strerror(code: int) -> str:
    try:
        return load().fanout_strerror(int(code)).decode()
    except RuntimeError:
        return f"status {code}"


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise FanoutError(rc, what)


def _i32arr(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(_i32p)


def version() -> str:
    return load().fanout_version().decode()


def fork(prefix_pages, suffix_lens, page_size: int, free_pages, max_pages: int) -> np.ndarray:
    """Branch page tables (host): row b = prefix ids + branch b's private ids, then -1."""
    pre, sl, fr = _i32arr(prefix_pages), _i32arr(suffix_lens), _i32arr(free_pages)
    nb = int(sl.shape[0])
    table = np.full((max(nb, 1), int(max_pages)), -1, dtype=np.int32)
    _check(load().fanout_fork(_ptr(pre), int(pre.shape[0]), nb, _ptr(sl), int(page_size),
                              _ptr(fr), int(fr.shape[0]), _ptr(table), int(max_pages)),
           "fanout_fork")
    return table[:nb]


def fork_cow(prefix_pages, prefix_len: int, suffix_lens, page_size: int, free_pages,
             max_pages: int):
    """Fork with a prefix that may end inside a page: (tables, cow_pairs [B, 2], used)."""
    pre, sl, fr = _i32arr(prefix_pages), _i32arr(suffix_lens), _i32arr(free_pages)
    nb = int(sl.shape[0])
    table = np.full((max(nb, 1), int(max_pages)), -1, dtype=np.int32)
    pairs = np.full((max(nb, 1), 2), -1, dtype=np.int32)
    used = ctypes.c_int32(0)
    _check(load().fanout_fork_cow(_ptr(pre), int(prefix_len), nb, _ptr(sl), int(page_size),
                                  _ptr(fr), int(fr.shape[0]), _ptr(table), int(max_pages),
                                  _ptr(pairs), ctypes.byref(used)), "fanout_fork_cow")
    return table[:nb], pairs[:nb], int(used.value)


def copy_pages(k_pages, v_pages, pairs, rows: int, stream=None) -> None:
    """Device copy of token slots [0, rows) for page pairs (int32 [n, 2] on the device)."""
    n, h_kv, page, d = (int(x) for x in k_pages.shape)
    _check(load().fanout_copy_pages(k_pages.data_ptr(), v_pages.data_ptr(), pairs.data_ptr(),
                                    int(pairs.shape[0]), int(rows), n, h_kv, d, page,
                                    _stream_handle(stream)), "fanout_copy_pages")


def extend(page_table, prefix_len: int, suffix_lens, add_lens, page_size: int, free_pages):
    """Grown copy of host page tables [B][max_pages] and the free pages used."""
    t = np.array(page_table, dtype=np.int32, copy=True, order="C")
    sl, al, fr = _i32arr(suffix_lens), _i32arr(add_lens), _i32arr(free_pages)
    used = ctypes.c_int32(0)
    _check(load().fanout_extend(_ptr(t), int(t.shape[0]), int(t.shape[1]), int(prefix_len),
                                _ptr(sl), _ptr(al), int(page_size), _ptr(fr), int(fr.shape[0]),
                                ctypes.byref(used)), "fanout_extend")
    return t, int(used.value)


def kv_append(k_new, v_new, k_pages, v_pages, page_table, prefix_len: int, suffix_lens,
              add_lens, page_size: int, stream=None) -> None:
    """Write new K/V rows [R, H_kv, d] (bf16, device) into the page pools in place."""
    import torch
    for name, t in (("k_new", k_new), ("v_new", v_new), ("k_pages", k_pages),
                    ("v_pages", v_pages)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    sl, al = _i32arr(suffix_lens), _i32arr(add_lens)
    _check(load().fanout_kv_append(
        k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        page_table.data_ptr(), int(prefix_len), _ptr(sl), _ptr(al), int(sl.shape[0]),
        int(page_table.shape[1]), int(k_pages.shape[0]), int(k_pages.shape[1]),
        int(k_pages.shape[3]), int(page_size), _stream_handle(stream)), "fanout_kv_append")


def _device_call(name: str, dev, stream, *args) -> None:
    """Call the library with `dev` current, on `stream` or on dev's current one.

    The serving calls below take a few microseconds of GPU time for a decode step,
    so their host side is kept short: raw stream handles, a device switch only when
    another device is current, one conversion for a call's host lengths."""
    import torch
    idx = dev.index
    handle = torch._C._cuda_getCurrentRawStream(idx) if stream is None else _stream_handle(stream)
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == idx:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(idx):
            rc = fn(*args, handle)
    if rc:
        raise FanoutError(rc, name)


_I32_MAX = 2 ** 31 - 1  # ctypes would take the low 32 bits of more


def _fit32(name: str, v: int) -> None:
    """For integers with bits past the 31st: negative ones are the library's to refuse."""
    if not -_I32_MAX - 1 <= v <= _I32_MAX:
        raise ValueError(f"{name}: {v} does not fit 32 bits")


def _empty_on(dev, stream):
    """torch.empty for the results of a call on `stream` (calls without one use
    torch.empty itself: dev's current stream).

    From another stream's pool than the one the call runs on, a result's block could
    still be read or written there by work queued before it was freed, and a result
    that is dropped early would be lent out again while the call has yet to write it.
    The caller may use and drop it on the current stream: its reuse waits for that."""
    import torch
    handle, here = _stream_handle(stream), torch.cuda.current_stream(dev)
    if handle == here.cuda_stream:
        return torch.empty
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(handle, device=dev) if handle > 1 else
                  torch.cuda.default_stream(dev))  # 0 and 1 name the default stream

    def empty(shape, dtype, device):
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
        t.record_stream(here)
        return t
    return empty


def _need(name: str, t, dtype, dev, shape=None) -> None:
    """A contiguous tensor of this type, on this CUDA device (and of this shape)."""
    if t.dtype is not dtype or t.device != dev or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on one CUDA device ({dev})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def fork_device(prefix_pages, prefix_len: int, suffix_lens, page_size: int, free_pages,
                max_pages: int, used=None, out=None, want_cow: bool = True, stream=None):
    """fork / fork_cow on the device: (tables [B, max_pages], cow_pairs, used).

    prefix_pages, suffix_lens, free_pages: int32 CUDA tensors; `used` (int32 [1],
    None: 0) counts the free-list entries already taken, the returned one those
    taken after this call. cow_pairs (int32 [B, 2]) is None when the prefix ends
    with its page or want_cow is false. What the lengths get wrong on the device
    is reported by last_error(); the call then hands out no page: cow_pairs and a
    table allocated here are -1 throughout, a given `out` is left as it was."""
    import torch
    i32, dev = torch.int32, suffix_lens.device
    B = suffix_lens.numel()
    if page_size <= 0:
        raise ValueError("page_size must be positive")
    if prefix_len >> 31 or page_size >> 31 or max_pages >> 31:
        _fit32("prefix_len", prefix_len)
        _fit32("page_size", page_size)
        _fit32("max_pages", max_pages)
    _need("suffix_lens", suffix_lens, i32, dev, (B,))
    _need("prefix_pages", prefix_pages, i32, dev)
    _need("free_pages", free_pages, i32, dev)
    if prefix_pages.numel() < -(-prefix_len // page_size):
        raise ValueError("prefix_pages holds fewer pages than the prefix")
    if used is not None:
        _need("used", used, i32, dev, (1,))
    empty = torch.empty if stream is None else _empty_on(dev, stream)
    name = "fanout_fork_device"
    if out is None:
        name = "fanout_fork_device_new"
        out = empty((B, max_pages), dtype=i32, device=dev)
    else:
        _need("out", out, i32, dev, (B, max_pages))
    cow = None
    if want_cow and prefix_len % page_size:
        cow = empty((B, 2), dtype=i32, device=dev)
    after = empty((1,), dtype=i32, device=dev)
    _device_call(name, dev, stream, prefix_pages.data_ptr(), prefix_len, B,
                 suffix_lens.data_ptr(), page_size, free_pages.data_ptr(), free_pages.numel(),
                 _ptr_or_none(used), after.data_ptr(), out.data_ptr(), max_pages,
                 _ptr_or_none(cow))
    return out, cow, after


def extend_device(page_table, prefix_len: int, suffix_lens, add_lens, page_size: int, free_pages,
                  n_slots: int, used=None, slots=None, stream=None):
    """extend on the device, page_table (int32 [B, max_pages]) in place: (slots, used).

    slots (int64 [n_slots]) maps the new tokens' rows for kv_append_q4; rows
    behind the last one get -1. `used` as in fork_device."""
    import torch
    i32, dev = torch.int32, page_table.device
    B, width = page_table.shape
    if prefix_len >> 31 or page_size >> 31:
        _fit32("prefix_len", prefix_len)
        _fit32("page_size", page_size)
    _need("page_table", page_table, i32, dev)
    _need("suffix_lens", suffix_lens, i32, dev, (B,))
    _need("add_lens", add_lens, i32, dev, (B,))
    _need("free_pages", free_pages, i32, dev)
    if used is not None:
        _need("used", used, i32, dev, (1,))
    empty = torch.empty if stream is None else _empty_on(dev, stream)
    if slots is None:
        slots = empty((n_slots,), dtype=torch.int64, device=dev)
    else:
        _need("slots", slots, torch.int64, dev, (n_slots,))
    after = empty((1,), dtype=i32, device=dev)
    _device_call("fanout_extend_device", dev, stream, page_table.data_ptr(), B, width, prefix_len,
                 suffix_lens.data_ptr(), add_lens.data_ptr(), page_size, free_pages.data_ptr(),
                 free_pages.numel(), _ptr_or_none(used), after.data_ptr(), slots.data_ptr(),
                 n_slots)
    return slots, after


# Bytes of one token and KV head in a 4-bit pool (FANOUT_Q4_ROW_BYTES in include/fanout.h).
Q4_ROW_BYTES = 72


def q4_pool(num_pages: int, h_kv: int, page_size: int, device="cuda"):
    """A zeroed 4-bit pool: uint8 [num_pages, H_kv, page_size * 72]."""
    import torch
    return torch.zeros((int(num_pages), int(h_kv), int(page_size) * Q4_ROW_BYTES),
                       dtype=torch.uint8, device=device)


def _q4_pools(k_pages, v_pages, page_size: int, dev):
    """(num_pages, H_kv) of a pair of 4-bit pools."""
    import torch
    shape = k_pages.shape
    _need("k_pages", k_pages, torch.uint8, dev)
    _need("v_pages", v_pages, torch.uint8, dev, shape)
    if len(shape) != 3 or shape[2] != page_size * Q4_ROW_BYTES:
        raise ValueError(f"k_pages / v_pages must be [num_pages, H_kv, page_size * {Q4_ROW_BYTES}]")
    return shape[0], shape[1]


def _rows_of(name: str, t, n: int, h_kv: int, dev) -> int:
    """Elements between the rows of a bf16 [n, H_kv, d] tensor whose heads are packed."""
    import torch
    if t.dtype is not torch.bfloat16 or t.device != dev or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 tensor on {dev}")
    shape = t.shape
    if len(shape) != 3 or shape[0] != n or shape[1] != h_kv:
        raise ValueError(f"{name} must be [{n}, {h_kv}, d]")
    row = h_kv * shape[2]
    if n == 0:
        return row
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h_kv > 1 and s1 != shape[2]):
        raise ValueError(f"{name}: a row's heads must be packed")
    return s0 if n > 1 else row


def kv_append_q4(k_new, v_new, k_pages, v_pages, slots, page_size: int, k_scale: float = 1.0,
                 v_scale: float = 1.0, stream=None) -> None:
    """Write new K/V rows (bf16 [R, H_kv, 128], rows may be strided) into 4-bit
    pools at `slots` (int64 [R]; negative: the row is skipped)."""
    import torch
    dev, n = k_pages.device, slots.numel()
    num_pages, h_kv = _q4_pools(k_pages, v_pages, page_size, dev)
    _need("slots", slots, torch.int64, dev, (n,))
    ks, vs = _rows_of("k_new", k_new, n, h_kv, dev), _rows_of("v_new", v_new, n, h_kv, dev)
    d = k_new.shape[2]
    if v_new.shape[2] != d:
        raise ValueError("k_new / v_new differ in shape")
    _device_call("fanout_kv_append_q4", dev, stream, k_new.data_ptr(), v_new.data_ptr(), ks, vs,
                 k_pages.data_ptr(), v_pages.data_ptr(), slots.data_ptr(), n, num_pages, h_kv, d,
                 page_size, k_scale, v_scale)


def kv_read_q4(k_pages, v_pages, slots, page_size: int, k_scale: float = 1.0,
               v_scale: float = 1.0, k_out=None, v_out=None, stream=None):
    """The bf16 rows [R, H_kv, 128] that `slots` of 4-bit pools stand for: (k, v).
    Rows with a negative slot are left as they were (undefined when allocated here)."""
    import torch
    dev, n = k_pages.device, slots.numel()
    num_pages, h_kv = _q4_pools(k_pages, v_pages, page_size, dev)
    _need("slots", slots, torch.int64, dev, (n,))
    empty = torch.empty if stream is None else _empty_on(dev, stream)
    if k_out is None:
        k_out = empty((n, h_kv, 128), dtype=torch.bfloat16, device=dev)
    if v_out is None:
        v_out = empty((n, h_kv, 128), dtype=torch.bfloat16, device=dev)
    ks, vs = _rows_of("k_out", k_out, n, h_kv, dev), _rows_of("v_out", v_out, n, h_kv, dev)
    d = k_out.shape[2]
    if v_out.shape[2] != d:
        raise ValueError("k_out / v_out differ in shape")
    _device_call("fanout_kv_read_q4", dev, stream, k_pages.data_ptr(), v_pages.data_ptr(),
                 slots.data_ptr(), n, num_pages, h_kv, d, page_size, k_scale, v_scale,
                 k_out.data_ptr(), v_out.data_ptr(), ks, vs)
    return k_out, v_out


def copy_pages_q4(k_pages, v_pages, pairs, page_size: int, stream=None) -> None:
    """Copy whole pages of 4-bit pools for page pairs (int32 [n, 2] on the device):
    the copy-on-write step of a fork whose prefix ends inside a page."""
    import torch
    if page_size % 2:
        raise ValueError("page_size of a 4-bit pool is 16, 32, 64 or 128")
    dev = k_pages.device
    num_pages, h_kv = _q4_pools(k_pages, v_pages, page_size, dev)
    _need("pairs", pairs, torch.int32, dev, (pairs.shape[0], 2))
    # a block of page_size * 72 bytes as page_size / 2 rows of 72 16-bit values
    _device_call("fanout_copy_pages", dev, stream, k_pages.data_ptr(), v_pages.data_ptr(),
                 pairs.data_ptr(), pairs.shape[0], page_size // 2, num_pages, h_kv, Q4_ROW_BYTES,
                 page_size // 2)


def q8_pool(num_pages: int, h_kv: int, page_size: int, device="cuda"):
    """A zeroed 8-bit pool: float8_e4m3fn [num_pages, H_kv, page_size, 128]."""
    import torch
    shape = (int(num_pages), int(h_kv), int(page_size), 128)
    return torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)


def _q8_pools(k_pages, v_pages, dev):
    """(num_pages, H_kv, page_size, d) of a pair of 8-bit pools."""
    import torch
    shape = k_pages.shape
    _need("k_pages", k_pages, torch.float8_e4m3fn, dev)
    _need("v_pages", v_pages, torch.float8_e4m3fn, dev, shape)
    if len(shape) != 4:
        raise ValueError("k_pages / v_pages must be [num_pages, H_kv, page_size, d]")
    return shape


def kv_append_q8(k_new, v_new, k_pages, v_pages, slots, k_scale: float = 1.0,
                 v_scale: float = 1.0, stream=None) -> None:
    """Write new K/V rows (bf16 [R, H_kv, 128], rows may be strided) into 8-bit
    pools at `slots` (int64 [R]; negative: the row is skipped)."""
    (_host or _host_calls()).kv_append_q8(k_new, v_new, k_pages, v_pages, slots, k_scale, v_scale,
                                          stream)


def kv_read_q8(k_pages, v_pages, slots, k_scale: float = 1.0, v_scale: float = 1.0, k_out=None,
               v_out=None, stream=None):
    """The bf16 rows [R, H_kv, 128] that `slots` of 8-bit pools stand for: (k, v).
    Rows with a negative slot are left as they were (undefined when allocated here)."""
    return (_host or _host_calls()).kv_read_q8(k_pages, v_pages, slots, k_scale, v_scale, k_out,
                                               v_out, stream)


def copy_pages_q8(k_pages, v_pages, pairs, rows: int, stream=None) -> None:
    """copy_pages for 8-bit pools: token slots [0, rows) of page pairs (int32 [n, 2])."""
    import torch
    dev = k_pages.device
    num_pages, h_kv, page_size, d = _q8_pools(k_pages, v_pages, dev)
    _need("pairs", pairs, torch.int32, dev, (pairs.shape[0], 2))
    # a row of d bytes as d / 2 16-bit values
    _device_call("fanout_copy_pages", dev, stream, k_pages.data_ptr(), v_pages.data_ptr(),
                 pairs.data_ptr(), pairs.shape[0], rows, num_pages, h_kv, d // 2, page_size)


def tree_rows(parents, page_table, prefix_len: int, suffix_lens, add_lens, page_size: int,
              max_nodes: int, window: int = 0, masks=None, positions=None, slots=None, stream=None,
              sinks: int = 0):
    """What a step's drafted rows need: (masks int32 [R, words], positions int32 [R],
    slots int64 [R]).

    parents (int32 [R], rows grouped by branch): each drafted token's parent in its
    branch, or -1; suffix_lens / add_lens (int32 [B]): private tokens before the draft, and
    drafted ones, at most max_nodes (<= 1024) each. Bit u of a token's mask is set for
    itself and its ancestors (with a window, those less than `window` levels above it and
    those at positions below `sinks`: give what the layer's attention is given);
    its position is prefix + suffix + its depth; its slot is where its K/V row belongs.
    Rows behind the last token get no bits, position 0 and slot -1."""
    if max_nodes < 1 or max_nodes > 1024:
        raise ValueError("max_nodes must be 1 .. 1024")
    if window >> 31 or sinks >> 31:
        window, sinks = max(-1, min(window, _I32_MAX)), max(-1, min(sinks, _I32_MAX))
    host, words = _host or _host_calls(), (max_nodes + 31) // 32
    if sinks:
        return host.tree_rows_sinks(parents, page_table, prefix_len, suffix_lens, add_lens, page_size,
                                    words, window, sinks, masks, positions, slots, stream)
    return host.tree_rows(parents, page_table, prefix_len, suffix_lens, add_lens, page_size, words,
                          window, masks, positions, slots, stream)


def tree_accept(parents, draft_tokens, target_tokens, first_tokens, add_lens, stream=None):
    """The drafted tokens that the model agrees with: (path int32 [R], counts int32
    [B], next_tokens int64 [B]).

    draft_tokens / target_tokens (int64 [R]): each node's token, and the one the model
    picked behind it; first_tokens (int64 [B]): the one picked behind the context. Of each
    branch's rows of `path` the first counts[b] hold the accepted nodes, the others -1."""
    return (_host or _host_calls()).tree_accept(parents, draft_tokens, target_tokens, first_tokens,
                                                add_lens, stream)


def kv_keep(k_pages, v_pages, page_table, prefix_len: int, suffix_lens, add_lens, path, counts,
            page_size: int, stream=None) -> None:
    """Move the accepted rows together in pools of any kind: drafted row path[i] of a
    branch becomes its row i (path, counts as tree_accept gives them; suffix_lens without
    the drafted tokens)."""
    (_host or _host_calls()).kv_keep(k_pages, v_pages, page_table, prefix_len, suffix_lens, add_lens,
                                     path, counts, page_size, stream)


def plan(suffix_lens, q_rows, prefix_len: int, h_q: int, h_kv: int, page_size: int,
         causal: bool, num_sms: int = 152) -> Tuple[np.ndarray, np.ndarray, int]:
    """The work plan fanout_attn would run: (units [n, 8], cta_first [n_cta+1], n_parts)."""
    sl, tq = _i32arr(suffix_lens), _i32arr(q_rows)
    lib = load()
    n_units, n_ctas, n_parts = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    args = (_ptr(sl), _ptr(tq), int(sl.shape[0]), int(prefix_len), int(h_q), int(h_kv),
            int(page_size), int(bool(causal)), int(num_sms))
    _check(lib.fanout_plan(*args, None, 0, ctypes.byref(n_units), None, 0, ctypes.byref(n_ctas),
                           ctypes.byref(n_parts)), "fanout_plan")
    units = np.zeros((max(n_units.value, 1), 8), dtype=np.int32)
    cta = np.zeros(n_ctas.value + 1, dtype=np.int32)
    _check(lib.fanout_plan(*args, _ptr(units), int(units.shape[0]), ctypes.byref(n_units),
                           _ptr(cta), int(cta.shape[0]), ctypes.byref(n_ctas),
                           ctypes.byref(n_parts)), "fanout_plan")
    return units[:n_units.value], cta, int(n_parts.value)


def plan_step(prev_suffix_lens, suffix_lens, q_rows, prefix_len: int, h_q: int, h_kv: int,
              page_size: int, causal: bool, num_sms: int = 152):
    """The plan fanout_attn runs after a call that differed only in suffix
    lengths: (units [n, 8], cta_first [n_cta+1], n_parts, reused)."""
    ps_, sl, tq = _i32arr(prev_suffix_lens), _i32arr(suffix_lens), _i32arr(q_rows)
    lib = load()
    n_units, n_ctas, n_parts, reused = (ctypes.c_int32(0) for _ in range(4))
    args = (_ptr(ps_), _ptr(sl), _ptr(tq), int(sl.shape[0]), int(prefix_len), int(h_q),
            int(h_kv), int(page_size), int(bool(causal)), int(num_sms))
    _check(lib.fanout_plan_step(*args, None, 0, ctypes.byref(n_units), None, 0,
                                ctypes.byref(n_ctas), ctypes.byref(n_parts), None),
           "fanout_plan_step")
    units = np.zeros((max(n_units.value, 1), 8), dtype=np.int32)
    cta = np.zeros(n_ctas.value + 1, dtype=np.int32)
    _check(lib.fanout_plan_step(*args, _ptr(units), int(units.shape[0]), ctypes.byref(n_units),
                                _ptr(cta), int(cta.shape[0]), ctypes.byref(n_ctas),
                                ctypes.byref(n_parts), ctypes.byref(reused)), "fanout_plan_step")
    return units[:n_units.value], cta, int(n_parts.value), bool(reused.value)


def set_option(option: int, value: int) -> None:
    _check(load().fanout_set_option(int(option), int(value)), "fanout_set_option")


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(getattr(stream, "cuda_stream", stream))


def attn(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens: Sequence[int],
         q_rows: Sequence[int], h_q: int, h_kv: int, page_size: int, scale: float,
         causal: bool, out=None, lse=None, out_dtype: str = "f32", want_lse: bool = True,
         stream=None):
    """Fan-out attention through fanout_attn. Device tensors in, (out, lse) back.

    q: bf16 [R, H_q, d]; k_pages / v_pages: bf16 [num_pages, H_kv, page, d];
    page_table: int32 [B, max_pages] on the same device; suffix_lens / q_rows:
    host sequences of length B. `out` / `lse` are allocated when not given.
    """
    import torch
    lib = load()
    sl, tq = _i32arr(suffix_lens), _i32arr(q_rows)
    R = int(tq.sum())
    d = int(q.shape[-1])
    dev = q.device
    for name, t, dt in (("q", q, torch.bfloat16), ("k_pages", k_pages, torch.bfloat16),
                        ("v_pages", v_pages, torch.bfloat16), ("page_table", page_table, torch.int32)):
        if t.dtype != dt or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} tensor on {dev}")
    if tuple(q.shape) != (R, h_q, d):
        raise ValueError(f"q shape {tuple(q.shape)} != {(R, h_q, d)}")
    if k_pages.shape != v_pages.shape or k_pages.dim() != 4:
        raise ValueError("k_pages / v_pages must be [num_pages, H_kv, page, d]")
    odt = {"f32": (torch.float32, OUT_F32), "bf16": (torch.bfloat16, OUT_BF16)}[out_dtype]
    empty = torch.empty if stream is None else _empty_on(dev, stream)
    if out is None:
        out = empty((R, h_q, d), dtype=odt[0], device=dev)
    if lse is None and want_lse:
        lse = empty((R, h_q), dtype=torch.float32, device=dev)
    if out.dtype != odt[0] or not out.is_contiguous():
        raise ValueError("out dtype/layout mismatch")
    rc = lib.fanout_attn(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                         page_table.data_ptr(), int(prefix_len), _ptr(sl), _ptr(tq),
                         int(sl.shape[0]), int(page_table.shape[1]) if page_table.dim() == 2 else 0,
                         int(k_pages.shape[0]), int(h_q), int(h_kv), d, int(page_size),
                         float(scale), int(bool(causal)), out.data_ptr(), odt[1],
                         lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    _check(rc, "fanout_attn")
    return out, lse


def _lens(suffix_lens, q_rows):
    """Host lengths of a call as one int32 array [2, B]: (array, address, B, rows)."""
    if len(suffix_lens) != len(q_rows):
        raise ValueError("suffix_lens and q_rows differ in length")
    if type(suffix_lens) is list and type(q_rows) is list:
        ints = array("i", suffix_lens + q_rows)
        return ints, ints.buffer_info()[0], len(q_rows), sum(q_rows)
    wide = np.array((suffix_lens, q_rows), dtype=np.int64)
    if wide.ndim != 2:
        raise ValueError("suffix_lens and q_rows must be sequences of integers")
    both = wide.astype(np.int32)
    if (both != wide).any():
        raise ValueError("suffix_lens / q_rows: a length does not fit 32 bits")
    return both, both.ctypes.data, both.shape[1], int(both[1].sum())


def _attn_out(q, page_table, R: int, B: int, h_q: int, out, lse, out_dtype: str, want_lse: bool,
              stream):
    """Checks and outputs the two calls below share: (out dtype code, out, lse)."""
    import torch
    dev, d = q.device, q.shape[-1]
    if out_dtype not in ("f32", "bf16"):
        raise ValueError("out_dtype must be 'f32' or 'bf16'")
    dt, code = (torch.float32, OUT_F32) if out_dtype == "f32" else (torch.bfloat16, OUT_BF16)
    shape = (R, h_q, d)
    _need("q", q, torch.bfloat16, dev, shape)
    _need("page_table", page_table, torch.int32, dev)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [num_branches, max_pages]")
    empty = torch.empty if stream is None else _empty_on(dev, stream)
    if out is None:
        out = empty(shape, dtype=dt, device=dev)
    else:
        _need("out", out, dt, dev, shape)
    if lse is not None:
        _need("lse", lse, torch.float32, dev, (R, h_q))
    elif want_lse:
        lse = empty((R, h_q), dtype=torch.float32, device=dev)
    return code, out, lse


def attn_window(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens, q_rows, h_q: int,
                h_kv: int, page_size: int, scale: float, window: int, sinks: int = 0, out=None,
                lse=None, out_dtype: str = "f32", want_lse: bool = True, stream=None):
    """attn(), causal, where a row at pos sees keys j <= pos with j > pos - window
    or j < sinks. Pages that no row sees may have been given back."""
    import torch
    if window >> 31 or sinks >> 31:
        window, sinks = max(-1, min(window, _I32_MAX)), max(-1, min(sinks, _I32_MAX))
    if prefix_len >> 31:
        _fit32("prefix_len", prefix_len)
    held, lens, B, R = _lens(suffix_lens, q_rows)
    code, out, lse = _attn_out(q, page_table, R, B, h_q, out, lse, out_dtype, want_lse,
                               stream)
    dev, d = q.device, q.shape[-1]
    num_pages = k_pages.shape[0]
    pool = (num_pages, h_kv, page_size, d)
    _need("k_pages", k_pages, torch.bfloat16, dev, pool)
    _need("v_pages", v_pages, torch.bfloat16, dev, pool)
    _device_call("fanout_attn_window", dev, stream, q.data_ptr(), k_pages.data_ptr(),
                 v_pages.data_ptr(), page_table.data_ptr(), prefix_len, lens, lens + 4 * B, B,
                 page_table.shape[1], num_pages, h_q, h_kv, d, page_size, scale, window, sinks,
                 out.data_ptr(), code, _ptr_or_none(lse))
    return out, lse


def attn_q4(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens, q_rows, h_q: int,
            h_kv: int, page_size: int, scale: float, causal: bool, k_scale: float = 1.0,
            v_scale: float = 1.0, window: int = 0, sinks: int = 0, out=None, lse=None,
            out_dtype: str = "f32", want_lse: bool = True, stream=None):
    """attn() over 4-bit pools (uint8 [num_pages, H_kv, page_size * 72]); window and
    sinks as in attn_window (0, 0: none)."""
    if window >> 31 or sinks >> 31:
        window, sinks = max(-1, min(window, _I32_MAX)), max(-1, min(sinks, _I32_MAX))
    if prefix_len >> 31:
        _fit32("prefix_len", prefix_len)
    held, lens, B, R = _lens(suffix_lens, q_rows)
    code, out, lse = _attn_out(q, page_table, R, B, h_q, out, lse, out_dtype, want_lse,
                               stream)
    dev = q.device
    num_pages, heads = _q4_pools(k_pages, v_pages, page_size, dev)
    if heads != h_kv:
        raise ValueError(f"pools hold {heads} KV heads, not {h_kv}")
    _device_call("fanout_attn_q4", dev, stream, q.data_ptr(), k_pages.data_ptr(),
                 v_pages.data_ptr(), page_table.data_ptr(), prefix_len, lens, lens + 4 * B, B,
                 page_table.shape[1], num_pages, h_q, h_kv, q.shape[-1], page_size, scale,
                 1 if causal else 0, k_scale, v_scale, window, sinks, out.data_ptr(), code,
                 _ptr_or_none(lse))
    return out, lse


def _bf16_out(out_dtype: str) -> bool:
    if out_dtype not in ("f32", "bf16"):
        raise ValueError("out_dtype must be 'f32' or 'bf16'")
    return out_dtype == "bf16"


def attn_q8(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens, q_rows, h_q: int,
            h_kv: int, page_size: int, scale: float, causal: bool, k_scale: float = 1.0,
            v_scale: float = 1.0, window: int = 0, sinks: int = 0, out=None, lse=None,
            out_dtype: str = "f32", want_lse: bool = True, stream=None):
    """attn() over 8-bit pools (float8_e4m3fn [num_pages, H_kv, page_size, 128]); window
    and sinks as in attn_window (0, 0: none)."""
    if window >> 31 or sinks >> 31:
        window, sinks = max(-1, min(window, _I32_MAX)), max(-1, min(sinks, _I32_MAX))
    if prefix_len >> 31:
        _fit32("prefix_len", prefix_len)
    held, lens, B, R = _lens(suffix_lens, q_rows)
    return (_host or _host_calls()).attn_q8(
        q, k_pages, v_pages, page_table, prefix_len, lens, B, R, h_q, h_kv, page_size, scale, causal,
        window, sinks, k_scale, v_scale, out, lse, _bf16_out(out_dtype), want_lse, stream)


def attn_tree(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens, q_rows, h_q: int,
              h_kv: int, page_size: int, scale: float, masks, positions=None, window: int = 0,
              sinks: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None,
              out_dtype: str = "f32", want_lse: bool = True, stream=None):
    """attn() for trees of drafted tokens, the last q_rows[b] <= 1024 tokens of a branch's
    suffix (suffix_lens counts them): a row sees the keys before its branch's draft (with
    a window those past position - window and the first `sinks`), itself, and the drafted
    tokens that its mask names (masks int32 [R, words], positions int32 [R]: tree_rows
    gives them; positions are read with a window only, and keys that a token right behind the
    context would see must be good whatever they say). Pools of any kind: bf16, 4 bits
    (uint8), 8 bits (float8_e4m3fn)."""
    if window >> 31 or sinks >> 31:
        window, sinks = max(-1, min(window, _I32_MAX)), max(-1, min(sinks, _I32_MAX))
    if prefix_len >> 31:
        _fit32("prefix_len", prefix_len)
    held, lens, B, R = _lens(suffix_lens, q_rows)
    return (_host or _host_calls()).attn_tree(
        q, k_pages, v_pages, page_table, prefix_len, lens, B, R, h_q, h_kv, page_size, scale, masks,
        positions, window, sinks, k_scale, v_scale, out, lse, _bf16_out(out_dtype), want_lse, stream)


# Fixed scratch of fanout_attn_noalloc (FANOUT_NOALLOC_SCRATCH_BYTES in include/fanout.h).
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def attn_noalloc(q, k_pages, v_pages, page_table, prefix_len: int, suffix_lens, q_rows,
                 h_q: int, h_kv: int, page_size: int, scale: float, causal: bool, out, lse,
                 out_dtype: str = "f32", stream=None) -> int:
    """fanout_attn_noalloc: same call as attn() into caller-allocated out/lse,
    for callers that must not allocate device memory during a call (the library
    uses its fixed scratch array instead of a cudaMalloc'd workspace). Returns
    the status code (FANOUT_ENOMEM when the problem needs more scratch than the
    fixed array holds) instead of raising, and allocates nothing itself."""
    sl, tq = _i32arr(suffix_lens), _i32arr(q_rows)
    odt = {"f32": OUT_F32, "bf16": OUT_BF16}[out_dtype]
    return int(load().fanout_attn_noalloc(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
        int(prefix_len), _ptr(sl), _ptr(tq), int(sl.shape[0]), int(page_table.shape[1]),
        int(k_pages.shape[0]), int(h_q), int(h_kv), int(q.shape[-1]), int(page_size),
        float(scale), int(bool(causal)), out.data_ptr(), odt,
        lse.data_ptr() if lse is not None else None, _stream_handle(stream)))


def lse_merge(part_o, part_ml, out=None, lse=None, out_dtype: str = "f32", stream=None):
    """Merge partials: part_o fp32 [P, N, d], part_ml fp32 [P, N, 2] -> (out [N, d], lse [N])."""
    import torch
    n_parts, n_out, d = (int(x) for x in part_o.shape)
    odt = {"f32": (torch.float32, OUT_F32), "bf16": (torch.bfloat16, OUT_BF16)}[out_dtype]
    empty = torch.empty if stream is None else _empty_on(part_o.device, stream)
    if out is None:
        out = empty((n_out, d), dtype=odt[0], device=part_o.device)
    if lse is None:
        lse = empty((n_out,), dtype=torch.float32, device=part_o.device)
    _check(load().fanout_lse_merge(part_o.data_ptr(), part_ml.data_ptr(), n_parts, n_out, d,
                                   out.data_ptr(), odt[1], lse.data_ptr(), _stream_handle(stream)),
           "fanout_lse_merge")
    return out, lse


def last_error(stream=None) -> int:
    return int(load().fanout_last_error(_stream_handle(stream)))


def last_error_detail(stream=None) -> Tuple[int, int, int]:
    """(status, wait site, CTA) of the device error word, then cleared."""
    site, block = ctypes.c_int32(0), ctypes.c_int32(0)
    rc = load().fanout_last_error_detail(_stream_handle(stream), ctypes.byref(site),
                                         ctypes.byref(block))
    return int(rc), int(site.value), int(block.value)


def set_profile_events(before=None, after=None) -> None:
    """Record torch.cuda.Event objects around the split-KV kernel (None, None: off)."""
    b = before.cuda_event if before is not None else None
    a = after.cuda_event if after is not None else None
    _check(load().fanout_set_profile_events(b, a), "fanout_set_profile_events")


def selftest_wait_timeout(limit_ns: int = 20_000_000, stream=None) -> int:
    return int(load().fanout_selftest_wait_timeout(int(limit_ns), _stream_handle(stream)))


def read_floor(buf, xor_out, stream=None) -> None:
    """One plain streaming read of the device tensor `buf` (all its bytes);
    *xor_out (a 1-element int32/uint32 CUDA tensor) ^= the xor of its words."""
    import torch
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    if not xor_out.is_cuda or xor_out.dtype not in (torch.int32, torch.uint32):
        raise ValueError("xor_out must be an int32 CUDA tensor")
    _check(load().fanout_read_floor(buf.data_ptr(), int(buf.numel() * buf.element_size()),
                                    xor_out.data_ptr(), _stream_handle(stream)),
           "fanout_read_floor")


def release() -> None:
    _check(load().fanout_release(), "fanout_release")
