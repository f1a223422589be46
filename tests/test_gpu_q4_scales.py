"""The 4-bit cache with a scale of its own for K and for V, at the ends of the pool
scales and at the ends of the group scales."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import ensure_lib
from .q4_problem import TwoScales
from .test_gpu_q4_rows import rows_like, same_codes

pytestmark = pytest.mark.gpu
P_STEP = 2.0 ** -11  # half a step of f16, the type P is rounded to


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


SHAPES = [  # S, T, P, hq, hkv, page: single tokens, ragged ones, a prefill behind a prefix
    ([1, 70, 300], [1, 1, 1], 500, 16, 2, 32), ([40, 3, 90], [7, 0, 33], 77, 10, 2, 16),
    ([330], [330], 50, 8, 1, 64), ([90, 64], [40, 25], 130, 14, 2, 128),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 60, 4),
                                                 (True, 200, 150), (True, 1, 0)])
@pytest.mark.parametrize("ks,vs", [(0.5, 4.0), (3.0, 0.02)])
def test_attention(shape, causal, window, sinks, ks, vs):
    prob = TwoScales(*shape, ks, vs, causal=causal, window=window, sinks=sinks, seed=11)
    want = prob.reference()
    for out_dtype in ("f32", "bf16"):
        out, lse = prob.run(out_dtype)
        assert binding.last_error() == binding.OK
        ref.check_attention(out, lse, want, P_STEP)


def held_rows(pools, slots, page):
    """(code words, scale bytes) of slots of a pool, [rows, H_kv, ...]."""
    w, b = ref.parts_of(pools.cpu().numpy(), page)
    return w[slots // page, :, slots % page], b[slots // page, :, slots % page]


@pytest.mark.parametrize("ks,vs", [(0.5, 4.0), (1e-30, 1e30), (1e30, 1e-30), (3.3e-30, 7.7e29)])
@pytest.mark.parametrize("page", [16, 64])
def test_append_and_read(ks, vs, page):
    rng = np.random.default_rng(page)
    n, hkv = 150, 3
    pages = -(-n // page) + 1
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    k, v = rows_like(rng, n, hkv, ks), rows_like(rng, n, hkv, 0.3 * vs)
    k[0], v[1] = 0.0, float("inf")
    k[2], v[3] = float("-inf"), torch.finfo(torch.bfloat16).tiny
    pools = [binding.q4_pool(pages, hkv, page) for _ in range(2)]
    at = torch.from_numpy(slots).cuda()
    binding.kv_append_q4(k.cuda(), v.cuda(), *pools, at, page, ks, vs)
    got = binding.kv_read_q4(*pools, at, page, ks, vs)
    assert binding.last_error() == binding.OK
    for x, pool, out, gs in ((k, pools[0], got[0], ks), (v, pools[1], got[1], vs)):
        words, byte = ref.encode(x.float().numpy(), gs)
        gw, gb = held_rows(pool, slots, page)
        assert np.array_equal(gb, byte)
        same_codes(gw, words, byte)
        want = torch.from_numpy(ref.decode(words, byte, gs).astype(np.float32)).bfloat16()
        assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("gs", [1e-30, 1.7e-30, 1e30, 0.37])
def test_every_border_between_codes(gs):
    """Values on and beside every border between two codes, for every group scale but 0,
    at the ends of the pool scales: there a quotient's remainder is a subnormal."""
    ties = (ref.LEVELS[1:] + ref.LEVELS[:-1]) / 2
    rows = []
    for byte in range(1, 127):
        den = np.float32(ref.E4M3[byte]) * np.float32(gs)
        x = np.concatenate([ties * den, -ties * den, [6.0 * den, 0.0]])
        for nudge in (0, 1, -1):
            b = torch.tensor(x, dtype=torch.float32).bfloat16()
            b = torch.where(b == 0, b, (b.view(torch.int16) + nudge).view(torch.bfloat16))
            b[14] = float(6.0 * den)
            rows.append(b)
    x = torch.stack(rows)[:len(rows) // 8 * 8].reshape(-1, 1, 128)
    n = x.shape[0]
    pools = [binding.q4_pool(-(-n // 16), 1, 16) for _ in range(2)]
    binding.kv_append_q4(x.cuda(), -x.cuda(), *pools, torch.arange(n, device="cuda"), 16, gs, gs)
    assert binding.last_error() == binding.OK
    for pool, y in zip(pools, (x, -x)):
        words, byte = ref.encode(y.float().numpy(), gs)
        gw, gb = held_rows(pool, np.arange(n), 16)
        assert np.array_equal(gb, byte)
        same_codes(gw, words, byte)


# scale bytes a pool may hold, and the K scale that brings its scores near 1
BYTES = {"zero and subnormal": (0x00, 0x08, 32.0), "subnormal": (0x01, 0x08, 32.0),
         "smallest normal": (0x08, 0x10, 16.0), "middle": (0x30, 0x48, 0.25),
         "largest": (0x78, 0x7f, 2.0 ** -9), "saturated": (0x7e, 0x7f, 2.0 ** -9),
         "all": (0x00, 0x7f, 2.0 ** -9)}


@pytest.mark.parametrize("name", list(BYTES))
@pytest.mark.parametrize("S,T,P,window", [([100], [5], 60, 0), ([200, 31], [60, 2], 70, 90)])
def test_attention_over_every_group_scale(name, S, T, P, window):
    """Any codes under any group scales: subnormal ones and the largest among them, codes
    up to 6 (2688 in the widened tile) and both zeros."""
    lo, hi, ks = BYTES[name]
    prob = TwoScales(S, T, P, 8, 2, 16, ks, 3.0, window=window, sinks=2 if window else 0, seed=4)
    rng = np.random.default_rng(lo + hi)
    pools = []
    for pool in (prob.k_pool, prob.v_pool):
        words, byte = ref.parts_of(pool.numpy(), 16)
        words = rng.integers(0, 1 << 32, words.shape, dtype=np.uint32)
        byte = rng.integers(lo, hi, byte.shape).astype(np.uint8)
        byte[np.broadcast_to(prob.hidden[:, None, :], byte.shape[:3])] = 0x7f
        pools.append(torch.from_numpy(ref.pool_of(words, byte)))
    prob.k_pool, prob.v_pool = pools
    prob.hold()
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    ref.check_attention(out, lse, prob.reference(), P_STEP, name)


def test_decode_steps():
    """Fork inside a page, then steps of: grow the tables, append, attend (with and
    without a window), K and V under scales of their own."""
    page, hkv, hq, P, ks, vs, W, sinks = 16, 2, 8, 40, 0.25, 2.0, 30, 3
    rng = np.random.default_rng(2)
    to = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    ids = rng.permutation(40).astype(np.int32)
    pools = [binding.q4_pool(40, hkv, page) for _ in range(2)]
    k, v = rows_like(rng, P, hkv, 1.0), rows_like(rng, P, hkv, 1.0)
    slots = ids[np.arange(P) // page].astype(np.int64) * page + np.arange(P) % page
    binding.kv_append_q4(k.cuda(), v.cuda(), *pools, torch.from_numpy(slots).cuda(), page, ks, vs)
    S = np.zeros(3, np.int64)
    table, cow, used = binding.fork_device(to(ids[:3]), P, to(S), page, to(ids[3:]), 6)
    binding.copy_pages_q4(*pools, cow, page)
    for step in range(8):
        A = np.array([1, 2, 1 + step % 3])
        R = int(A.sum())
        slots, used = binding.extend_device(table, P, to(S), to(A), page, to(ids[3:]), R, used)
        k, v = rows_like(rng, R, hkv, 1.0), rows_like(rng, R, hkv, 1.0)
        binding.kv_append_q4(k.cuda(), v.cuda(), *pools, slots, page, ks, vs)
        at = slots.cpu().numpy()
        for x, pool, gs in ((k, pools[0], ks), (v, pools[1], vs)):
            words, byte = ref.encode(x.float().numpy(), gs)
            gw, gb = held_rows(pool, at, page)
            assert np.array_equal(gb, byte)
            same_codes(gw, words, byte)
        S = S + A
        q = torch.from_numpy(rng.standard_normal((R, hq, 128)).astype(np.float32)).bfloat16()
        w, s0 = (W, sinks) if step % 2 else (0, 0)
        out, lse = binding.attn_q4(q.cuda(), *pools, table, P, S, A, hq, hkv, page, 128 ** -0.5,
                                   True, ks, vs, w, s0)
        assert binding.last_error() == binding.OK
        k64, v64 = (ref.decode(*ref.parts_of(p.cpu().numpy(), page), gs)
                    for p, gs in zip(pools, (ks, vs)))
        want = ref.attention(q.double().numpy(), k64, v64, table.cpu().numpy(), P, S, A, page,
                             128 ** -0.5, True, w, s0)
        ref.check_attention(out, lse, want, P_STEP, f"step {step}")
