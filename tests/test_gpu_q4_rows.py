"""Rows into the 4-bit cache and back, against the definition: the pool's bytes
are equal but for the sign of a zero, and so is what they stand for."""
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


def rows_like(rng, n, h, amp):
    x = rng.standard_normal((n, h, 128)) * amp * np.exp(rng.standard_normal((n, h, 1)))
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def same_codes(got, want, byte):
    """Equal codes; where a magnitude is 0 its sign says nothing."""
    g, w = ((x[..., None] >> ref.SHIFT) & 15 for x in (got, want))
    assert np.array_equal(g & 7, w & 7)
    live = (g & 7) > 0
    assert np.array_equal(g[live], w[live])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n,hkv,gs", [(1, 1, 1.0), (3, 3, 0.5), (33, 8, 0.25), (200, 5, 3.7),
                                      (257, 2, 1e-3)])
def test_append_and_read(page, n, hkv, gs):
    rng = np.random.default_rng(n * page + hkv)
    pages = -(-n // page) + 2
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    drop = rng.random(n) < 0.1
    slots[drop] = -1 - rng.integers(0, 9, int(drop.sum()))
    k, v = rows_like(rng, n, hkv, gs), rows_like(rng, n, hkv, 0.05 * gs)
    start = rng.integers(0, 256, (2, pages, hkv, page * 72)).astype(np.uint8)
    pools = torch.from_numpy(start).cuda()
    s_dev = torch.from_numpy(slots).cuda()
    binding.kv_append_q4(k.cuda(), v.cuda(), pools[0], pools[1], s_dev, page, gs, gs)
    k_out, v_out = (torch.full((n, hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda")
                    for _ in range(2))
    binding.kv_read_q4(pools[0], pools[1], s_dev, page, gs, gs, k_out, v_out)
    assert binding.last_error() == binding.OK
    live = slots >= 0
    at, off = slots[live] // page, slots[live] % page
    for x, pool, before, out in ((k, pools[0], start[0], k_out), (v, pools[1], start[1], v_out)):
        words, byte = ref.encode(x.float().numpy()[live], gs)
        gw, gb = ref.parts_of(pool.cpu().numpy(), page)
        bw, bb = (a.copy() for a in ref.parts_of(before, page))
        assert np.array_equal(gb[at, :, off], byte)
        same_codes(gw[at, :, off], words, byte)
        bw[at, :, off], bb[at, :, off] = gw[at, :, off], gb[at, :, off]
        assert np.array_equal(bw, gw) and np.array_equal(bb, gb)  # nothing else was written
        want = torch.from_numpy(ref.decode(words, byte, gs).astype(np.float32)).bfloat16()
        assert torch.equal(out.cpu()[torch.from_numpy(live)], want)
        assert (out.cpu()[torch.from_numpy(~live)] == 9.0).all()


def test_every_code_tie_and_scale():
    """Values on and next to every border between two codes, for every group scale
    of normal size, and groups whose scale rounds to 0 or saturates."""
    grid = ref.LEVELS
    ties = (grid[1:] + grid[:-1]) / 2
    rows = []
    for byte in range(1, 127):
        s = ref.E4M3[byte]
        x = np.concatenate([ties * s, -ties * s, [6 * s, 0.0]])  # 16 values: one group
        for nudge in (0, 1, -1):
            b = torch.tensor(x, dtype=torch.float32).bfloat16()
            bits = b.view(torch.int16)
            b = torch.where(b == 0, b, (bits + nudge).view(torch.bfloat16))
            b[14] = float(6 * s)
            rows.append(b)
    for top in (0.0, 1e-30, 2.0 ** -12, 2000.0, 3000.0, 3e38):
        rows.append(torch.linspace(-top, top, 16).bfloat16())
    while len(rows) % 8:
        rows.append(torch.zeros(16, dtype=torch.bfloat16))
    x = torch.stack(rows).reshape(-1, 1, 128)
    n = x.shape[0]
    pools = torch.zeros((2, -(-n // 16), 1, 16 * 72), dtype=torch.uint8, device="cuda")
    slots = torch.arange(n, device="cuda")
    binding.kv_append_q4(x.cuda(), x.cuda(), pools[0], pools[1], slots, 16)
    words, byte = ref.encode(x.float().numpy(), 1.0)
    gw, gb = ref.parts_of(pools[0].cpu().numpy(), 16)
    gw = gw.transpose(0, 2, 1, 3).reshape(-1, 1, 16)[:n]
    gb = gb.transpose(0, 2, 1, 3).reshape(-1, 1, 8)[:n]
    assert np.array_equal(gb, byte)
    same_codes(gw, words, byte)
    assert torch.equal(pools[0], pools[1])
    # the widest linspace overflows fp32 inside: a NaN among the values is reported
    assert binding.last_error() == (binding.EINVAL if x.isnan().any() else binding.OK)


# What a group of ones is held as: its scale is e4m3(1 / 6) = 0.171875 (11 / 64; the
# neighbours are 10 / 64 and 12 / 64), and 1 / 0.171875 = 5.8 is nearest to 6.
ONE = 6 * 0.171875


def test_infinity_and_nan():
    x = torch.ones((2, 1, 128), dtype=torch.bfloat16)
    x[0, 0, 3] = float("inf")
    x[0, 0, 20] = float("-inf")
    pools = torch.zeros((2, 1, 1, 16 * 72), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, 1], device="cuda")
    binding.kv_append_q4(x.cuda(), x.cuda(), pools[0], pools[1], slots, 16)
    assert binding.last_error() == binding.OK
    k, _ = binding.kv_read_q4(pools[0], pools[1], slots, 16)
    assert float(k[0, 0, 3]) == 6 * 448 and float(k[0, 0, 20]) == -6 * 448
    assert float(k[0, 0, 0]) == 0.0 and (k[1] == ONE).all()
    x[1, 0, 64] = float("nan")
    binding.kv_append_q4(x.cuda(), x.cuda(), pools[0], pools[1], slots, 16)
    assert binding.last_error() == binding.EINVAL
    k, _ = binding.kv_read_q4(pools[0], pools[1], slots, 16)
    assert float(k[1, 0, 64]) == 0 and (k[1, 0, :64] == ONE).all() and (k[1, 0, 65:] == ONE).all()


def test_slices_of_wider_rows():
    rng = np.random.default_rng(3)
    qkv = rows_like(rng, 20, 1, 1.0).reshape(20, 128)
    wide = torch.from_numpy(rng.standard_normal((20, 8 + 2 * 2 * 128)).astype(np.float32))
    wide = wide.bfloat16().cuda()
    k, v = (wide[:, 8 + 256 * i:8 + 256 * (i + 1)].unflatten(1, (2, 128)) for i in (0, 1))
    assert not k.is_contiguous() and qkv.numel()
    a = torch.zeros((2, 2, 2, 16 * 72), dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    slots = torch.arange(20, device="cuda")
    binding.kv_append_q4(k, v, a[0], a[1], slots, 16)
    binding.kv_append_q4(k.contiguous(), v.contiguous(), b[0], b[1], slots, 16)
    assert torch.equal(a, b)
    out = torch.zeros_like(wide)
    ko, vo = (out[:, 8 + 256 * i:8 + 256 * (i + 1)].unflatten(1, (2, 128)) for i in (0, 1))
    binding.kv_read_q4(a[0], a[1], slots, 16, k_out=ko, v_out=vo)
    kr, vr = binding.kv_read_q4(a[0], a[1], slots, 16)
    assert torch.equal(ko, kr) and torch.equal(vo, vr) and (out[:, :8] == 0).all()


def test_slots_outside_the_pool():
    x = torch.ones((3, 1, 128), dtype=torch.bfloat16, device="cuda")
    pools = torch.zeros((2, 2, 1, 16 * 72), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([32, 5, 1 << 60], device="cuda")
    binding.kv_append_q4(x, x, pools[0], pools[1], slots, 16)
    assert binding.last_error() == binding.EINVAL
    k = torch.full((3, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    binding.kv_read_q4(pools[0], pools[1], slots, 16, k_out=k, v_out=v)
    assert binding.last_error() == binding.EINVAL
    assert (k[0] == 7).all() and (k[1] == ONE).all() and (k[2] == 7).all()


def test_pool_past_32_bit_offsets():
    """Rows whose bytes lie past 4 GB into the pool."""
    page, hkv = 128, 8
    pages = (5 << 30) // (hkv * page * 72)
    pool = torch.zeros((pages, hkv, page * 72), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(4)
    x = rows_like(rng, 6, hkv, 1.0).cuda()
    last = pages * page
    slots = torch.tensor([last - 1, last - 128, last // 2, 0, last - 300, 77], device="cuda")
    binding.kv_append_q4(x, x, pool, pool, slots, page)
    k, v = binding.kv_read_q4(pool, pool, slots, page)
    words, byte = ref.encode(x.cpu().float().numpy(), 1.0)
    want = torch.from_numpy(ref.decode(words, byte, 1.0).astype(np.float32)).bfloat16()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    assert binding.last_error() == binding.OK


def test_copy_pages():
    rng = np.random.default_rng(5)
    for page in (16, 128):
        pools = torch.from_numpy(rng.integers(0, 256, (2, 6, 3, page * 72)).astype(np.uint8)).cuda()
        want = pools.clone()
        want[:, 4], want[:, 5] = pools[:, 1], pools[:, 0]
        binding.copy_pages_q4(pools[0], pools[1],
                              torch.tensor([[1, 4], [0, 5]], dtype=torch.int32).cuda(), page)
        assert torch.equal(pools, want)
    assert binding.last_error() == binding.OK


def test_captured_and_replayed():
    rng = np.random.default_rng(6)
    x = rows_like(rng, 8, 2, 1.0).cuda()
    pools = torch.zeros((2, 2, 2, 16 * 72), dtype=torch.uint8, device="cuda")
    slots = torch.arange(8, device="cuda")
    binding.kv_append_q4(x, x, pools[0], pools[1], slots, 16)
    graph = torch.cuda.CUDAGraph()
    k, v = (torch.empty((8, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with torch.cuda.graph(graph):
        binding.kv_append_q4(x, x, pools[0], pools[1], slots, 16)
        binding.kv_read_q4(pools[0], pools[1], slots, 16, k_out=k, v_out=v)
    x.copy_(rows_like(rng, 8, 2, 2.0))
    slots.copy_(torch.arange(20, 28))
    graph.replay()
    words, byte = ref.encode(x.cpu().float().numpy(), 1.0)
    want = torch.from_numpy(ref.decode(words, byte, 1.0).astype(np.float32)).bfloat16()
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
