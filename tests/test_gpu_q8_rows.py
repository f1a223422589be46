"""Rows into 8-bit pools and back, byte by byte against the plain 64-bit form."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import tree_ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def pool_bytes(pool):
    return pool.view(torch.uint8).cpu().numpy()


def same(got, want):
    bad = np.argwhere(got != want)
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


def every_bf16():
    return torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("gs", [1.0, 0.25, 0.07, 3.0, 1e-30, 1e30, 1.1e-28])
def test_every_bf16_value(gs):
    """All 65536 bit patterns, as K in their order and as V in reverse."""
    x = every_bf16().view(512, 1, 128)
    nan = torch.isnan(x)
    k_pool, v_pool = binding.q8_pool(32, 1, 16), binding.q8_pool(32, 1, 16)
    slots = torch.arange(512, device="cuda")
    binding.kv_append_q8(x.cuda(), x.flip(0).contiguous().cuda(), k_pool, v_pool, slots, gs, gs)
    assert binding.last_error() == binding.EINVAL  # the NaN patterns
    want = tree_ref.encode8(x.float().numpy(), gs)
    same(pool_bytes(k_pool).reshape(512, 1, 128), want)
    same(pool_bytes(v_pool).reshape(512, 1, 128), want[::-1])
    k, v = binding.kv_read_q8(k_pool, v_pool, slots, gs, gs)
    assert binding.last_error() == binding.OK
    # a value's product with gs in fp32, then in bf16: from the exact one at most half a step
    # of each, but for results below the normal range, whose steps are absolute
    exact = tree_ref.decode8(want, gs)
    for got, ref in ((k, exact), (v, exact[::-1])):
        d = np.abs(got.double().cpu().numpy() - ref)
        assert (d <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133).all()
    assert not torch.isnan(k).any() and nan.any()


@pytest.mark.parametrize("page,hkv,n", [(16, 1, 1), (32, 3, 5), (64, 8, 77), (128, 2, 300)])
def test_rows_land_in_their_slots(page, hkv, n):
    """Scattered slots, padded rows and strided input; all other bytes stay."""
    rng = np.random.default_rng(page + n)
    pages = -(-n // page) + 3
    wide = torch.from_numpy(rng.standard_normal((n, 2 * hkv + 1, 128)).astype(np.float32)).bfloat16().cuda()
    k_new, v_new = wide[:, :hkv], wide[:, hkv:2 * hkv]
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64))
    if n > 3:
        slots[2] = -1
    k_pool, v_pool = (torch.full((pages, hkv, page, 128), 0x55, dtype=torch.uint8, device="cuda"
                                 ).view(torch.float8_e4m3fn) for _ in range(2))
    binding.kv_append_q8(k_new, v_new, k_pool, v_pool, slots.cuda(), 0.5, 0.3)
    assert binding.last_error() == binding.OK
    for pool, x, gs in ((k_pool, k_new, 0.5), (v_pool, v_new, 0.3)):
        want = np.full((pages, hkv, page, 128), 0x55, np.uint8)
        code = tree_ref.encode8(x.float().cpu().numpy(), gs)
        for r, s in enumerate(slots.tolist()):
            if s >= 0:
                want[s // page, :, s % page] = code[r]
        assert np.array_equal(pool_bytes(pool), want)
    out = torch.full((n, 2 * hkv + 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.kv_read_q8(k_pool, v_pool, slots.cuda(), 0.5, 0.3, out[:, :hkv], out[:, hkv:2 * hkv])
    got = out.cpu()
    assert (got[:, -1] == 7.0).all()
    for r, s in enumerate(slots.tolist()):
        if s < 0:
            assert (got[r] == 7.0).all()
            continue
        for lo, x, gs in ((0, k_new, 0.5), (hkv, v_new, 0.3)):
            ref = tree_ref.decode8(tree_ref.encode8(x[r].float().cpu().numpy(), gs), gs)
            d = np.abs(got[r, lo:lo + hkv].double().numpy() - ref)
            assert (d <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -23)).all()


def test_rows_off_a_32_byte_boundary():
    """Rows that start on 16 bytes only take the other loads and stores."""
    flat = torch.randn(4 * 136 + 8, device="cuda").bfloat16()
    x = flat[8:8 + 4 * 136].view(4, 136)[:, :128].unsqueeze(1)  # rows 136 apart
    k_pool, v_pool = binding.q8_pool(1, 1, 16), binding.q8_pool(1, 1, 16)
    slots = torch.tensor([3, 1, 0, 15], device="cuda")
    binding.kv_append_q8(x, x, k_pool, v_pool, slots)
    want = tree_ref.encode8(x[:, 0].float().cpu().numpy(), 1.0)
    assert np.array_equal(pool_bytes(k_pool)[0, 0, slots.cpu()], want)
    out = torch.zeros(4 * 136 + 8, device="cuda").bfloat16()
    o = out[8:8 + 4 * 136].view(4, 136)[:, :128].unsqueeze(1)
    binding.kv_read_q8(k_pool, v_pool, slots, k_out=o, v_out=torch.empty_like(o.contiguous()))
    assert np.array_equal(o[:, 0].double().cpu().numpy(), tree_ref.decode8(want, 1.0))
    assert (out[:8] == 0).all() and (out[8:].view(4, 136)[:, 128:] == 0).all()


def test_slots_outside_the_pool_are_skipped_and_reported():
    x = torch.randn((3, 1, 128), device="cuda").bfloat16()
    k_pool, v_pool = binding.q8_pool(2, 1, 16), binding.q8_pool(2, 1, 16)
    slots = torch.tensor([32, 1, 2 ** 40], device="cuda")
    binding.kv_append_q8(x, x, k_pool, v_pool, slots)
    assert binding.last_error() == binding.EINVAL
    got = pool_bytes(k_pool)
    assert np.array_equal(got[0, 0, 1], tree_ref.encode8(x[1, 0].float().cpu().numpy(), 1.0))
    got[0, 0, 1] = 0
    assert not got.any()
    k = torch.full((3, 1, 128), 3.0, device="cuda").bfloat16()
    binding.kv_read_q8(k_pool, v_pool, slots, k_out=k, v_out=k.clone())
    assert binding.last_error() == binding.EINVAL
    assert (k[0] == 3.0).all() and (k[2] == 3.0).all()


def test_infinities_are_held_as_the_largest_value():
    x = torch.full((1, 1, 128), float("inf"), device="cuda").bfloat16()
    x[..., ::2] *= -1
    k_pool, v_pool = binding.q8_pool(1, 1, 16), binding.q8_pool(1, 1, 16)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    binding.kv_append_q8(x, x, k_pool, v_pool, slots, 0.5)
    assert binding.last_error() == binding.OK
    k, _ = binding.kv_read_q8(k_pool, v_pool, slots, 0.5)
    assert (k[..., ::2] == -224).all() and (k[..., 1::2] == 224).all()


def test_pools_past_32_bit_offsets():
    """Rows behind 4 GiB of a pool."""
    pages, hkv, page = 34000, 8, 128
    k_pool, v_pool = binding.q8_pool(pages, hkv, page), binding.q8_pool(pages, hkv, page)
    assert k_pool.numel() > 2 ** 32
    x = torch.randn((3, hkv, 128), device="cuda").bfloat16()
    slots = torch.tensor([pages * page - 1, 17, pages * page - 200], device="cuda")
    binding.kv_append_q8(x, x.flip(0), k_pool, v_pool, slots)
    k, v = binding.kv_read_q8(k_pool, v_pool, slots)
    assert binding.last_error() == binding.OK
    want = torch.from_numpy(tree_ref.decode8(tree_ref.encode8(x.float().cpu().numpy(), 1.0), 1.0))
    assert torch.equal(k.double().cpu(), want) and torch.equal(v.double().cpu(), want.flip(0))
    assert torch.equal(k_pool.view(torch.uint8)[slots // page, :, slots % page].cpu(),
                       torch.from_numpy(tree_ref.encode8(x.float().cpu().numpy(), 1.0)))


def test_captured_rows_replay_on_new_contents():
    x = torch.randn((4, 2, 128), device="cuda").bfloat16()
    k_pool, v_pool = binding.q8_pool(2, 2, 16), binding.q8_pool(2, 2, 16)
    slots = torch.tensor([3, 30, -1, 8], device="cuda")
    out = torch.zeros((4, 2, 128), device="cuda").bfloat16()
    binding.kv_append_q8(x, x, k_pool, v_pool, slots)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.kv_append_q8(x, x, k_pool, v_pool, slots)
        binding.kv_read_q8(k_pool, v_pool, slots, k_out=out, v_out=out.clone())
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        slots.copy_(torch.tensor([seed, 20 + seed, -1, 8]))
        g.replay()
        want = tree_ref.decode8(tree_ref.encode8(x.float().cpu().numpy(), 1.0), 1.0)
        got = out.double().cpu().numpy()
        assert np.array_equal(got[[0, 1, 3]], want[[0, 1, 3]]) and not got[2].any()


def test_copied_pages():
    k_pool, v_pool = (torch.randint(0, 256, (5, 3, 32, 128), dtype=torch.uint8, device="cuda"
                                    ).view(torch.float8_e4m3fn) for _ in range(2))
    before = [pool_bytes(x).copy() for x in (k_pool, v_pool)]
    pairs = torch.tensor([[1, 4], [2, 0], [-1, 3]], dtype=torch.int32, device="cuda")
    binding.copy_pages_q8(k_pool, v_pool, pairs, 7)
    assert binding.last_error() == binding.EINVAL  # the pair without a page
    for pool, old in ((k_pool, before[0]), (v_pool, before[1])):
        old[4, :, :7], old[0, :, :7] = old[1, :, :7], old[2, :, :7]
        assert np.array_equal(pool_bytes(pool), old)
