"""Codes of rows where pool scales are so small that a quotient's remainder would be less than
the smallest fp32 number: bit by bit against IEEE quotients. Scales whose last bits are ones
give quotients next to the midpoint of two fp32 numbers beside a tie of two codes."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from . import tree_ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

# (2^24 - g) 2^(e - 24): one step and more below a power of two, from 1e-30 to 1e30
SCALES = [float((2 ** 24 - g) * 2.0 ** (e - 24)) for g, e in
          [(1, -99), (9, -99), (2, -98), (1, -96), (5, -95), (3, -94), (2, -93), (1, -92), (1, -91), (1, -60),
           (3, -59), (1, -40), (1, 0), (5, 1), (1, 60), (1, 99)]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def bf16_values():
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return torch.where(torch.isfinite(x), x, torch.zeros_like(x))


@pytest.mark.parametrize("gs", SCALES)
def test_8_bit_codes(gs):
    x = bf16_values().view(512, 1, 128)
    k_pool, v_pool = binding.q8_pool(32, 1, 16), binding.q8_pool(32, 1, 16)
    binding.kv_append_q8(x.cuda(), x.flip(0).contiguous().cuda(), k_pool, v_pool, torch.arange(512, device="cuda"),
                         gs, gs)
    assert binding.last_error() == binding.OK
    want = tree_ref.encode8(x.float().numpy(), gs).reshape(512, 128)
    for pool, w in ((k_pool, want), (v_pool, want[::-1])):
        got = pool.view(torch.uint8).cpu().numpy().reshape(512, 128)
        bad = np.argwhere(got != w)
        assert len(bad) == 0, (len(bad), got[tuple(bad[0])], w[tuple(bad[0])])


@pytest.mark.parametrize("gs", SCALES)
def test_4_bit_codes(gs):
    """Groups of 16 around the ties of their scale: its own quotient, and the codes'."""
    rng = np.random.default_rng(7)
    e = np.floor(np.log2(gs))
    n = 4096
    # magnitudes of few bits over 2^-5 .. 2^12 pool scales, the group's own size in front
    top = np.ldexp(rng.integers(1, 65, size=(n, 8, 1)) / 64.0, rng.integers(-4, 13, size=(n, 8, 1)))
    x = top * np.ldexp(rng.choice([1, 3, 5, 7, 12, 20, 28, 2], size=(n, 8, 16)) / 32.0, 0)
    x = np.ldexp(np.concatenate([top, x[..., 1:]], -1) * rng.choice([-1, 1], size=(n, 8, 16)), int(e) + 1)
    x = torch.from_numpy(x.reshape(n, 1, 128).astype(np.float32)).bfloat16()
    pools = [binding.q4_pool(n // 16, 1, 16) for _ in range(2)]
    binding.kv_append_q4(x.cuda(), x.flip(0).contiguous().cuda(), *pools, torch.arange(n, device="cuda"), 16, gs, gs)
    assert binding.last_error() == binding.OK
    words, scales = ref.encode(x.float().numpy().reshape(n, 128), gs)
    for pool, flip in zip(pools, (False, True)):
        got = pool.cpu().numpy().reshape(n // 16, 16 * 72)
        gw = got[:, :16 * 64].reshape(n, 64).copy().view("<u4")
        gb = got[:, 16 * 64:].reshape(n, 8)
        if flip:
            gw, gb = gw[::-1], gb[::-1]
        assert np.array_equal(gb, scales), np.argwhere(gb != scales)[:4].tolist()
        assert np.array_equal(gw, words), (len(np.argwhere(gw != words)), np.argwhere(gw != words)[:4].tolist())
