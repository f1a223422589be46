"""4-bit attention at the ends of the accepted softmax scales, against the plain
64-bit form and its derived bounds."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import ensure_lib
from .q4_problem import TwoScales

pytestmark = pytest.mark.gpu
P_STEP = 2.0 ** -11  # half a step of f16, the type P is rounded to


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


SHAPES = [([130, 37], [1, 1], 75), ([130, 37], [3, 37], 75), ([61], [1], 0)]


@pytest.mark.parametrize("S,T,P", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("scale,ks", [(1.2e-7, 1e-30), (128 ** -0.5, 1e-19), (1e-20, 1.0),
                                      (128 ** -0.5, 1.0)])
def test_zero_and_tiny_queries(S, T, P, window, sinks, scale, ks):
    """Rows of zeros (a padded batch's) and rows whose elements are tiny: every score is
    close to 0, whatever power of two a row was scaled with, and a hidden key stays
    hidden."""
    prob = TwoScales(S, T, P, 8, 2, 16, ks, 1.0, scale, window=window, sinks=sinks, seed=3)
    R = prob.q.shape[0]
    amp = torch.tensor([0.0, 2.0 ** -14, 2.0 ** -90, 2.0 ** -126, 1.0]).bfloat16()
    rows = amp[(torch.arange(R)[:, None] * 3 + torch.arange(8)[None]) % 5]
    prob.q = prob.q * rows[:, :, None]
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    ref.check_attention(out, lse, prob.reference(), P_STEP)


@pytest.mark.parametrize("S,T,P", SHAPES)
@pytest.mark.parametrize("scale,ks,amp", [(1e-44, 1e30, 1e13), (2.9e38, 1e-30, 1e-10)])
def test_scale_product_in_range_and_a_factor_at_its_end(S, T, P, scale, ks, amp):
    """scale * k_scale is what has to be in range: a subnormal scale loses no bits and a
    large one does not overflow on the way to the product."""
    prob = TwoScales(S, T, P, 8, 2, 16, ks, 1.0, scale, seed=5)
    prob.q = (prob.q.float() * amp).bfloat16()
    assert np.isfinite(prob.q.float().numpy()).all()
    out, lse = prob.run()
    assert binding.last_error() == binding.OK
    ref.check_attention(out, lse, prob.reference(), P_STEP)


@pytest.mark.parametrize("S,T,P", SHAPES)
@pytest.mark.parametrize("windowed", [False, True])
def test_largest_scale_on_bf16_pools(S, T, P, windowed):
    """Queries of zeros under the largest accepted scale: the mean of the visible V."""
    prob = ref.Problem(S, T, P, 8, 2, 16, window=50 if windowed else 10 ** 6, seed=6)
    prob.q.zero_()
    prob.scale = float(np.float32(2.9e38))
    if windowed:
        out, lse = prob.run()
    else:
        q, k, v = (x.cuda() for x in (prob.q, prob.k_pool, prob.v_pool))
        out, lse = binding.attn(q, k, v, torch.from_numpy(prob.table).cuda(), P, S, T, 8, 2, 16,
                                prob.scale, True)
    assert binding.last_error() == binding.OK
    ref.check_attention(out, lse, prob.reference(), 2.0 ** -8)
