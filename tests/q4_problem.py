"""Problems on 4-bit pools whose K and V scales differ: test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

from . import serving_ref as ref


class TwoScales(ref.Problem):
    """A 4-bit problem with a scale of its own for K and for V, and any softmax scale.
    The pools' bytes are those of scale 1: what they stand for follows the scales."""

    def __init__(self, S, T, P, hq, hkv, page, ks, vs, scale=128 ** -0.5, **kw):
        super().__init__(S, T, P, hq, hkv, page, q4=True, gs=1.0, **kw)
        self.ks, self.vs, self.scale = ks, vs, float(np.float32(scale))
        self.hold()

    def hold(self):
        """Takes the values to compare with from the pools' bytes."""
        self.k64, self.v64 = (ref.decode(*ref.parts_of(pool.numpy(), self.page), gs)
                              for pool, gs in ((self.k_pool, self.ks), (self.v_pool, self.vs)))

    def run(self, out_dtype="f32", stream=None, **kw):
        from shared_prefix_fan_gb300 import binding
        dev = [x.cuda() for x in (self.q, self.k_pool, self.v_pool)]
        return binding.attn_q4(*dev, torch.from_numpy(self.call_table).cuda(), self.P, self.S,
                               self.T, self.hq, self.hkv, self.page, self.scale, self.causal,
                               self.ks, self.vs, self.window, self.sinks, out_dtype=out_dtype,
                               stream=stream, **kw)
