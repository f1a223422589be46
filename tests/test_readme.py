"""The drafting loop that users are shown, run against a stand-in of the binding that records its
calls (CPU only): every call fits its signature, and masks are made for what attention is given."""
import inspect
import os
import re

import pytest
import torch

from shared_prefix_fan_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Recorder:
    def __init__(self, results):
        self.calls, self.results = [], results

    def __getattr__(self, name):
        signature = inspect.signature(getattr(binding, name))

        def call(*args, **kw):
            bound = signature.bind(*args, **kw)
            bound.apply_defaults()
            self.calls.append((name, bound.arguments))
            return self.results.get(name)
        return call


@pytest.fixture
def drafting():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    block, = (b for b in blocks if "tree_rows" in b)
    one = torch.ones(1, dtype=torch.int32)
    b = Recorder({"extend_device": ("slots", "used"), "tree_rows": ("masks", "positions", "slots"),
                  "attn_tree": ("out", "lse"), "tree_accept": ("path", one, "next")})
    names = re.findall(r"[A-Za-z_]\w*", block)
    scope = dict.fromkeys(names, "given")
    scope.update(binding=b, suffix_dev=one.clone(), nodes_dev=one * 3, reserved=one.clone(),
                 suffix_lens=[1], nodes=[3], sum=sum, zip=zip)
    exec(block, scope)  # noqa: S102
    return b.calls, scope


def test_masks_are_made_for_the_layers_window(drafting):
    calls, scope = drafting
    by_name = dict(calls)
    rows, attn = by_name["tree_rows"], by_name["attn_tree"]
    assert attn["window"] > 0
    assert (rows["window"], rows["sinks"]) == (attn["window"], attn["sinks"])
    assert attn["masks"] == "masks" and attn["positions"] == "positions"
    assert attn["suffix_lens"] == [4] and scope["suffix_lens"] == [2]


def test_order_of_a_step(drafting):
    assert [name for name, _ in drafting[0]] == ["extend_device", "tree_rows", "kv_append_q8", "attn_tree",
                                                 "tree_accept", "kv_keep"]
