"""Drafting steps in a layer with a window and first keys, from a context shorter than those
on: every row sees what decoding its path token by token would see, step after step."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from . import tree_ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("kind", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("P,window,sinks", [(2, 3, 12), (7, 2, 7), (0, 5, 30)])
def test_windowed_drafting_steps(kind, P, window, sinks):
    rng = np.random.default_rng(P + window)
    page, hq, hkv, B, t_max, gs = 16, 8, 2, 3, 14, 1.0 if kind == "bf16" else 0.5
    pages = B * 8
    dev32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    ids = rng.permutation(pages).reshape(B, 8)
    table = dev32(ids)  # (prefix tokens in pages of the branch's own, too)
    if kind == "bf16":
        pools = [torch.zeros((pages, hkv, page, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    else:
        pools = [(binding.q4_pool if kind == "q4" else binding.q8_pool)(pages, hkv, page) for _ in range(2)]

    def held(x):
        if kind == "bf16":
            return x.double().numpy()
        x = x.float().numpy()
        return tree_ref.decode8(tree_ref.encode8(x, gs), gs) if kind == "q8" else \
            ref.decode(*ref.encode(x, gs), gs)

    def append(k, v, slots):
        if kind == "bf16":
            for pool, x in zip(pools, (k, v)):
                pool[slots // page, :, slots % page] = x.cuda()
        elif kind == "q4":
            binding.kv_append_q4(k.cuda(), v.cuda(), *pools, slots, page, gs, gs)
        else:
            binding.kv_append_q8(k.cuda(), v.cuda(), *pools, slots, gs, gs)
    rows = lambda n: [torch.from_numpy(rng.standard_normal((n, hkv, 128)).astype(np.float32)).bfloat16()  # noqa: E731
                      for _ in range(2)]
    cache = [[] for _ in range(B)]
    k, v = rows(P)
    for b in range(B):  # the prefix, the same in every branch
        if P:
            append(k, v, torch.tensor([int(ids[b, i // page]) * page + i % page for i in range(P)], device="cuda"))
        cache[b] = list(zip(held(k), held(v)))
    suffix, S, deep = dev32([0] * B), [0] * B, 0
    for step in range(4):
        T = rng.integers(1, t_max + 1, size=B).tolist()
        trees = [tree_ref.random_tree(rng, t, "chain" if (step + b) % 2 else "random") for b, t in enumerate(T)]
        parents, add, R = dev32([p for t in trees for p in t]), dev32(T), sum(T)
        masks, positions, slots = binding.tree_rows(parents, table, P, suffix, add, page, t_max, window,
                                                    sinks=sinks)
        k, v = rows(R)
        append(k, v, slots)
        q = torch.from_numpy(rng.standard_normal((R, hq, 128)).astype(np.float32) * 1.5).bfloat16()
        # (the branches' own copies of a prefix shorter than a page: none of it is shared)
        out, lse = binding.attn_tree(q.cuda(), *pools, table, P, [s + t for s, t in zip(S, T)], T, hq, hkv, page,
                                     128 ** -0.5, masks, positions, window, sinks, gs, gs)
        draft, target = rng.integers(0, 2, size=R), rng.integers(0, 2, size=R)
        first = rng.integers(0, 2, size=B)
        tok = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
        path, counts, _ = binding.tree_accept(parents, tok(draft), tok(target), tok(first), add)
        binding.kv_keep(*pools, table, P, suffix, add, path, counts, page)
        suffix += counts
        assert binding.last_error() == binding.OK
        p64, c64, _ = tree_ref.accept(trees, draft, target, first, R)
        assert np.array_equal(path.cpu().numpy(), p64) and np.array_equal(counts.cpu().numpy(), c64)
        kh, vh, r = held(k), held(v), 0
        prob = tree_ref.Problem.__new__(tree_ref.Problem)
        prob.kind, prob.q, prob.hq, prob.hkv, prob.page = kind, q, hq, hkv, 1
        prob.scale, prob.see, every, prob.table = 128 ** -0.5, [], [], {}
        for b in range(B):
            n = len(cache[b])
            context = cache[b] + [(kh[r + t], vh[r + t]) for t in range(T[b])]
            prob.table[b] = np.arange(len(every), len(every) + len(context))
            every += context
            for t in range(T[b]):
                line, depth = tree_ref.lineage(trees[b], t)
                # as decoded: the context's keys, then the path's, at positions 0, 1, ...
                keys = list(range(n)) + [n + u for u in reversed(line)]
                m = np.zeros(len(context), bool)
                for position, key in enumerate(keys):
                    m[key] = position > n + depth - window or position < sinks
                prob.see.append((b, m))
                deep += depth >= window and n < sinks
            r += T[b]
        prob.k64 = np.array([x[0] for x in every])[:, :, None]
        prob.v64 = np.array([x[1] for x in every])[:, :, None]
        prob.check(out, lse, f"step {step}")
        r = 0
        for b in range(B):
            cache[b] += [(kh[r + u], vh[r + u]) for u in p64[r:r + c64[b]]]
            S[b] += int(c64[b])
            r += T[b]
    assert sum(S) > 0 and (deep > 0 or sinks <= P)
