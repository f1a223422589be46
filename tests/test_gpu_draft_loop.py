"""Drafting steps as a user runs them: pages, rows, attention, accepted path, kept rows,
step after step, against a cache kept on the host."""
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


def to_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16()


@pytest.mark.parametrize("kind", ["bf16", "q4", "q8"])
def test_drafting_steps(kind):
    """Six steps: each branch's logical cache is kept on the host, row by row."""
    rng = np.random.default_rng(5)
    P, page, hq, hkv, B, steps = 40, 16, 8, 2, 4, 6
    n_pre, t_max, gs = -(-P // page), 12, 1.0 if kind == "bf16" else 0.5
    pages = n_pre + B * 14
    ids = rng.permutation(pages).astype(np.int32)
    if kind == "bf16":
        pools = [torch.zeros((pages, hkv, page, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    else:
        pools = [(binding.q4_pool if kind == "q4" else binding.q8_pool)(pages, hkv, page) for _ in range(2)]

    def held(x):  # what the cache holds for rows x
        if kind == "bf16":
            return x.double().numpy()
        if kind == "q8":
            return tree_ref.decode8(tree_ref.encode8(x.float().numpy(), gs), gs)
        return ref.decode(*ref.encode(x.float().numpy(), gs), gs)

    def append(k, v, slots, T=None):
        if kind == "bf16" and T is not None:
            binding.kv_append(k.cuda(), v.cuda(), *pools, table, P, S, T, page)
        elif kind == "bf16":
            for pool, x in zip(pools, (k, v)):
                pool[slots // page, :, slots % page] = x.cuda()
        else:
            put = binding.kv_append_q4 if kind == "q4" else binding.kv_append_q8
            extra = (page,) if kind == "q4" else ()
            put(k.cuda(), v.cuda(), *pools, slots, *extra, gs, gs)

    dev32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # the prefix
    k, v = (to_bf16(rng.standard_normal((P, hkv, 128))) for _ in range(2))
    slots = torch.tensor([int(ids[i // page]) * page + i % page for i in range(P)], device="cuda")
    append(k, v, slots)
    cache = [[[*zip(held(k), held(v))][i] for i in range(P)] for _ in range(B)]
    S, suffix = [0] * B, torch.zeros(B, dtype=torch.int32, device="cuda")
    free, used = dev32(ids[n_pre:].tolist()), None
    table, cow, used = binding.fork_device(dev32(ids[:n_pre].tolist()), P, suffix, page, free, 14)
    if kind == "bf16":
        binding.copy_pages(*pools, cow, P % page)
    elif kind == "q4":
        binding.copy_pages_q4(*pools, cow, page)
    else:
        binding.copy_pages_q8(*pools, cow, P % page)
    reserved = suffix.clone()  # private tokens that have a page
    accepted = 0
    for step in range(steps):
        T = rng.integers(1, t_max + 1, size=B).tolist()
        if step == 3:
            T[1] = 0
        trees = [tree_ref.random_tree(rng, t) for t in T]
        R = sum(T)
        parents, add = dev32([p for t in trees for p in t]), dev32(T)
        grow = (suffix + add - reserved).clamp(min=0)
        _, used = binding.extend_device(table, P, reserved, grow, page, free, 0, used)
        reserved += grow
        masks, positions, slots = binding.tree_rows(parents, table, P, suffix, add, page, t_max)
        k, v = (to_bf16(rng.standard_normal((R, hkv, 128))) for _ in range(2))
        q = to_bf16(rng.standard_normal((R, hq, 128)) * 1.5)
        append(k, v, slots, T)
        out, lse = binding.attn_tree(q.cuda(), *pools, table, P, [s + t for s, t in zip(S, T)], T, hq, hkv,
                                     page, 128 ** -0.5, masks, positions, 0, 0, gs, gs)
        draft = rng.integers(0, 4, size=R)
        target, first = rng.integers(0, 4, size=R), rng.integers(0, 4, size=B)
        tok = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
        path, counts, after = binding.tree_accept(parents, tok(draft), tok(target), tok(first), add)
        binding.kv_keep(*pools, table, P, suffix, add, path, counts, page)
        suffix += counts
        assert binding.last_error() == binding.OK
        # the host's own step
        p64, c64, n64 = tree_ref.accept(trees, draft, target, first, R)
        assert np.array_equal(path.cpu().numpy(), p64) and np.array_equal(counts.cpu().numpy(), c64)
        assert np.array_equal(after.cpu().numpy(), n64)
        kh, vh, r = held(k), held(v), 0
        prob = tree_ref.Problem.__new__(tree_ref.Problem)
        prob.kind, prob.q, prob.hq, prob.hkv, prob.page = kind, q, hq, hkv, 1
        prob.scale, prob.see, rows, prob.table = 128 ** -0.5, [], [], {}
        for b in range(B):
            ctx = cache[b] + [(kh[r + t], vh[r + t]) for t in range(T[b])]
            prob.table[b] = np.arange(len(rows), len(rows) + len(ctx))
            rows += ctx
            for t in range(T[b]):
                m = np.zeros(len(ctx), bool)
                m[:len(cache[b])] = True
                m[[len(cache[b]) + u for u in tree_ref.lineage(trees[b], t)[0]]] = True
                prob.see.append((b, m))
            r += T[b]
        prob.k64 = np.array([x[0] for x in rows])[:, :, None]
        prob.v64 = np.array([x[1] for x in rows])[:, :, None]
        prob.check(out, lse, f"step {step}")
        r = 0
        for b in range(B):
            cache[b] += [(kh[r + u], vh[r + u]) for u in p64[r:r + c64[b]]]
            S[b] += int(c64[b])
            r += T[b]
        accepted += int(c64.sum())
        assert suffix.tolist() == S
    assert accepted > B
    assert int(used) <= free.numel() and sum(reserved.tolist()) >= sum(S)


def test_two_threads_on_two_streams():
    """Both run whole steps at once; each gets what it got alone."""
    import threading

    def inputs(seed):
        rng = np.random.default_rng(seed)
        T = [12, 5, 30]
        trees = [tree_ref.random_tree(rng, t) for t in T]
        prob = tree_ref.Problem([40, 61, 7], T, 300, 16, 2, 16, kind="q8", trees=trees, seed=seed)
        prob.args()
        flat = torch.tensor([p for t in trees for p in t], dtype=torch.int32, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        tok = [torch.from_numpy(rng.integers(0, 3, size=47)).cuda() for _ in range(2)]
        return prob, flat, i32([40, 61, 7]), i32(T), tok, torch.from_numpy(rng.integers(0, 3, size=3)).cuda()

    def step(x, stream):
        prob, flat, S, T, (draft, target), first = x
        m, p, s = binding.tree_rows(flat, prob.dev[3], prob.P, S, T, 16, 30, stream=stream)
        out, lse = binding.attn_tree(*prob.dev[:4], prob.P, prob.S, prob.T, 16, 2, 16, prob.scale, m, p,
                                     stream=stream)
        return (m, p, s, out, lse) + tuple(binding.tree_accept(flat, draft, target, first, T,
                                                               stream=stream))
    work = [inputs(1), inputs(2)]
    alone = [step(x, None) for x in work]
    torch.cuda.synchronize()
    streams, got, errors = [torch.cuda.Stream() for _ in work], [None, None], []

    def run(i):
        try:
            for _ in range(40):
                got[i] = step(work[i], streams[i])
            streams[i].synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert binding.last_error() == binding.OK
