"""Calls right behind one another: their kernels start up while the one before still runs, and
see all that it wrote. Every result is bit for bit that of the same calls with a wait between."""
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


def both(make, step, rounds):
    """What `step` gives in each round, with and without a wait behind every call."""
    got = []
    for wait in (True, False):
        state = make()
        torch.cuda.synchronize()
        sync = torch.cuda.synchronize if wait else lambda: None
        results = [step(state, i, sync) for i in range(rounds)]
        torch.cuda.synchronize()
        got.append(results)
    for i, (a, b) in enumerate(zip(*got)):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), f"round {i}"


@pytest.mark.parametrize("R,hkv", [(1, 1), (8, 8), (700, 4), (6000, 8)])
def test_rows_in_and_out(R, hkv):
    """New rows at the same slots each round, read back at once."""
    g = torch.Generator("cuda").manual_seed(R)
    rows = torch.randn((40, 2, R, hkv, 128), generator=g, device="cuda").bfloat16()
    slots = torch.randperm(64 * (R // 64 + 2), generator=g, device="cuda")[:R].contiguous()
    outs = []

    def make():
        outs.append(torch.empty((40, 2, R, hkv, 128), dtype=torch.bfloat16, device="cuda"))
        return [binding.q8_pool(R // 64 + 2, hkv, 64) for _ in range(2)]

    def step(pools, i, sync):
        binding.kv_append_q8(rows[i, 0], rows[i, 1], *pools, slots)
        sync()
        out = binding.kv_read_q8(*pools, slots, k_out=outs[-1][i, 0], v_out=outs[-1][i, 1])
        sync()
        return out
    both(make, step, 40)


@pytest.mark.parametrize("kind", ["bf16", "q8"])
@pytest.mark.parametrize("B,T,P,page", [(3, 8, 96, 16), (8, 32, 2048, 64), (96, 20, 128, 16)])
def test_steps(kind, B, T, P, page):
    """Drafting steps that write the same masks, slots, rows and results again and again."""
    rng = np.random.default_rng(B)
    hq, hkv, S, R, rounds = 16, 2, 60, B * T, 12
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    parents = i32([np.concatenate([tree_ref.random_tree(rng, T, "random") for _ in range(B)])
                   for _ in range(rounds)])
    draft, target = (torch.tensor(rng.integers(0, 3, (rounds, R)), device="cuda") for _ in range(2))
    first = torch.tensor(rng.integers(0, 3, (rounds, B)), device="cuda")
    g = torch.Generator("cuda").manual_seed(B)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    width = -(-(P + S + T) // page)
    n_pre = P // page
    own = width - n_pre
    table = torch.cat([torch.arange(n_pre, device="cuda").expand(B, -1),
                       n_pre + torch.arange(B * own, device="cuda").view(B, own)], 1).int().contiguous()
    q, k_new, v_new = rand(R, hq, 128), rand(rounds, R, hkv, 128), rand(rounds, R, hkv, 128)
    pool = rand(2, n_pre + B * own, hkv, page, 128)
    lens, suffix = i32([T] * B), i32([S] * B)

    def make():
        k, v = (p.clone() if kind == "bf16" else p.to(torch.float8_e4m3fn) for p in pool)
        return dict(k=k, v=v, masks=torch.zeros((R, 1), dtype=torch.int32, device="cuda"),
                    positions=torch.zeros(R, dtype=torch.int32, device="cuda"),
                    slots=torch.full((R,), -1, dtype=torch.int64, device="cuda"))

    def step(s, i, sync):
        binding.tree_rows(parents[i], table, P, suffix, lens, page, T, 0, s["masks"], s["positions"],
                          s["slots"])
        sync()
        if kind == "q8":
            binding.kv_append_q8(k_new[i], v_new[i], s["k"], s["v"], s["slots"])
        else:
            binding.kv_append(k_new[i], v_new[i], s["k"], s["v"], table, P, [S] * B, [T] * B, page)
        sync()
        out, lse = binding.attn_tree(q, s["k"], s["v"], table, P, [S + T] * B, [T] * B, hq, hkv, page,
                                     0.09, s["masks"], s["positions"])
        sync()
        path, counts, after = binding.tree_accept(parents[i], draft[i], target[i], first[i], lens)
        sync()
        binding.kv_keep(s["k"], s["v"], table, P, suffix, lens, path, counts, page)
        sync()
        kept = (binding.kv_read_q8(s["k"], s["v"], s["slots"]) if kind == "q8"
                else (s["k"].clone(), s["v"].clone()))
        sync()
        return [out, lse, path, counts, after, *kept, s["masks"].clone(), s["slots"].clone()]
    both(make, step, rounds)


def test_captured_chain():
    """The same chain in a graph that is replayed with other contents."""
    rng = np.random.default_rng(5)
    B, T, P, page, hkv, S, R = 8, 32, 64, 16, 4, 30, 256
    width = (P + S + T) // page + 1
    table = torch.arange(B * width, device="cuda").int().view(B, width)
    table[:, :P // page] = table[0, :P // page]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    parents, lens, suffix = i32([0] * R), i32([T] * B), i32([S] * B)
    draft, target, first = (torch.zeros(n, dtype=torch.int64, device="cuda") for n in (R, R, B))
    new = torch.zeros((2, R, hkv, 128), dtype=torch.bfloat16, device="cuda")
    pools = [binding.q8_pool(B * width, hkv, page) for _ in range(2)]

    def chain():
        masks, positions, slots = binding.tree_rows(parents, table, P, suffix, lens, page, T)
        binding.kv_append_q8(new[0], new[1], *pools, slots)
        path, counts, after = binding.tree_accept(parents, draft, target, first, lens)
        binding.kv_keep(*pools, table, P, suffix, lens, path, counts, page)
        return [masks, positions, slots, path, counts, after, *binding.kv_read_q8(*pools, slots)]

    def fill(i):
        parents.copy_(i32(np.concatenate([tree_ref.random_tree(rng, T, "random") for _ in range(B)])))
        for t in (draft, target, first):
            t.copy_(torch.tensor(rng.integers(0, 3, t.numel())))
        new.copy_(torch.randn(new.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
    fill(0)
    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = chain()
    for i in range(20):
        fill(i)
        before = [p.clone() for p in pools]
        graph.replay()
        graph.replay()  # (the rows are written anew, so the second does what the first did)
        torch.cuda.synchronize()
        got = [r.clone() for r in results]
        for p, b in zip(pools, before):
            p.copy_(b)
        want = [r for _ in range(2) for r in chain()][-len(got):]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i
    assert binding.last_error() == binding.OK


def test_behind_another_stream_and_behind_copies():
    """What lies between two calls (an event of another stream, a copy from the host, a kernel of
    another kind) is waited for as ever."""
    R, hkv = 512, 4
    pools = [binding.q8_pool(R // 64, hkv, 64) for _ in range(2)]
    slots = torch.arange(R, device="cuda")
    new = torch.zeros((2, R, hkv, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((30, 2, R, hkv, 128), dtype=torch.bfloat16, device="cuda")
    host = torch.zeros_like(new, device="cpu").pin_memory()
    big = torch.randn((4096, 4096), device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    for i in range(30):
        binding.kv_read_q8(*pools, slots)
        if i % 3 == 0:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                for _ in range(4):
                    big = torch.tanh(big @ big)
                new.fill_(i + 1)
            main.wait_stream(side)
        elif i % 3 == 1:
            torch.cuda.synchronize()
            host.fill_(i + 1)
            big = torch.tanh(big @ big)
            binding.kv_read_q8(*pools, slots)
            new.copy_(host, non_blocking=True)
        else:
            new.fill_(i + 1)
        binding.kv_append_q8(new[0], new[1], *pools, slots)
        binding.kv_read_q8(*pools, slots, k_out=out[i, 0], v_out=out[i, 1])
    torch.cuda.synchronize()
    want = (torch.arange(30, device="cuda") + 1).to(torch.float8_e4m3fn).bfloat16()
    assert torch.equal(out, want.view(30, 1, 1, 1, 1).expand_as(out))
