"""Masks, positions, slots, accepted paths and kept rows of drafted trees on the device,
against the plain forms, exactly."""
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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda").reshape(np.shape(x))


def i64(x):
    return torch.tensor(np.asarray(x), dtype=torch.int64, device="cuda").reshape(np.shape(x))


def flat(trees, pad=0):
    return i32([p for t in trees for p in t] + [-9] * pad)


def draft_problem(seed, B, t_hi, shape="random", P=37, page=16, vocab=9):
    """Trees, table and tokens; a small vocabulary, so that siblings share a token."""
    rng = np.random.default_rng(seed)
    trees = [tree_ref.random_tree(rng, int(t), shape) for t in rng.integers(0, t_hi + 1, size=B)]
    S = rng.integers(0, 60, size=B).tolist()
    ends = [P + s + len(t) for s, t in zip(S, trees)]
    width = max(-(-e // page) for e in ends) + 2
    pages = 5 + sum(-(-e // page) for e in ends)
    table = np.full((B, width), -1, np.int32)
    ids, at = rng.permutation(pages), 0
    for b, e in enumerate(ends):
        n = -(-e // page)
        table[b, :n] = ids[at:at + n]
        at += n
    R = sum(len(t) for t in trees)
    return trees, S, table, pages, rng.integers(0, vocab, size=R), rng.integers(0, vocab, size=R), \
        rng.integers(0, vocab, size=B), rng


SIZES = [(1, 1, "random"), (3, 8, "random"), (8, 64, "chain"), (5, 40, "flat"), (2, 1024, "chain"),
         (2, 1024, "random"), (40, 33, "star"), (700, 6, "random"), (4096, 3, "random")]


@pytest.mark.parametrize("window", [0, 1, 5])
@pytest.mark.parametrize("B,t_hi,shape", SIZES)
def test_tree_rows(B, t_hi, shape, window):
    trees, S, table, *_ = draft_problem(B + t_hi, B, t_hi, shape)
    T, R = [len(t) for t in trees], sum(len(t) for t in trees)
    masks, positions, slots = binding.tree_rows(flat(trees, 3), i32(table), 37, i32(S), i32(T), 16,
                                                t_hi, window)
    assert binding.last_error() == binding.OK
    m, p, s = tree_ref.tree_rows(trees, table, 37, S, 16, R + 3, -(-t_hi // 32), window)
    assert np.array_equal(masks.cpu().numpy().view(np.uint32), m)
    assert np.array_equal(positions.cpu().numpy(), p)
    assert np.array_equal(slots.cpu().numpy(), s)


def test_tree_rows_match_the_slots_of_an_extension():
    trees, S, table, *_ = draft_problem(5, 9, 20)
    T = [len(t) for t in trees]
    _, _, slots = binding.tree_rows(flat(trees), i32(table), 37, i32(S), i32(T), 16, 20)
    grown, want, _ = ref.extend(table, 37, S, T, 16, np.arange(5000, 6000), 0, sum(T))
    same = grown == table
    # every page is held already, so the extension's own take others: compare where kept
    assert np.array_equal(slots.cpu().numpy() % 16, want % 16)
    assert same.any()


@pytest.mark.parametrize("what", ["negative", "long", "rows", "table", "suffix", "deep"])
def test_bad_lengths_give_no_rows(what):
    trees, S, table, *_ = draft_problem(6, 4, 12)
    trees[1] = [-1] * 5
    T, R = [len(t) for t in trees], sum(len(t) for t in trees)
    n, words, width = R, 1, table.shape[1]
    if what == "negative":
        T[1] = -1
    elif what == "long":
        T[1] = 33
    elif what == "rows":
        n = R - 1
    elif what == "table":
        width = 2
    elif what == "suffix":
        S[2] = -3
    else:
        S[2] = 2 ** 31 - 1
    parents = flat(trees)[:n].contiguous()
    masks, positions, slots = binding.tree_rows(parents, i32(table[:, :width].copy()), 37, i32(S),
                                                i32(T), 16, 32 * words)
    assert binding.last_error() == binding.EINVAL
    assert not masks.any() and not positions.any() and (slots == -1).all()


def test_bad_parents_are_reported_and_count_as_none():
    table = np.arange(8, dtype=np.int32)[None]
    masks, positions, _ = binding.tree_rows(i32([-1, 1, 5, -7, 2]), i32(table), 0, i32([10]), i32([5]),
                                            16, 5)
    assert binding.last_error() == binding.EINVAL
    assert masks[:, 0].tolist() == [1, 2, 4, 8, 0b10100] and positions.tolist() == [10, 10, 10, 10, 11]


def test_rows_without_a_page_are_reported():
    table = np.array([[3, -1]], np.int32)
    masks, _, slots = binding.tree_rows(i32([-1, 0, 1]), i32(table), 0, i32([15]), i32([3]), 16, 3)
    assert binding.last_error() == binding.EINVAL
    assert slots.tolist() == [3 * 16 + 15, -1, -1] and masks[:, 0].tolist() == [1, 3, 7]


@pytest.mark.parametrize("B,t_hi,shape", SIZES)
def test_tree_accept(B, t_hi, shape):
    trees, _, _, _, draft, target, first, rng = draft_problem(B * t_hi, B, t_hi, shape, vocab=3)
    if shape == "chain":  # so that long paths come up
        target[:] = np.roll(draft, -1)
        first[:] = [draft[sum(len(t) for t in trees[:b])] if trees[b] else 0 for b in range(B)]
    R, T = sum(len(t) for t in trees), [len(t) for t in trees]
    pad = 2
    path, counts, after = binding.tree_accept(
        flat(trees, pad), i64(np.append(draft, [0] * pad)), i64(np.append(target, [0] * pad)),
        i64(first), i32(T))
    assert binding.last_error() == binding.OK
    p, c, n = tree_ref.accept(trees, draft, target, first, R + pad)
    assert np.array_equal(path.cpu().numpy(), p)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(after.cpu().numpy(), n)
    if shape == "chain":
        assert c.max() == max(T)


@pytest.mark.parametrize("T", [[3, -1], [3, 1025], [4, 4]])
def test_bad_lengths_accept_nothing(T):
    path, counts, after = binding.tree_accept(i32([-1] * 6), i64([1] * 6), i64([1] * 6), i64([1, 1]), i32(T))
    assert binding.last_error() == binding.EINVAL
    assert (path == -1).all() and not counts.any() and (after == -1).all()


def test_accept_without_rows():
    path, counts, after = binding.tree_accept(i32([]), i64([]), i64([]), i64([4, 5]), i32([0, 0]))
    assert binding.last_error() == binding.OK
    assert path.numel() == 0 and counts.tolist() == [0, 0] and after.tolist() == [4, 5]


def pools_of(kind, pages, hkv, page, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "bf16":
        return [torch.randn((pages, hkv, page, 128), generator=g).bfloat16().cuda() for _ in range(2)]
    shape = (pages, hkv, page * 72) if kind == "q4" else (pages, hkv, page, 128)
    x = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    return x if kind == "q4" else [y.view(torch.float8_e4m3fn) for y in x]


def raw(pool):
    return pool.view(torch.uint8).cpu().numpy().copy() if pool.dtype != torch.uint8 else pool.cpu().numpy().copy()


def move(pool, kind, page, src, dst):
    """One row, all heads, of the pool's bytes."""
    (ps, ss), (pd, sd) = src, dst
    if kind == "q4":
        pool[pd, :, sd * 64:sd * 64 + 64] = pool[ps, :, ss * 64:ss * 64 + 64]
        a, b = page * 64 + ss * 8, page * 64 + sd * 8
        pool[pd, :, b:b + 8] = pool[ps, :, a:a + 8]
    else:
        pool[pd, :, sd] = pool[ps, :, ss]


@pytest.mark.parametrize("kind", ["bf16", "q4", "q8"])
@pytest.mark.parametrize("B,t_hi,hkv,page", [(1, 1, 1, 16), (6, 30, 3, 16), (3, 300, 5, 32), (1, 1024, 8, 128),
                                             (900, 8, 2, 64)])
def test_kv_keep(kind, B, t_hi, hkv, page):
    trees, S, table, pages, *_, rng = draft_problem(B + page, B, t_hi, page=page)
    path, counts = [], []
    for t in trees:  # any ascending path, dense ones and the whole branch among them
        n = len(t)
        keep = np.nonzero(rng.random(n) < rng.choice([0.1, 0.5, 0.95, 1.0]))[0].tolist()
        counts.append(len(keep))
        path += keep + [-1] * (n - len(keep))
    pools = pools_of(kind, pages, hkv, page)
    want = [raw(x) for x in pools]
    T = [len(t) for t in trees]
    r = 0
    for b, t in enumerate(trees):
        place = lambda i: (table[b][(37 + S[b] + i) // page], (37 + S[b] + i) % page)  # noqa: E731
        for x in want:
            for i in range(counts[b]):
                move(x, kind, page, place(path[r + i]), place(i))
        r += len(t)
    binding.kv_keep(*pools, i32(table), 37, i32(S), i32(T), i32(path + [-1, -1]), i32(counts), page)
    assert binding.last_error() == binding.OK
    for x, w in zip(pools, want):
        assert np.array_equal(raw(x), w)


@pytest.mark.parametrize("path,count", [([1, 0, 2], 3), ([0, 0, 1], 3), ([0, 1, 3], 3), ([-1, 1, 2], 2),
                                        ([0, 1, 2], 4), ([0, 1, 2], -1)])
def test_paths_that_do_not_ascend_move_nothing(path, count):
    pools = pools_of("q8", 6, 2, 16)
    before = [raw(x) for x in pools]
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    # the other branch's path is good: its row 2 moves to row 0
    binding.kv_keep(*pools, i32(table), 0, i32([4, 5]), i32([3, 3]), i32(path + [2, -1, -1]),
                    i32([count, 1]), 16)
    assert binding.last_error() == binding.EINVAL
    for x, w in zip(pools, before):
        w[3, :, 5] = w[3, :, 7]
        assert np.array_equal(raw(x), w)


def test_kept_rows_outside_the_pools_are_skipped():
    pools = pools_of("bf16", 4, 2, 16)
    before = [raw(x) for x in pools]
    table = np.array([[0, 99, -5]], np.int32)
    binding.kv_keep(*pools, i32(table), 0, i32([14]), i32([20]), i32([1, 4, 19] + [-1] * 17), i32([3]), 16)
    assert binding.last_error() == binding.EINVAL
    for x, w in zip(pools, before):
        w[0, :, 14] = w[0, :, 15]  # the only move inside
        assert np.array_equal(raw(x), w)


def test_captured_tools_replay_on_new_contents():
    trees, S, table, pages, draft, target, first, rng = draft_problem(11, 5, 12, vocab=3)
    T, R = [len(t) for t in trees], sum(len(t) for t in trees)
    pools = pools_of("q8", pages, 2, 16)
    dev = dict(parents=flat(trees), table=i32(table), S=i32(S), T=i32(T), draft=i64(draft),
               target=i64(target), first=i64(first))

    def step():
        m = binding.tree_rows(dev["parents"], dev["table"], 37, dev["S"], dev["T"], 16, 12)
        a = binding.tree_accept(dev["parents"], dev["draft"], dev["target"], dev["first"], dev["T"])
        binding.kv_keep(*pools, dev["table"], 37, dev["S"], dev["T"], a[0], a[1], 16)
        return m, a
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m, a = step()
    for seed in range(3):
        rng = np.random.default_rng(seed)
        trees = [tree_ref.random_tree(rng, t) for t in T]
        draft, target = rng.integers(0, 2, size=R), rng.integers(0, 2, size=R)
        dev["parents"].copy_(flat(trees))
        dev["draft"].copy_(i64(draft))
        dev["target"].copy_(i64(target))
        want = [raw(x) for x in pools]
        g.replay()
        masks, positions, slots = tree_ref.tree_rows(trees, table, 37, S, 16, R, 1)
        assert np.array_equal(m[0].cpu().numpy().view(np.uint32), masks)
        assert np.array_equal(m[1].cpu().numpy(), positions) and np.array_equal(m[2].cpu().numpy(), slots)
        path, counts, after = tree_ref.accept(trees, draft, target, first, R)
        assert np.array_equal(a[0].cpu().numpy(), path) and np.array_equal(a[1].cpu().numpy(), counts)
        assert np.array_equal(a[2].cpu().numpy(), after)
        r = 0
        for b, t in enumerate(trees):
            for x in want:
                for i in range(counts[b]):
                    s, d = slots[r + path[r + i]], slots[r + i]
                    move(x, "q8", 16, divmod(s, 16), divmod(d, 16))
            r += len(t)
        for x, w in zip(pools, want):
            assert np.array_equal(raw(x), w)
    assert binding.last_error() == binding.OK


def test_on_another_stream():
    trees, S, table, pages, draft, target, first, _ = draft_problem(12, 5, 12, vocab=3)
    T = [len(t) for t in trees]
    args = (flat(trees), i64(draft), i64(target), i64(first), i32(T))
    here = binding.tree_accept(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    there = binding.tree_accept(*args, stream=s)
    rows = binding.tree_rows(args[0], i32(table), 37, i32(S), args[4], 16, 12)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(here, there)) and len(rows) == 3


def test_kept_rows_past_32_bit_offsets():
    pages, hkv, page = 34000, 8, 128
    pools = [torch.zeros((pages, hkv, page, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x in pools:
        x[-2:] = torch.randint(0, 256, (2, hkv, page, 128), dtype=torch.uint8, device="cuda")
    want = [x[-2:].cpu().numpy().copy() for x in pools]
    table = np.array([[pages - 1, pages - 2]], np.int32)
    for x in want:  # rows 126, 127 of the first page, 0 and on of the second
        x[1, :, 127], x[0, :, 0] = x[0, :, 0].copy(), x[0, :, 3].copy()
    _, _, slots = binding.tree_rows(i32([-1, 0, 1, 2, 3, 4]), i32(table), 100, i32([26]), i32([6]), page, 6)
    assert slots.tolist() == [(pages - 1) * page + 126, (pages - 1) * page + 127] + \
        [(pages - 2) * page + i for i in range(4)]
    binding.kv_keep(pools[0].view(torch.float8_e4m3fn), pools[1].view(torch.float8_e4m3fn), i32(table), 100,
                    i32([26]), i32([6]), i32([0, 2, 5, -1, -1, -1]), i32([3]), page)
    assert binding.last_error() == binding.OK
    for x, w in zip(pools, want):
        assert np.array_equal(x[-2:].cpu().numpy(), w)
        assert not x[0].any() and not x[:-2:1000].any()


@pytest.mark.parametrize("window", [0, 1, 5, 31, 32, 33, 70, 1023])
def test_masks_of_deep_trees(window):
    """Ancestors over many words of 32 tokens, windows that end inside and at a word."""
    rng = np.random.default_rng(window)
    deep = [-1] + [t - 1 - int(rng.integers(0, 3)) if t > 3 else t - 1 for t in range(1, 900)]
    trees = [list(range(-1, 1023)), deep, [-1] * 40, [-1] + [0] * 99, list(range(-1, 63))]
    T, S = [len(t) for t in trees], [3, 0, 17, 5, 40]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    width = 1200 // 16
    table = i32(rng.permutation(5 * width).reshape(5, width))
    masks, positions, _ = binding.tree_rows(i32(np.concatenate(trees)), table, 32, i32(S), i32(T), 16,
                                            1024, window)
    words = masks.cpu().numpy().view(np.uint32).reshape(-1, 32)
    bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little").astype(bool)
    row = 0
    for tree, s in zip(trees, S):
        for t in range(len(tree)):
            up, line = t, []
            while up >= 0:
                line.append(up)
                up = tree[up]
            want = np.zeros(1024, bool)
            want[line[:window] if window else line] = True
            assert np.array_equal(bits[row], want) and int(positions[row]) == 32 + s + len(line) - 1
            row += 1
