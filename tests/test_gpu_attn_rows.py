"""Windowed attention and attention over 4-bit pools against a plain 64-bit form.
In every problem the slots that no row sees hold NaN, and with a window the table
entries of pages that nobody sees are no page at all."""
import numpy as np
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu
# half a step of the type P is rounded to for the product with V
P_STEP = {False: 2.0 ** -8, True: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def run(S, T, P, hq, hkv, page, out_dtype="f32", **kw):
    prob = ref.Problem(S, T, P, hq, hkv, page, **kw)
    out, lse = prob.run(out_dtype)
    rc = binding.last_error_detail()
    assert rc[0] == binding.OK, rc
    ref.check_attention(out, lse, prob.reference(), P_STEP[prob.q4], str(kw))
    return prob, out, lse


SHAPES = [  # S, T, P, hq, hkv, page
    ([1], [1], 0, 8, 1, 16), ([1], [1], 1, 4, 4, 16), ([16, 16, 16], [4, 4, 4], 256, 8, 1, 16),
    ([130], [1], 0, 8, 2, 64), ([5, 70, 300], [1, 1, 1], 500, 16, 2, 32),
    ([40, 3, 90], [7, 0, 33], 77, 10, 2, 16), ([200], [200], 50, 8, 1, 64),
    ([90, 64], [40, 25], 130, 14, 2, 128), ([129, 1, 255], [1, 1, 2], 128, 12, 4, 16),
    ([600], [100], 0, 128, 1, 16), ([33, 20], [2, 9], 640, 40, 8, 64),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (17, 4), (100, 0), (100, 20),
                                          (128, 128), (1000, 3), (40, 700)])
def test_window(shape, window, sinks):
    run(*shape, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal,window,sinks,gs", [(True, 0, 0, 1.0), (False, 0, 0, 0.3),
                                                    (True, 1, 0, 2.0), (True, 30, 4, 1.0),
                                                    (True, 200, 150, 0.01)])
def test_q4(shape, causal, window, sinks, gs):
    run(*shape, causal=causal, window=window, sinks=sinks, gs=gs, q4=True, seed=7)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("splits", [1, 2, 5])
def test_forced_splits(q4, splits):
    binding.set_option(binding.OPT_SPLITS, splits)
    try:
        run([300, 260], [3, 30], 700, 16, 2, 32, window=500, sinks=5, q4=q4, seed=splits)
    finally:
        binding.set_option(binding.OPT_SPLITS, 0)


@pytest.mark.parametrize("q4", [False, True])
def test_wide_scores_and_bf16_output(q4):
    """Scores far apart, so that references move and whole shards vanish."""
    run([400, 100], [40, 3], 600, 16, 2, 16, "bf16", window=700, sinks=2, q4=q4, k_amp=12.0)


def test_q4_infinite_scores_stay_out():
    """Group scales from the smallest to the largest in one cache."""
    prob = ref.Problem([100], [5], 60, 8, 2, 16, q4=True, seed=2, k_amp=40.0)
    out, lse = prob.run()
    ref.check_attention(out, lse, prob.reference(), P_STEP[True])


@pytest.mark.parametrize("q4", [False, True])
def test_many_branches(q4):
    rng = np.random.default_rng(1)
    S = rng.integers(1, 60, 200)
    run(S, np.ones(200, int), 96, 8, 1, 16, window=70, sinks=4, q4=q4)


@pytest.mark.parametrize("q4", [False, True])
def test_repeats_are_bitwise_equal(q4):
    prob = ref.Problem([300, 200], [20, 31], 400, 16, 2, 32, window=300, sinks=4, q4=q4)
    a = prob.run()
    for _ in range(3):
        b = prob.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q4", [False, True])
def test_streams_and_no_lse(q4):
    probs = [ref.Problem([90, 200], [3, 5], 300, 16, 2, 32, window=128, sinks=4, q4=q4, seed=s)
             for s in (1, 2)]
    for p in probs:
        p.run()
    torch.cuda.synchronize()
    outs = []
    for p in probs * 2:
        st = torch.cuda.Stream()
        out = torch.empty((8, 16, 128), device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        o, lse = p.run(stream=st, out=out, want_lse=False)
        assert lse is None
        outs.append((p, out))
    torch.cuda.synchronize()
    for p, out in outs:
        ref.check_attention(out, None, p.reference(), P_STEP[q4])


def test_kinds_alternate_on_one_stream():
    """Full, windowed and 4-bit layers in turn: each keeps its own plan."""
    probs = [ref.Problem([90, 200], [1, 1], 300, 16, 2, 32, window=w, sinks=s, q4=q, seed=3)
             for w, s, q in ((128, 4, False), (0, 0, True), (64, 1, True), (64, 1, False))]
    refs = [p.reference() for p in probs]
    for _ in range(3):
        for p, r in zip(probs, refs):
            out, lse = p.run()
            ref.check_attention(out, lse, r, P_STEP[p.q4])


@pytest.mark.parametrize("q4", [False, True])
def test_bad_page_ids_are_reported(q4):
    prob = ref.Problem([50], [2], 100, 8, 1, 16, window=400, q4=q4)
    prob.run()
    assert binding.last_error() == binding.OK
    for bad in (-1, prob.num_pages, 2 ** 31 - 1):
        prob.dev[3][0, 2] = bad
        prob.run()
        assert binding.last_error() == binding.EINVAL


@pytest.mark.parametrize("q4", [False, True])
def test_capture_is_refused(q4):
    prob = ref.Problem([50], [2], 100, 8, 1, 16, window=400, q4=q4)
    out, lse = prob.run()
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(binding.FanoutError) as e:
            prob.run(out=out, lse=lse)
    assert e.value.code == binding.EUNSUPPORTED


def test_other_group_sizes_in_the_full_attention():
    """G that does not divide 128, more than one query tile: fanout_attn itself."""
    import oracle
    from shared_prefix_fan_gb300.workloads import draw, small_spec
    from .gpu_helpers import DevWorkload, compare, oracle_ref
    assert oracle
    for hq, hkv in ((10, 2), (7, 1), (12, 4)):
        w = draw(small_spec(h_q=hq, h_kv=hkv, prefix_len=128, q_rows=[60, 3, 44],
                            suffix_lens=[100, 20, 44]))
        d = DevWorkload(w)
        compare(*d.run(), *oracle_ref(w))


def test_decode_loop_on_the_4_bit_cache():
    """Fork inside a page, copy the shared part, then steps of: grow the tables on
    the device, append, attend. Every step against the 64-bit form on the values
    the cache holds."""
    page, hkv, hq, P, gs, W, sinks = 16, 2, 8, 40, 0.5, 48, 4
    rng = np.random.default_rng(9)
    to = lambda a: torch.as_tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    n = 60
    ids = rng.permutation(n).astype(np.int32)
    prefix, free = ids[:3], ids[3:]
    pools = torch.zeros((2, n, hkv, page * 72), dtype=torch.uint8, device="cuda")
    kv = torch.from_numpy(rng.standard_normal((2, P, hkv, 128)).astype(np.float32)).bfloat16()
    slots = torch.from_numpy((prefix[np.arange(P) // page].astype(np.int64) * page +
                              np.arange(P) % page)).cuda()
    binding.kv_append_q4(kv[0].cuda(), kv[1].cuda(), pools[0], pools[1], slots, page, gs, gs)
    S = np.zeros(3, np.int64)
    table, cow, used = binding.fork_device(to(prefix), P, to(S), page, to(free), 12)
    binding.copy_pages_q4(pools[0], pools[1], cow, page)
    for step in range(25):
        A = rng.integers(1, 4, 3) if step % 3 == 0 else np.ones(3, np.int64)
        R = int(A.sum())
        slots, used = binding.extend_device(table, P, to(S), to(A), page, to(free), R + 2, used)
        new = torch.from_numpy(rng.standard_normal((2, R + 2, hkv, 128)).astype(np.float32))
        new = new.bfloat16().cuda()
        binding.kv_append_q4(new[0], new[1], pools[0], pools[1], slots, page, gs, gs)
        S = S + A
        q = torch.from_numpy(rng.standard_normal((R, hq, 128)).astype(np.float32)).bfloat16()
        window = W if step % 2 else 0
        out, lse = binding.attn_q4(q.cuda(), pools[0], pools[1], table, P, S, A, hq, hkv, page,
                                   128 ** -0.5, True, gs, gs, window, sinks if window else 0)
        assert binding.last_error() == binding.OK
        k64, v64 = (ref.decode(*ref.parts_of(p.cpu().numpy(), page), gs) for p in pools)
        r = ref.attention(q.double().numpy(), k64, v64, table.cpu().numpy(), P, S, A, page,
                          128 ** -0.5, True, window, sinks if window else 0)
        ref.check_attention(out, lse, r, P_STEP[True], f"step {step}")


def device_reference(prob):
    """`prob.reference()` of a problem with one branch, computed on the device (64
    bits): for lengths at which the host form takes minutes."""
    P, S, T, page, G = prob.P, prob.S[0], prob.T[0], prob.page, prob.hq // prob.hkv
    n = P + S
    j = torch.arange(n, device="cuda")
    pos = torch.arange(n - T, n, device="cuda")[:, None]
    see = (j <= pos) if prob.causal else torch.ones((T, n), dtype=torch.bool, device="cuda")
    if prob.window:
        see = see & ((j > pos - prob.window) | (j < prob.sinks))
    at = torch.from_numpy(prob.table[0].astype(np.int64)).cuda()[j // page], j % page
    q = prob.q.double().cuda()
    parts = []
    for h in range(prob.hkv):
        k, v = (torch.from_numpy(np.ascontiguousarray(x[:, h])).cuda()[at]
                for x in (prob.k64, prob.v64))
        for g in range(h * G, (h + 1) * G):
            x = (q[:, g] @ k.T * prob.scale).masked_fill(~see, -torch.inf)
            p = torch.softmax(x, -1)
            e = (q[:, g].abs() @ k.abs().T * prob.scale).masked_fill(~see, 0.0)
            parts.append((p @ v, torch.logsumexp(x, -1), p @ v.abs(), e.amax(-1),
                          see.double() @ v.abs()))
    return tuple(torch.stack([p[i] for p in parts], 1).cpu().numpy() for i in range(5))


@pytest.mark.parametrize("hq,hkv,page,P,T,window,sinks,gs", [
    (40, 8, 16, 4588, 1011, 2714, 100, 0.25), (64, 8, 16, 4500, 700, 0, 0, 1.0),
    (8, 8, 64, 3900, 515, 0, 0, 0.5), (16, 1, 32, 8000, 40, 5000, 7, 1.0)])
def test_long_sweeps_of_the_4_bit_cache(hq, hkv, page, P, T, window, sinks, gs):
    """Many key tiles through one ring: a stage that is refilled while a warp still
    reads its words gives wrong rows here, and other ones from run to run."""
    prob = ref.Problem([T], [T], P, hq, hkv, page, window=window, sinks=sinks, q4=True, gs=gs)
    want, first = device_reference(prob), None
    for _ in range(4):
        out, lse = prob.run()
        assert binding.last_error_detail()[0] == binding.OK
        ref.check_attention(out, lse, want, P_STEP[True])
        first = first or (out, lse)
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_output_aligned_to_16_bytes_only(q4, out_dtype):
    prob = ref.Problem([40, 300], [40, 3], 128, 8, 1, 16, window=200, sinks=3, q4=q4)
    dt = torch.float32 if out_dtype == "f32" else torch.bfloat16
    n, lead = 43 * 8 * 128, 16 // dt.itemsize
    buf = torch.full((n + 2 * lead,), 7.0, dtype=dt, device="cuda")
    out = buf[lead:lead + n].view(43, 8, 128)
    assert out.data_ptr() % 32 == 16
    _, lse = prob.run(out_dtype, out=out)
    ref.check_attention(out, lse, prob.reference(), P_STEP[q4])
    assert (buf[:lead] == 7).all() and (buf[lead + n:] == 7).all()


@pytest.mark.parametrize("q4", [False, True])
def test_table_validation_leaves_hidden_pages_alone(q4):
    """With the host-side check on: entries that the window hides may be anything,
    a bad one that it shows is refused."""
    prob = ref.Problem([40, 30, 9], [3, 2, 0], 300, 8, 2, 16, window=50, sinks=20, q4=q4)
    bad = prob.table.copy()
    bad[:, 2:] = -1  # hidden, except from the oldest key a row sees on
    for b, (s, t) in enumerate(((40, 3), (30, 2))):
        first = (300 + s - t - 50 + 1) // 16
        bad[b, first:] = prob.table[b, first:]
    low = min((300 + s - t - 50 + 1) // 16 for s, t in ((40, 3), (30, 2)))
    bad[0, low:18] = prob.table[0, low:18]  # row 0 stands for the shared pages
    bad[2] = -1                             # no rows: nothing of it is read
    binding.set_option(binding.OPT_VALIDATE_TABLE, 1)
    try:
        prob.call_table = bad
        out, lse = prob.run()
        ref.check_attention(out, lse, prob.reference(), P_STEP[q4])
        for b, i in ((0, 1), (1, bad.shape[1] - 3)):
            if bad[b, i] < 0:
                continue
            worse = bad.copy()
            worse[b, i] = prob.num_pages
            prob.dev[3] = torch.from_numpy(worse).cuda()
            with pytest.raises(binding.FanoutError) as e:
                prob.run()
            assert e.value.code == binding.EINVAL
    finally:
        binding.set_option(binding.OPT_VALIDATE_TABLE, 0)


@pytest.mark.parametrize("T", [1, 20])
def test_largest_queries_on_keys_of_zeros(T):
    """Scores are 0 whatever the scales: the output is the mean of V."""
    n, page, hkv, hq, ks = 200, 16, 2, 16, 1e6
    pools = [binding.q4_pool(13, hkv, page) for _ in range(2)]
    v = torch.from_numpy(np.random.default_rng(3).standard_normal((n, hkv, 128)).astype(np.float32))
    slots = torch.arange(n, device="cuda")
    binding.kv_append_q4(torch.zeros((n, hkv, 128), dtype=torch.bfloat16, device="cuda"),
                         v.bfloat16().cuda(), *pools, slots, page, ks, 1.0)
    q = torch.full((T, hq, 128), 3e38, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None]
    out, lse = binding.attn_q4(q, *pools, table, 0, [n], [T], hq, hkv, page, 1.0, False, ks, 1.0)
    held = ref.decode(*ref.parts_of(pools[1].cpu().numpy(), page), 1.0)
    held = held.transpose(0, 2, 1, 3).reshape(-1, hkv, 128)[:n]
    want = np.repeat(held.mean(0), hq // hkv, 0)
    # P is 1 for every key: exact in f16; the sums are of fp32 (see check_attention)
    tol = np.repeat(np.abs(held).mean(0), hq // hkv, 0) * 2.0 ** -16 + 1e-30
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (lse.double().cpu() - np.log(n)).abs().max() <= 2.0 ** -16 + 2.0 ** -22 * np.log(n)


@pytest.mark.parametrize("q4", [False, True])
def test_windows_wider_than_32_bits(q4):
    a = ref.Problem([40, 30], [3, 2], 64, 8, 2, 16, window=2 ** 31 - 1, sinks=0, q4=q4)
    x = a.run()
    a.window, a.sinks = 2 ** 32 + 5, 2 ** 40
    y = a.run()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("q4", [False, True])
def test_pools_past_32_bit_offsets(q4):
    """The same pages at both ends of pools of more than 4 GB."""
    prob = ref.Problem([200, 70], [3, 1], 128, 8, 8, 64, window=150, sinks=10, q4=q4)
    near = prob.run()
    block = prob.k_pool[0].numel() * prob.k_pool.element_size()
    far = 2 ** 32 // block + 7
    pools = [torch.zeros((far + prob.num_pages, *prob.k_pool.shape[1:]), dtype=prob.k_pool.dtype,
                         device="cuda") for _ in range(2)]
    for pool, x in zip(pools, (prob.k_pool, prob.v_pool)):
        pool[far:] = x.cuda()
    table = prob.table + np.where(prob.table >= 0, far, 0).astype(np.int32)
    prob.dev = [prob.dev[0], *pools, torch.from_numpy(table).cuda()]
    out, lse = prob.run()
    assert torch.equal(out, near[0]) and torch.equal(lse, near[1])
    if q4:  # and the rows of the last page
        slots = (torch.arange(64, device="cuda") + (far + prob.num_pages - 1) * 64)
        new = torch.randn((64, 8, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        binding.kv_append_q4(new.bfloat16(), -new.bfloat16(), *pools, slots, 64)
        small = [binding.q4_pool(1, 8, 64) for _ in range(2)]
        binding.kv_append_q4(new.bfloat16(), -new.bfloat16(), *small, slots % 64, 64)
        assert torch.equal(pools[0][-1], small[0][0]) and torch.equal(pools[1][-1], small[1][0])
        k, v = binding.kv_read_q4(*pools, slots, 64)
        ks, vs = binding.kv_read_q4(*small, slots % 64, 64)
        assert torch.equal(k, ks) and torch.equal(v, vs)
