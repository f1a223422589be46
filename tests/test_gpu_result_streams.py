"""Results of calls on a given stream come from that stream's memory: a block that is
dropped early goes back to the work it was written by."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding

from . import serving_ref as ref
from .gpu_helpers import DevWorkload, ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def stream_of(t):
    """The stream whose pool holds the tensor's block."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


def dev(a):
    return torch.as_tensor(a, dtype=torch.int32).cuda()


def calls():
    """name -> (a call's results, given stream=)."""
    prefix, S, A, free = dev([0, 1]), dev([20, 3]), dev([1, 1]), dev(list(range(2, 12)))
    table = binding.fork_device(prefix, 20, S, 16, free, 8)[0]
    pool = [binding.q4_pool(12, 2, 16) for _ in range(2)]
    slots = torch.arange(5, device="cuda")
    probs = [ref.Problem([90, 20], [3, 5], 30, 16, 2, 32, window=w, q4=q4)
             for w, q4 in ((50, False), (0, True))]
    for p in probs:
        p.run()
    from shared_prefix_fan_gb300.workloads import draw, small_spec
    w = DevWorkload(draw(small_spec(h_q=8, h_kv=2, prefix_len=128, q_rows=[6, 3],
                                    suffix_lens=[10, 20])))
    part_o = torch.randn((3, 10, 128), device="cuda")
    part_ml = torch.ones((3, 10, 2), device="cuda")
    torch.cuda.synchronize()
    return {
        "fork_device": lambda s: binding.fork_device(prefix, 20, S, 16, free, 8, stream=s),
        "extend_device": lambda s: binding.extend_device(table, 20, S, A, 16, free, 4, stream=s),
        "kv_read_q4": lambda s: binding.kv_read_q4(*pool, slots, 16, stream=s),
        "attn_window": lambda s: probs[0].run(stream=s),
        "attn_q4": lambda s: probs[1].run(stream=s),
        "attn": lambda s: w.run(stream=s),
        "lse_merge": lambda s: binding.lse_merge(part_o, part_ml, stream=s),
    }


NAMES = ["fork_device", "extend_device", "kv_read_q4", "attn_window", "attn_q4", "attn",
         "lse_merge"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_handle", [False, True])
def test_results_belong_to_the_given_stream(name, as_handle):
    call = calls()[name]
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = call(st.cuda_stream if as_handle else st)
    st.synchronize()
    here = torch.cuda.current_stream().cuda_stream
    for x, y in zip(got, want):
        assert stream_of(x) == st.cuda_stream != here
        assert torch.equal(x, y)
    for x in call(None):
        assert stream_of(x) == here
    for x in call(here):
        assert stream_of(x) == here
    assert torch.cuda.current_stream().cuda_stream == here


@pytest.mark.parametrize("name", NAMES)
def test_a_dropped_result_is_not_lent_to_the_current_stream(name):
    call = calls()[name]
    st = torch.cuda.Stream()
    got = call(st)
    sizes = [(tuple(x.shape), x.dtype, x.data_ptr()) for x in got]
    del got
    again = [torch.empty(shape, dtype=dt, device="cuda") for shape, dt, _ in sizes]
    assert not {x.data_ptr() for x in again} & {p for _, _, p in sizes}
    torch.cuda.synchronize()
