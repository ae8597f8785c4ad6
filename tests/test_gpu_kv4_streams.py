"""Rows written and read on a stream of their own while the current stream
allocates and writes (GPU)."""
import pytest
import torch

from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step
from gpu_helpers import workload
from kv4_helpers import bits

pytestmark = pytest.mark.gpu

COUNTS, STARTS = [17, 3, 40, 1], [2, 0, 9, 31]


def make():
    return DeviceKv4Step(workload(wl.small_variant(5, batch=4, hq=4, hkv=2, prefix=(60, 60), vocab=64, seed=5)))


def rows(st, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(2, sum(COUNTS), 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]


def busy():
    """Allocations of every small size on the current stream, filled: memory
    that was given back is written again."""
    keep = [torch.full((n,), 2 ** 30 + 7, dtype=torch.int32, device="cuda") for n in [5] * 64 + [128] * 64]
    keep += [torch.full((2, sum(COUNTS), 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    return keep


@pytest.mark.parametrize("kind", ["stream", "address"])
def test_rows_on_a_side_stream(kind):
    want = make()
    start = torch.tensor(STARTS, dtype=torch.int32, device="cuda")
    want.append(*rows(want, 3), COUNTS, start)
    want_k, want_v = want.read(COUNTS, start)
    st = make()
    side = torch.cuda.Stream()
    arg = side if kind == "stream" else side.cuda_stream
    torch.cuda.synchronize()
    for _ in range(3):
        st.k4.zero_()
        st.v4.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                # the call runs well after it was made
        k, v = rows(st, 3)
        s = torch.tensor(STARTS, dtype=torch.int32, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        st.append(k, v, COUNTS, s, arg)
        del k, v, s
        keep = busy()
        torch.cuda.synchronize()
        assert int(st.status[0]) == 0
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got_k, got_v = st.read(COUNTS, start, arg)
        keep += busy()
        torch.cuda.synchronize()
        assert int(st.status[0]) == 0
        assert torch.equal(bits(got_k), bits(want_k)) and torch.equal(bits(got_v), bits(want_v))
