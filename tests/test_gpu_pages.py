"""Page ids out of range in every attention kernel: flagged, and read as zeros
whatever number the table holds (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceStep, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits

pytestmark = pytest.mark.gpu

WIN = (250, 40)

# (name, plan kernel, workload, step, plan)
CASES = [
    ("full", 0, dict(dtype="f32", batch=2, tree="random:3,3,2"), lambda w: DeviceStep(w), lambda s: tv.tv_attn_plan(s.desc)),
    ("full", 1, dict(batch=2, tree="random:20,20,5"), lambda w: DeviceStep(w, out_f32=True),
     lambda s: tv.tv_attn_plan(s.desc)),
    ("full", 2, dict(batch=1, d=256, tree="random:60,60,6"), lambda w: DeviceStep(w), lambda s: tv.tv_attn_plan(s.desc)),
    ("full", 3, dict(batch=2, tree="random:20,20,5"), lambda w: DeviceStep(w), lambda s: tv.tv_attn_plan(s.desc)),
    ("window", 0, dict(dtype="f32", batch=2, tree="random:3,3,2"), lambda w: DeviceWindowStep(w, *WIN),
     lambda s: tv.tv_window_attn_plan(s.desc, s.win)),
    ("window", 1, dict(batch=2, tree="random:20,20,5"), lambda w: DeviceWindowStep(w, *WIN),
     lambda s: tv.tv_window_attn_plan(s.desc, s.win)),
] + [("4 bits" + (", window" if win else ""), kernel, kw, lambda w, win=win: DeviceKv4Step(w, win),
      lambda s: tv.tv_kv4_attn_plan(s.desc, s.win))
     for win in (None, WIN)
     for kernel, kw in ((0, dict(dtype="f32", batch=2, tree="random:3,3,2")), (4, dict(batch=2, tree="random:20,20,5")),
                        (4, dict(batch=2, d=512, tree="random:20,20,5")), (5, dict(batch=2, tree="random:2,2,1")),
                        (5, dict(batch=2, d=512, tree="random:1,1,1")))]


@pytest.mark.parametrize("name,kernel,kw,make,plan", CASES, ids=[f"{c[0]}-{c[1]}-{i}" for i, c in enumerate(CASES)])
def test_any_number_out_of_range_reads_as_zeros(name, kernel, kw, make, plan):
    # pages 0 (sinks) and 33 (positions 528 .. 543, in every row's window)
    w = workload(wl.small_variant(5, hq=8, hkv=2, prefix=(600, 700), vocab=64, paged=True, **kw))
    st = make(w)
    assert plan(st)["kernel"] == kernel
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    good = st.out.clone()
    for page in (0, 33):
        table = st.page_table.clone()
        outs = []
        for bad in (-1, -2 ** 31, 2 ** 31 - 1, st.desc.num_pages):
            st.page_table[0, page] = bad
            st.status.zero_()
            st.attn()
            torch.cuda.synchronize()
            assert int(st.status[0]) == 8, f"id {bad}"
            outs.append(st.out.clone())
        st.page_table.copy_(table)
        assert bool(torch.isfinite(outs[0]).all()) and not torch.equal(bits(outs[0]), bits(good))
        for out in outs[1:]:
            assert torch.equal(bits(out), bits(outs[0]))
