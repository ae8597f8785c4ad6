"""A sequence's answer does not depend on what its neighbours' rows hold: the
tree rows behind its own belong to the next sequence or KV head, and may be
NaN or infinite (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceStep, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits

pytestmark = pytest.mark.gpu

WIN = (100, 20)
STEPS = {
    "full": lambda w: DeviceStep(w),
    "full, fp32 out": lambda w: DeviceStep(w, out_f32=True),
    "window": lambda w: DeviceWindowStep(w, *WIN),
    "4 bits": lambda w: DeviceKv4Step(w),
    "4 bits, window": lambda w: DeviceKv4Step(w, WIN),
}

# (step, plan kernel, workload)
CASES = [
    ("full", 0, dict(dtype="f32", batch=3)),
    ("full, fp32 out", 1, dict(batch=3)),
    ("full, fp32 out", 1, dict(batch=3, d=256)),
    ("full", 2, dict(batch=1, hq=16)),
    ("full", 2, dict(batch=1, hq=16, d=256)),
    ("full", 3, dict(batch=3)),
    ("window", 0, dict(dtype="f32", batch=3)),
    ("window", 1, dict(batch=3)),
    ("window", 1, dict(batch=3, d=256)),
    ("4 bits", 0, dict(dtype="f32", batch=3)),
    ("4 bits", 4, dict(batch=3)),
    ("4 bits, window", 4, dict(batch=3, d=512)),
    ("4 bits", 5, dict(batch=3)),
    ("4 bits, window", 5, dict(batch=3, d=512)),
]


def run(st):
    st.out.fill_(float("nan"))
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    return st.out.clone()


@pytest.mark.parametrize("nodes", [1, 16, 33, 64])
@pytest.mark.parametrize("prefix", [(0, 0), (130, 300)])
@pytest.mark.parametrize("kind,kernel,kw", CASES, ids=[f"{c[0]}-{c[1]}-{i}" for i, c in enumerate(CASES)])
def test_neighbours_rows_do_not_matter(kind, kernel, kw, prefix, nodes):
    if kernel == 5:
        nodes = min(nodes, 2)                            # 8 rows of a KV head at most
    elif kernel and nodes == 1:
        nodes = 40 if kernel == 2 else 17
    if kernel == 2 and nodes == 16:
        nodes = 20                                       # two row tiles at 8 heads a KV head
    w = workload(wl.small_variant(5, **dict(dict(hq=8, hkv=2, prefix=prefix, tree=f"random:{nodes},{nodes},5", vocab=64,
                                                 seed=nodes), **kw)))
    st = STEPS[kind](w)
    assert (st.plan())["kernel"] == kernel
    good = run(st)
    G, n = w.spec.hq // 2, nodes
    for bad in (float("nan"), float("inf")):
        k, v, q = st.k_tree.clone(), st.v_tree.clone(), st.q.clone()
        if w.batch > 1:                                  # the middle sequence
            mine = [slice(0, n), slice(2 * n, 3 * n)]
            st.k_tree[:, n:2 * n] = bad
            st.v_tree[:, n:2 * n] = bad
            st.q[n:2 * n] = bad
            outs = lambda o: [o[m] for m in mine]
        else:                                            # the next KV head
            st.k_tree[1] = bad
            st.v_tree[1] = bad
            outs = lambda o: [o[:, :G]]
        for a, b in zip(outs(run(st)), outs(good)):
            assert torch.equal(bits(a.contiguous()), bits(b.contiguous()))
        st.k_tree.copy_(k)
        st.v_tree.copy_(v)
        st.q.copy_(q)
