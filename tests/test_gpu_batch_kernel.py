"""The batch kernel (persistent CTA pairs) gives the same bits in every call,
and the one-CTA kernel's result within the roundings of both."""
import pytest
import torch

from gpu_helpers import workload
from speculative_decoding_tree_gb300 import tv_attn_plan
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceStep

pytestmark = pytest.mark.gpu


def attention(w, out_f32=False, absolute=False):
    st = DeviceStep(w, out_f32=out_f32)
    if absolute:
        st.v_cache = st.v_cache.abs()
        st.v_tree = st.v_tree.abs()
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    return tv_attn_plan(st.desc), st.out.float()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("batch,seed", [(6, 62), (4, 61), (9, 63)])
def test_batch_kernel_repeats_and_matches(batch, seed, paged):
    # trees of 16 to 64 nodes over 3 or 4 key chunks: both row tiles of a pair
    # live, partly live or empty, several units per CTA pair
    w = workload(wl.CONFIGS[5].replace(batch=batch, prefix=(4096, 8192), vocab=301, seed=seed, paged=paged))
    plan, one = attention(w, out_f32=True)
    assert plan["kernel"] == 1
    _, size = attention(w, out_f32=True, absolute=True)
    plan, first = attention(w)
    assert plan["kernel"] == 3
    # With A = sum_j p_j |v_j|, the roundings to bf16 are: p in either kernel
    # (2^-8 A each), the batch kernel's partials (2^-8 A) and its output
    # (2^-8 A, |out| <= A).  `size` is A within its own 2^-8; fp32 sums of
    # 8192 terms add less than 2^-10 A.
    tol = (4 * 2.0 ** -8 + 2.0 ** -10) * size * (1 + 2.0 ** -7)
    assert bool(((first - one).abs() <= tol).all())
    for _ in range(12):
        _, again = attention(w)
        assert torch.equal(again, first)
