"""The 4-bit and the windowed attention with an fp32 output, a scale of their
own and a descriptor wider than the call (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits, check_attn

pytestmark = pytest.mark.gpu

KINDS = {"4 bits": (lambda w, **kw: DeviceKv4Step(w, **kw), True, None),
         "4 bits, window": (lambda w, **kw: DeviceKv4Step(w, (150, 20), **kw), True, (150, 20)),
         "window": (lambda w, **kw: DeviceWindowStep(w, 150, 20, **kw), False, (150, 20))}


def run(st):
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    return st


def make(nodes, prefix, **kw):
    return workload(wl.small_variant(5, **dict(dict(batch=2, hq=8, hkv=2, prefix=prefix, tree=f"random:1,{nodes},5", vocab=64,
                                                    seed=nodes), **kw)))


@pytest.mark.parametrize("prefix", [(30, 200), (2500, 3000)])     # one chunk, and several to merge
@pytest.mark.parametrize("nodes,d", [(2, 128), (2, 512), (20, 128), (64, 256)])
@pytest.mark.parametrize("kind", KINDS)
def test_fp32_output_rounds_to_the_bf16_one(kind, nodes, d, prefix):
    make_step, four, win = KINDS[kind]
    w = make(nodes, prefix, d=d)
    wide, narrow = run(make_step(w, out_f32=True)), run(make_step(w))
    assert wide.out.dtype == torch.float32
    check_attn(w, wide, four, win)
    # the same arithmetic up to the last rounding
    assert torch.equal(bits(wide.out.to(torch.bfloat16)), bits(narrow.out))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_wider_descriptor_gives_the_same_answer(kind, dtype):
    # 64 nodes and a longer prefix are announced, fewer come: another plan, the same values
    make_step, four, win = KINDS[kind]
    w = make(5, (100, 300), dtype=dtype)
    st = run(make_step(w, max_nodes=64, max_prefix=w.capacity))
    check_attn(w, st, four, win)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nodes", [2, 20])
def test_a_scale_of_its_own(kind, nodes):
    make_step, four, win = KINDS[kind]
    w = make(nodes, (100, 300))
    st = make_step(w)
    plain = run(st).out.clone()
    st.desc.scale = 0.25 * w.scale
    quarter = run(st).out.clone()
    st.desc.scale = 0.0
    st.q.mul_(0.25)                                      # exact in bf16: the same scores
    assert torch.equal(bits(run(st).out), bits(quarter)) and not torch.equal(bits(plain), bits(quarter))
