"""The softmax's exponent reference in the 4-bit attention: it is the first
key's score, and moves when a score lies more than 2^60 above it.  Each place
where the larger key can stand, in both tensor-core kernels (GPU)."""
import math

import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step
from gpu_helpers import workload
from kv4_helpers import check_attn, cached_prefix

pytestmark = pytest.mark.gpu

P, CHUNK = 1500, 512
# positions of the larger key.  Kernel 5: spans of 64 keys, warp = span % 4;
# kernel 4: tiles of 128 keys.  Chunks of 512.
PLACES = {"second key": [1], "same span": [40], "another warp": [64 + 5], "later tile": [128 + 7],
          "same warp, later": [256 + 10], "another chunk": [CHUNK + 3], "last key": [P - 1], "tree": ["tree"],
          "rising": [30, 70, 300, 400, CHUNK + 300]}


def plant(w, place, gap):
    """Channel 0 of every key is -h, of the keys at `place` +h (rising: a
    multiple each), so that their scores differ by at least `gap` in log2."""
    q0 = 16.0
    h = gap / (2 * q0 * w.scale * math.log2(math.e))
    w.q[..., 0] = q0
    w.k_cache[:, :, :P, 0] = -h
    w.k_tree[..., 0] = -h
    for i, at in enumerate(place):
        if at == "tree":
            for b in range(w.batch):
                w.k_tree[:, w.seq_rows(b)[0], 0] = h
        else:
            w.k_cache[:, :, at, 0] = h * (1 + 2 * i)


def case(G, nodes, d, place, gap, win=None):
    w = workload(wl.small_variant(5, batch=2, hq=2 * G, hkv=2, d=d, prefix=(P, P), tree=f"random:{nodes},{nodes},4",
                                  vocab=64, paged=False, seed=G + nodes + d))
    plant(w, PLACES[place], gap)
    st = DeviceKv4Step(w, win)
    plan = st.plan()
    assert plan["chunk"] == CHUNK
    k, _ = cached_prefix(w, 0, True)                     # what the format holds of the first key and the planted one
    first = 0 if win is None else P - win[0] + 1 if not win[1] else 0
    if place != "tree":
        score = k[0, :, 0] * float(w.q[0, 0, 0]) * w.scale * math.log2(math.e)
        assert score[PLACES[place][0]] - score[first] > 60
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    return w, st, plan["kernel"]


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("gap", [80, 300])
@pytest.mark.parametrize("G,nodes,d", [(1, 1, 128), (4, 2, 256), (4, 2, 512)])
def test_registers(G, nodes, d, gap, place):
    w, st, kernel = case(G, nodes, d, place, gap)
    assert kernel == 5
    check_attn(w, st, True)


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("G,nodes,d", [(4, 3, 512), (4, 8, 256), (4, 16, 512), (4, 40, 128)])   # 16 .. 128 columns
def test_tensor_memory(G, nodes, d, place):
    w, st, kernel = case(G, nodes, d, place, 80)
    assert kernel == 4
    check_attn(w, st, True)


@pytest.mark.parametrize("place", ["same span", "another warp", "last key", "tree", "rising"])
@pytest.mark.parametrize("d", [128, 512])
@pytest.mark.parametrize("nodes,kernel", [(2, 5), (20, 4)])
def test_in_a_window(nodes, kernel, d, place):
    win = (1300, 100)                                    # keys 100 .. 200 are seen by no row
    w, st, got = case(4, nodes, d, place, 80, win)
    assert got == kernel
    check_attn(w, st, True, win)
