"""Attention over a sliding window with sinks (fp32 and bf16 caches) vs the
oracle, within the bounds that kv4_helpers.reference derives (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceStep, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits, check_attn

pytestmark = pytest.mark.gpu


def step(w, win, **kw):
    st = DeviceWindowStep(w, *win, **kw)
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    return st


def spec(n=5, **kw):
    kw.setdefault("vocab", 64)
    return wl.small_variant(n, **kw)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("win", [(20, 4), (300, 0)])
def test_small_variant(n, win):
    w = workload(spec(n))
    check_attn(w, step(w, win), False, win)


@pytest.mark.parametrize("dtype,d,nodes", [("bf16", 128, 20), ("f32", 128, 1), ("f32", 256, 20), ("bf16", 512, 3),
                                           ("bf16", 256, 64), ("bf16", 128, 1)])
@pytest.mark.parametrize("win", [(1, 0), (1, 300), (2, 1), (5, 16), (16, 4), (100, 4), (130, 130), (257, 128),
                                 (10 ** 6, 0)])
@pytest.mark.parametrize("paged", [False, True])
def test_windows(dtype, d, nodes, win, paged):
    w = workload(spec(5, batch=2, hq=4, hkv=2, d=d, dtype=dtype, prefix=(280, 700), seed=sum(win) % 89 + d,
                      tree=f"random:{nodes},{nodes},9", paged=paged))
    check_attn(w, step(w, win), False, win)


@pytest.mark.parametrize("P", [0, 1, 15, 16, 127, 128, 129, 143, 144, 145, 500])
@pytest.mark.parametrize("win", [(16, 3), (112, 16)])
def test_ragged_prefixes(P, win):
    w = workload(spec(3, prefix=(P, P), tree="random:13,13,5", seed=P))
    check_attn(w, step(w, win), False, win)


@pytest.mark.parametrize("batch", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_chunks(batch, dtype):
    win = (4000, 140)
    w = workload(spec(5, batch=batch, hq=4, hkv=2, prefix=(5000, 6000), tree="random:3,9,3", dtype=dtype, seed=7))
    st = step(w, win)
    assert tv.tv_window_attn_plan(st.desc, st.win)["num_splits"] > 1
    check_attn(w, st, False, win)


@pytest.mark.parametrize("dtype,nodes", [("bf16", 9), ("f32", 9), ("bf16", 1)])
@pytest.mark.parametrize("win", [(30, 5), (100, 100), (300, 0)])
def test_contents_that_no_row_sees_do_not_matter(dtype, nodes, win):
    # NaN in every cache row that is neither a sink nor in the root's window
    w = workload(spec(4, prefix=(450, 450), tree=f"random:{nodes},{nodes},5", dtype=dtype, seed=nodes))
    a = step(w, win)
    lo, hi = win[1], 450 - win[0] + 1
    for bad in (float("nan"), float("inf")):
        w.k_cache[:, :, lo:hi] = bad
        w.v_cache[:, :, lo:hi] = bad
        st = step(w, win)
        check_attn(w, st, False, win)
        assert torch.equal(bits(st.out), bits(a.out))


def test_unseen_pages_may_hold_any_id():
    win = (100, 20)
    for dtype in ("bf16", "f32"):
        w = workload(spec(5, batch=2, prefix=(700, 800), tree="random:5,9,4", dtype=dtype, seed=12))
        a = step(w, win)
        b = DeviceWindowStep(w, *win)
        b.page_table[:, 3:30] = -7                       # positions 48..479
        b.mask()
        b.attn()
        torch.cuda.synchronize()
        assert int(b.status[0]) == 0 and torch.equal(bits(a.out), bits(b.out))
        b.page_table[1, 0] = -1                          # a page with sinks
        b.attn()
        torch.cuda.synchronize()
        assert int(b.status[0]) == 8


def test_a_window_over_everything_is_full_attention():
    # the same kernels run in both calls (CUDA cores; one tensor-core CTA per tile, with fp32 partials for an fp32
    # output): the same bytes
    for n, kw in ((1, {}), (3, dict(tree="random:16,16,5"))):
        w = workload(spec(n, **kw))
        full = DeviceStep(w, out_f32=True)
        full.mask()
        full.attn()
        st = step(w, (10 ** 9, 0), out_f32=True)
        assert torch.equal(bits(st.out), bits(full.out))


def test_repeats_streams_and_graphs_give_the_same_bytes():
    win = (600, 4)
    w = workload(spec(5, batch=4, prefix=(40, 2500), seed=21))
    st = step(w, win)
    want = st.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    st.attn(side)
    side.synchronize()
    assert torch.equal(bits(st.out), bits(want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            st.attn()
    for _ in range(4):
        st.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(st.out), bits(want))


def test_window_then_commit_then_window():
    win = (40, 4)
    w = workload(spec(5, batch=3, hq=8, hkv=2, prefix=(20, 90), seed=31))
    st = DeviceWindowStep(w, *win, max_prefix=w.capacity)
    for _ in range(2):
        st.mask()
        st.attn()
        torch.cuda.synchronize()
        check_attn(w, st, False, win)
        st.accept_commit()
        torch.cuda.synchronize()
        w.k_cache, w.v_cache, w.prefix_len = st.k_cache.cpu(), st.v_cache.cpu(), st.prefix_len.cpu()


def test_the_same_window_on_both_caches():
    # a cache whose values the 4-bit format holds exactly: both attentions answer the same within rounding
    win = (200, 10)
    w = workload(spec(5, batch=2, hq=4, hkv=2, prefix=(300, 600), seed=2))
    w.k_cache.copy_(torch.nan_to_num(w.k_cache).clamp(-3, 3).round())
    w.v_cache.copy_(torch.nan_to_num(w.v_cache).clamp(-3, 3).round())
    w.k_cache[..., ::32] = 7
    w.v_cache[..., 0] = 7
    a = step(w, win)
    b = DeviceKv4Step(w, win)
    b.mask()
    b.attn()
    torch.cuda.synchronize()
    check_attn(w, a, False, win)
    check_attn(w, b, False, win)
