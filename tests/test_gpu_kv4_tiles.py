"""The 4-bit attention's kernels tile by tile: each query tile width and
head_dim over many key tiles per CTA, with and without a window, and two calls
in flight."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits, check_attn

pytestmark = pytest.mark.gpu

# (heads of one KV head, nodes): rows 3, 8 (registers), 12, 24, 40, 64, 75 and
# 2 x 80, 100 (tcgen05 tiles of 16 .. 128 columns), groups of 40 and of 64
SHAPES = [(3, 1), (2, 4), (4, 3), (8, 3), (40, 1), (16, 4), (5, 15), (40, 4), (10, 10), (64, 3)]


def two_sequences(G, nodes, d, paged, dtype="bf16", prefix=(1500, 1790)):
    # a chunk of a batch has four tiles or more
    return workload(wl.small_variant(5, batch=2, hq=G, hkv=1, d=d, dtype=dtype, prefix=prefix, paged=paged, vocab=64,
                                     tree=f"random:{nodes},{nodes},4", seed=G + nodes + d))


def run(w, win=None, kind=DeviceKv4Step):
    st = kind(w, win) if kind is DeviceKv4Step else kind(w, *win)
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    return st


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("G,nodes", SHAPES)
def test_many_tiles(G, nodes, d, paged):
    w = two_sequences(G, nodes, d, paged)
    st = run(w)
    plan = tv.tv_kv4_attn_plan(st.desc)
    assert plan["chunk"] >= 512 and plan["kernel"] == (5 if G * nodes <= 8 else 4)
    check_attn(w, st, True)
    again = run(w)
    assert torch.equal(bits(st.out), bits(again.out))


@pytest.mark.parametrize("win", [(1000, 200), (700, 0), (9, 1300)])
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("G,nodes", [(3, 1), (4, 3), (8, 3), (16, 4), (10, 10)])
def test_many_tiles_of_a_window(G, nodes, d, win):
    w = two_sequences(G, nodes, d, True)
    check_attn(w, run(w, win), True, win)


@pytest.mark.parametrize("win", [(1000, 200), (700, 0), (9, 1300)])
@pytest.mark.parametrize("d,paged", [(128, True), (128, False), (256, True), (256, False)])
@pytest.mark.parametrize("G,nodes", [(3, 1), (8, 3), (10, 30)])
def test_many_tiles_of_a_window_in_16_bits(G, nodes, d, paged, win):
    w = two_sequences(G, nodes, d, paged)
    st = run(w, win, DeviceWindowStep)
    assert tv.tv_window_attn_plan(st.desc, st.win)["kernel"] == 1
    check_attn(w, st, False, win)


@pytest.mark.parametrize("G,dtype", [(65, "bf16"), (4, "f32")])
def test_what_the_tensor_cores_do_not_take(G, dtype):
    w = two_sequences(G, 2, 128, True, dtype, (100, 300))
    st = run(w)
    assert tv.tv_kv4_attn_plan(st.desc)["kernel"] == 0
    check_attn(w, st, True)


@pytest.mark.parametrize("G,nodes", [(2, 4), (4, 3), (10, 10)])
def test_two_calls_in_flight(G, nodes):
    # two sequences of calls on two streams, each with its own workspace,
    # captured into two graphs and replayed at once
    steps, wants, graphs = [], [], []
    for seed in (0, 1):
        w = two_sequences(G, nodes, 128, True, prefix=(3000 + 500 * seed, 5000))
        st = run(w)
        steps.append(st)
        wants.append(st.out.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            stream = torch.cuda.current_stream()
            for _ in range(5):
                st.attn(stream)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in steps:
        st.out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for st, want in zip(steps, wants):
        assert int(st.status[0]) == 0 and torch.equal(bits(st.out), bits(want))


def test_the_longest_rows_of_a_batch_merge_alike():
    # one long and many short sequences: splits that a short one does not have
    # are neither written nor read
    w = workload(wl.small_variant(5, batch=6, hq=8, hkv=2, prefix=(1, 9000), tree="random:1,8,4", vocab=64, seed=77))
    w.prefix_len[0], w.prefix_len[1] = 1, 0
    a = DeviceKv4Step(w)
    a.attn_workspace.fill_(255)                          # NaN wherever nothing is written
    a.mask()
    a.attn()
    torch.cuda.synchronize()
    check_attn(w, a, True)


@pytest.mark.parametrize("G,nodes", [(2, 4), (4, 9), (65, 2)])
def test_blocks_beyond_32_bit_offsets(G, nodes):
    # the sequences' pages sit at the end of a pool of more than 2^32 bytes of K and of V
    w = workload(wl.small_variant(5, batch=2, hq=8 * G, hkv=8, prefix=(100, 300), tree=f"random:{nodes},{nodes},4",
                                  vocab=64, seed=G))
    a = run(w)
    b = DeviceKv4Step(w)
    kb, vb = 8 * 1088, 8 * 1040                          # bytes of a page
    old, new = b.desc.num_pages, (1 << 32) // vb + 1000
    k4, v4 = (torch.empty(new * size, dtype=torch.uint8, device="cuda") for size in (kb, vb))
    k4.view(new, kb)[new - old:] = b.k4.view(old, kb)
    v4.view(new, vb)[new - old:] = b.v4.view(old, vb)
    b.k4, b.v4 = k4, v4
    b.page_table = torch.where(b.page_table >= 0, b.page_table + (new - old), b.page_table)
    b.desc.num_pages = new
    b.mask()
    b.attn()
    argmax = torch.zeros(w.total_rows, dtype=torch.int32, device="cuda")
    lens = w.prefix_len.tolist()
    zero = torch.zeros_like(b.prefix_len)
    for st in (a, b):
        st.accept_commit_argmax(argmax)
    rows = [st.read(lens, zero) for st in (a, b)]
    torch.cuda.synchronize()
    assert int(b.status[0]) == 0 and torch.equal(bits(a.out), bits(b.out))
    for x, y in zip(*rows):
        assert torch.equal(bits(x), bits(y))
    assert torch.equal(a.k4.view(old, kb), k4.view(new, kb)[new - old:])
    assert torch.equal(a.v4.view(old, vb), v4.view(new, vb)[new - old:])
