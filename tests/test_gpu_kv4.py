"""The 4-bit cache on the GPU vs the oracle: writes and reads bit for bit, the
commit of an accepted path, and the attention within the bounds that
kv4_helpers.reference derives."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_gb300 as tv
from oracle import kv4
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step
from gpu_helpers import workload
from kv4_helpers import bits, blocks_of, check_attn

pytestmark = pytest.mark.gpu


def step(w, win=None, **kw):
    st = DeviceKv4Step(w, win, **kw)
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    return st


def spec(n=5, **kw):
    kw.setdefault("vocab", 64)
    return wl.small_variant(n, **kw)


# ------------------------------------------------------------------ writes and reads

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("paged", [False, True])
def test_append_bytes_equal_the_oracle(dtype, d, paged):
    w = workload(spec(5, batch=3, hq=4, hkv=2, d=d, dtype=dtype, prefix=(1, 60), paged=paged, seed=d))
    st = DeviceKv4Step(w)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    for b in range(3):
        P = int(w.prefix_len[b])
        kp, vp = oracle.prefix_kv(w, b)
        kb, vb = blocks_of(st, b)
        for g in range(2):
            for n in range(-(-P // 16)):
                rows = min(16, P - 16 * n)
                full = [np.zeros((16, d)), np.zeros((16, d))]
                full[0][:rows], full[1][:rows] = kp[g, 16 * n:16 * n + rows], vp[g, 16 * n:16 * n + rows]
                wk, wv = kv4.pack_block(*full)
                # a position that was not written keeps its bytes (zeros): compare the written ones
                gk, gv = kb[g, n].numpy(), vb[g, n].numpy()
                assert (gk[:8 * d].reshape(-1, 16, 16)[:, :rows] == wk[:8 * d].reshape(-1, 16, 16)[:, :rows]).all()
                assert (gk[8 * d:].reshape(-1, 16)[:, :rows] == wk[8 * d:].reshape(-1, 16)[:, :rows]).all()
                assert (gk[:8 * d].reshape(-1, 16, 16)[:, rows:] == 0).all()
                nib = lambda x: kv4_nibbles(x[:8 * d].reshape(d, 8))
                assert (nib(gv)[:, :rows] == nib(wv)[:, :rows]).all() and (nib(gv)[:, rows:] == 0).all()
                assert (gv[8 * d:8 * d + rows] == wv[8 * d:8 * d + rows]).all() and (gv[8 * d + rows:] == 0).all()


def kv4_nibbles(b):
    """[d, 8] V bytes -> [d, 16] codes by position."""
    w = b.astype(np.uint64).reshape(-1, 2, 4)
    word = (w * (1 << (8 * np.arange(4, dtype=np.uint64)))).sum(-1)
    e = np.arange(8)
    return ((word[..., None] >> (4 * (e // 2) + 16 * (e % 2)).astype(np.uint64)) & 15).reshape(-1, 16)


@pytest.mark.parametrize("first,more", [(5, 1), (15, 2), (16, 16), (3, 30), (40, 9)])
def test_append_in_pieces_equals_append_at_once(first, more):
    w = workload(spec(3, prefix=(first + more, first + more), paged=False))
    whole = DeviceKv4Step(w)
    parts = DeviceKv4Step(w)
    rows = [x[:, :, :first + more].squeeze(0) for x in (w.k_cache.cuda(), w.v_cache.cuda())]
    parts.k4.fill_(0)
    parts.v4.fill_(0)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    parts.append(rows[0][:, :first].contiguous(), rows[1][:, :first].contiguous(), [first], zero)
    parts.append(rows[0][:, first:].contiguous(), rows[1][:, first:].contiguous(), [more], zero + first)
    torch.cuda.synchronize()
    assert torch.equal(whole.k4, parts.k4) and torch.equal(whole.v4, parts.v4)
    # one row over: only that position changes
    before = [x.clone() for x in parts.read([first + more], zero)]
    one = [torch.full_like(r[:, :1], 3.0) for r in rows]
    parts.append(*one, [1], zero + first - 1)
    after = parts.read([first + more], zero)
    three = float(kv4.stored(np.full((1, 32), 3.0), 1)[0, 0])      # what a group of equal 3.0 is read as
    for x, y in zip(before, after):
        x[:, first - 1] = three
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_values_read_back(dtype, d):
    g = torch.Generator().manual_seed(d)
    T = 77
    k = torch.randn(2, T, d, generator=g) * torch.logspace(-6, 6, T)[None, :, None]
    v = torch.randn(2, T, d, generator=g) * 10
    k[0, 0] = 0
    k[0, 1, 3] = float("nan")
    v[1, 2, 5] = float("inf")
    v[0, 3, 7] = float("nan")
    k[1, 4] = -float("inf")
    k[0, 5], v[0, 5] = 1e30, -1e30
    k[1, 6], v[1, 6] = 1e-30, 1e-40
    k[0, 7, :16] = torch.arange(16) * 0.5                # ties on a grid of one
    k[0, 7, 16] = 7.0
    v[0, 8] = (torch.arange(d) % 29) * 0.25 - 3.5
    v[0, 8, 0] = 7.0
    k, v = k.to(dtype), v.to(dtype)
    w = workload(spec(3, hq=2, hkv=2, d=d, dtype="bf16" if dtype == torch.bfloat16 else "f32", prefix=(T, T)))
    st = DeviceKv4Step(w)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    st.append(k.cuda(), v.cuda(), [T], zero)
    gk, gv = st.read([T], zero)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    assert np.array_equal(gk.double().cpu().numpy(), kv4.stored(k, d // 32))
    assert np.array_equal(gv.double().cpu().numpy(), kv4.stored(v, 1))


def test_append_skips_what_does_not_fit():
    w = workload(spec(5, batch=3, hq=4, hkv=2, prefix=(20, 40), seed=6))
    n = 5
    cases = [("start", [-1, 0, 0], 4), ("start", [10 ** 6, 0, 0], 16), ("page", None, 8), ("offsets", None, 2)]
    for what, start, bit in cases:
        st = DeviceKv4Step(w)
        k4 = st.k4.clone()
        k = torch.randn(2, 3 * n, 128, device="cuda").to(torch.bfloat16)
        offs = torch.tensor([0, n, 2 * n, 3 * n], dtype=torch.int32, device="cuda")
        table = st.page_table.clone()
        s = torch.tensor(start or [0, 0, 0], dtype=torch.int32, device="cuda")
        if what == "page":
            table[0, 0] = st.desc.num_pages
        if what == "offsets":
            offs[1] = -3                                 # sequence 0 ends before it starts; 1 starts below 0
        tv.tv_kv4_append(st.desc, 3 * n, n, k, k, offs, s, st.k4, st.v4, table, st.status)
        torch.cuda.synchronize()
        assert int(st.status[0]) == bit, what
        changed = [not torch.equal(a, b) for a, b in zip(
            (blocks_of(st, b)[0] for b in range(3)),
            (k4.view(-1, 2, 8 * 128 + 64)[st.page_table[b].long().clamp(min=0)][st.page_table[b] >= 0].transpose(0, 1).cpu()
             for b in range(3)))]
        assert changed == ([False, True, True] if what != "offsets" else [False, False, True]), what


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("n", [1, 2, 3, 4, 5])
def test_small_variant(n):
    w = workload(spec(n))
    check_attn(w, step(w), True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("nodes", [1, 2, 17, 64])
def test_types_heads_and_trees(dtype, d, nodes):
    w = workload(spec(4, d=d, dtype=dtype, prefix=(300, 300), tree=f"random:{nodes},{nodes},9", seed=d + nodes))
    check_attn(w, step(w), True)


@pytest.mark.parametrize("P", [0, 1, 15, 16, 17, 127, 128, 129, 255, 1000])
@pytest.mark.parametrize("nodes", [1, 13])
def test_ragged_prefixes(P, nodes):
    w = workload(spec(3, prefix=(P, P), tree=f"random:{nodes},{nodes},5", seed=70 + P))
    check_attn(w, step(w), True)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (16, 1, 128), (10, 2, 128), (6, 2, 256), (1, 1, 512), (66, 1, 128),
                                      (128, 1, 128), (200, 1, 256)])
@pytest.mark.parametrize("paged", [False, True])
def test_head_shapes(hq, hkv, d, paged):
    w = workload(spec(5, batch=3, hq=hq, hkv=hkv, d=d, prefix=(0, 200), tree="random:1,3,3", paged=paged,
                      seed=hq + d))
    check_attn(w, step(w), True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_batch_with_many_chunks(dtype):
    w = workload(spec(5, batch=2, hq=4, hkv=2, prefix=(3900, 4500), tree="random:3,9,3", dtype=dtype, seed=11))
    st = step(w)
    assert tv.tv_kv4_attn_plan(st.desc)["num_splits"] > 1
    check_attn(w, st, True)


@pytest.mark.parametrize("dtype,d,nodes", [("bf16", 128, 20), ("f32", 256, 20), ("bf16", 512, 1), ("bf16", 256, 64)])
@pytest.mark.parametrize("win", [(1, 0), (1, 300), (2, 1), (5, 16), (16, 4), (100, 4), (130, 130), (10 ** 6, 0)])
def test_windows(dtype, d, nodes, win):
    w = workload(spec(5, batch=2, hq=4, hkv=2, d=d, dtype=dtype, prefix=(280, 700), seed=sum(win) % 97 + d,
                      tree=f"random:{nodes},{nodes},9"))
    check_attn(w, step(w, win), True, win)


def test_large_scores_and_scales():
    # scores of some hundreds: one key takes nearly all weight, and the running maximum moves often
    w = workload(spec(5, batch=2, hq=8, hkv=2, prefix=(300, 900), tree="random:4,20,4", seed=5))
    w.q.mul_(30)
    w.k_cache.mul_(torch.linspace(0.2, 3, w.k_cache.shape[0])[:, None, None, None].to(w.k_cache.dtype))
    check_attn(w, step(w), True)
    w.q.zero_()
    check_attn(w, step(w), True)


def test_bytes_behind_the_prefix_do_not_matter():
    w = workload(spec(5, batch=3, prefix=(10, 300), seed=8))
    a = step(w)
    b = DeviceKv4Step(w)
    for i in range(3):
        P = int(w.prefix_len[i])
        n = int((b.page_table[i] >= 0).sum()) * 16 - P
        junk = torch.full((w.spec.hkv, n, w.spec.d), float("inf"), dtype=torch.bfloat16, device="cuda")
        st = torch.tensor([P if j == i else 0 for j in range(3)], dtype=torch.int32, device="cuda")
        b.append(junk, junk, [n if j == i else 0 for j in range(3)], st)
    b.mask()
    b.attn()
    torch.cuda.synchronize()
    assert torch.equal(bits(a.out), bits(b.out))


def test_unseen_pages_may_hold_any_id():
    w = workload(spec(5, batch=2, prefix=(700, 800), tree="random:5,9,4", seed=12))
    win = (100, 20)
    a = step(w, win)
    b = DeviceKv4Step(w, win)
    b.page_table[:, 3:30] = -7                           # positions 48..479: no sink, below every window
    b.mask()
    b.attn()
    torch.cuda.synchronize()
    assert int(b.status[0]) == 0 and torch.equal(bits(a.out), bits(b.out))


def test_status_bits():
    w = workload(spec(5, batch=3, prefix=(100, 300), seed=4))
    st = step(w)
    st.page_table[1, 2] = st.desc.num_pages
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 8
    st.status.zero_()
    st = step(w)
    st.prefix_len[0] = -4
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 4


def test_repeats_streams_and_graphs_give_the_same_bytes():
    w = workload(spec(5, batch=4, prefix=(40, 2500), seed=21))
    st = step(w)
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
    # a second call in flight on another stream, with its own workspace
    other = step(w)
    for _ in range(5):
        st.attn()
        other.attn(side)
    torch.cuda.synchronize()
    assert torch.equal(bits(st.out), bits(want)) and torch.equal(bits(other.out), bits(want))


# ------------------------------------------------------------------ commit

@pytest.mark.parametrize("n,paged", [(1, False), (3, False), (3, True), (5, True)])
@pytest.mark.parametrize("hkv", [1, 4, 10])
def test_commit_matches_the_oracle(n, paged, hkv):
    w = workload(spec(n, hq=hkv, hkv=hkv, paged=paged, batch=1 if n < 5 else 4, prefix=(30, 30) if n < 5 else (0, 60)))
    st = DeviceKv4Step(w)
    before = [blocks_of(st, b) for b in range(w.batch)]
    am = torch.tensor(oracle.argmax_rows(w.logits), dtype=torch.int32, device="cuda")
    st.accept_commit_argmax(am)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    mn, d = st.desc.max_nodes, w.spec.d
    for b in range(w.batch):
        o0, o1 = w.seq_rows(b)
        k, path, tokens = oracle.accept(w.parents[b], w.draft_tokens[o0:o1].tolist(), am[o0:o1].tolist())
        P = int(w.prefix_len[b])
        assert int(st.accept_len[b]) == k and int(st.prefix_len[b]) == P + k + 1
        assert st.path[b].cpu().tolist() == path + [-1] * (mn - k - 1)
        assert st.tokens[b].cpu().tolist() == tokens + [-1] * (mn - k - 1)
        # the accepted rows, and nothing else, changed
        rows = [x[:, o0 + torch.tensor(path)] for x in (w.k_tree, w.v_tree)]
        want = [kv4.stored(rows[0], d // 32), kv4.stored(rows[1], 1)]
        after = blocks_of(st, b)
        for g in range(hkv):
            for blk in range(before[b][0].shape[1]):
                ob = kv4.unpack_block(before[b][0][g, blk].numpy(), before[b][1][g, blk].numpy(), d)
                ab = kv4.unpack_block(after[0][g, blk].numpy(), after[1][g, blk].numpy(), d)
                for x in range(2):
                    exp = ob[x].copy()
                    for t in range(k + 1):
                        if (P + t) // 16 == blk:
                            exp[(P + t) % 16] = want[x][g, t]
                    assert np.array_equal(ab[x], exp)


def test_commit_failures_leave_everything():
    for what, bit in (("capacity", 16), ("page", 8), ("prefix", 4), ("tree", 1), ("offsets", 2)):
        w = workload(spec(5, batch=3, hq=4, hkv=2, prefix=(30, 60), seed=3))
        st = DeviceKv4Step(w)
        am = torch.tensor(oracle.argmax_rows(w.logits), dtype=torch.int32, device="cuda")
        if what == "capacity":
            st.prefix_len[0] = st.desc.capacity
        if what == "page":
            st.page_table[0, int(w.prefix_len[0]) // 16] = -1
        if what == "prefix":
            st.prefix_len[0] = -1
        if what == "tree":
            st.parents[0] = 0                            # a root with a parent: flagged; the walk goes on
        if what == "offsets":
            st.node_offsets[1] = -2
        k4, v4, pl = st.k4.clone(), st.v4.clone(), st.prefix_len.clone()
        st.accept_commit_argmax(am)
        torch.cuda.synchronize()
        assert int(st.status[0]) == bit, what
        if what == "tree":
            continue
        assert int(st.prefix_len[0]) == int(pl[0]), what
        if what == "offsets":
            assert int(st.accept_len[0]) == -1 and (st.path[0] == -1).all()
        if what in ("capacity", "prefix"):
            st.page_table = st.page_table[:1].contiguous()
            st.desc.batch = 1
            ids = st.page_table[0].long()
            ids = ids[ids >= 0]
            assert torch.equal(st.k4.view(-1, 2, 1088)[ids], k4.view(-1, 2, 1088)[ids])
            assert torch.equal(st.v4.view(-1, 2, 1040)[ids], v4.view(-1, 2, 1040)[ids])


def test_steps_in_a_row():
    # prompt, then verify steps: mask, attention, commit, with the lengths on the device throughout
    w = workload(spec(5, batch=3, hq=8, hkv=2, prefix=(20, 90), seed=31))
    st = DeviceKv4Step(w, max_prefix=w.capacity)
    am = torch.tensor(oracle.argmax_rows(w.logits), dtype=torch.int32, device="cuda")
    acc = [oracle.accept(w.parents[b], w.draft_tokens[slice(*w.seq_rows(b))].tolist(), am[slice(*w.seq_rows(b))].tolist())
           for b in range(3)]
    for it in range(2):
        st.mask()
        st.attn()
        torch.cuda.synchronize()
        check_attn(w, st, True)
        st.accept_commit_argmax(am)
        torch.cuda.synchronize()
        assert int(st.status[0]) == 0
        kc, vc, new = oracle.commit(w, acc)              # the same rows, unrounded: the oracle rounds on reading
        w.k_cache, w.v_cache, w.prefix_len = kc, vc, new
        assert torch.equal(st.prefix_len.cpu(), new)
