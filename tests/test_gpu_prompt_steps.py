"""A serving loop's run of calls: prompts into the cache, attention over them,
verify steps on the same cache with steered logits, and the counts that the
steering goes by (GPU)."""
import numpy as np
import pytest
import torch

import oracle
import speculative_decoding_tree_gb300 as tv
from gpu_helpers import check_step, workload
from oracle import logits as ol, prompt as op
from prompt_helpers import reference
from speculative_decoding_tree_gb300 import runner, workloads as wl

pytestmark = pytest.mark.gpu


def spec(dtype, paged, d=128):
    return wl.small_variant(5, batch=3, hq=4, hkv=2, d=d, dtype=dtype, prefix=(20, 190), tree="random:3,17,5", vocab=501,
                            paged=paged, seed=31)


def rows_of(n, st, seed):
    g = torch.Generator().manual_seed(seed)
    h, kv, d = st.desc.num_q_heads, st.desc.num_kv_heads, st.desc.head_dim
    return [torch.randn(n, x, d, generator=g).to(st.q.dtype).cuda() for x in (h, kv, kv)]


def cached(st, b, n):
    """K and V of positions 0 .. n - 1, [Hkv, n, d] float64."""
    out = []
    for x in (st.k_cache, st.v_cache):
        if st.page_table is None:
            out.append(x[b, :, :n])
        else:
            out.append(x[st.page_table[b].long()].transpose(0, 1).flatten(1, 2)[:, :n])
    return [x.double().cpu().numpy() for x in out]


def check_prompt(st, pr, past, q, k, v):
    """The chunk's rows: turned queries attend to the cache before it and to its own rows."""
    torch.cuda.synchronize()
    got = pr.out.double().cpu().numpy()
    offs = pr.offsets.tolist()
    bf16 = st.q.dtype == torch.bfloat16
    for b, p in enumerate(past):
        sl = slice(offs[b], offs[b + 1])
        if sl.start == sl.stop:
            continue
        kp, vp = cached(st, b, p)
        ref, lim = reference(pr.q[sl].double().cpu().numpy(), kp, vp, pr.k_rows[:, sl].double().cpu().numpy(),
                             pr.v_rows[:, sl].double().cpu().numpy(), st.desc.head_dim ** -0.5, bf16, not bf16)
        assert (np.abs(got[sl] - ref) <= lim).all()
        n = sl.stop - sl.start
        kc, vc = cached(st, b, p + n)
        assert np.array_equal(kc[:, p:], pr.k_rows[:, sl].double().cpu().numpy())
        assert np.array_equal(vc[:, p:], v[sl].double().cpu().numpy().transpose(1, 0, 2))
        turned = op.rotate(k[sl].double().cpu().numpy(), p + np.arange(n), pr.theta).transpose(1, 0, 2)
        assert np.abs(kc[:, p:] - turned).max() <= (2.0 ** -8 if bf16 else 2.0 ** -20) * np.abs(turned).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("paged,d", [(True, 128), (False, 128), (True, 256), (False, 512)])
def test_prompt_then_steered_steps(paged, d, dtype):
    w = workload(spec(dtype, paged, d))
    st = runner.DeviceStep(w)
    lens = w.prefix_len.tolist()
    st.k_cache.fill_(float("nan"))
    st.v_cache.fill_(float("nan"))
    st.prefix_len.zero_()
    # the prompt in two chunks: the second attends to the first
    first = [n // 3 for n in lens]
    for i, (past, chunk) in enumerate((([0] * 3, first), (first, [n - f for n, f in zip(lens, first)]))):
        pr = runner.DevicePrompt(st, chunk, max_prefix=max(past))
        q, k, v = rows_of(pr.rows, st, i)
        pr.run(q, k, v)
        check_prompt(st, pr, past, q, k, v)
    assert int(st.status[0]) == 0 and st.prefix_len.tolist() == lens
    # steering: the prompt's tokens and the drafts on a row's path count
    g = torch.Generator().manual_seed(5)
    V, B, R = st.vocab, 3, w.total_rows
    said = torch.randint(0, V, (sum(lens),), generator=g).to(torch.int32)
    pen = torch.tensor([[1.3, 0.2, 0.1], [0.8, 0.0, 0.4], [1.0, 0.5, 0.0]])
    bo = torch.tensor([0, 3, 3, 5], dtype=torch.int32)
    bt, bv = torch.tensor([5, 9, 5, 0, 500], dtype=torch.int32), torch.tensor([1.0, -2.0, 4.0, 3.0, -1.0])
    mask = torch.randint(-2 ** 31, 2 ** 31, (R, (V + 31) // 32), generator=g).to(torch.int32)
    ctl = runner.LogitControl(st, pen.cuda(), (bo.cuda(), bt.cuda(), bv.cuda()), mask.cuda())
    offs = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32)
    ctl.read(said.cuda(), offs.cuda())
    counts = [ol.add_counts(np.zeros(V, np.int64), said[offs[b]:offs[b + 1]].tolist(), True) for b in range(B)]
    st.mask()
    raw = st.logits.clone()
    ctl.process()
    torch.cuda.synchronize()
    got = st.logits.double().cpu().numpy()
    half = 2.0 ** -8 if st.logits.dtype == torch.bfloat16 else 2.0 ** -24
    for b in range(B):
        o0, o1 = w.seq_rows(b)
        bias = (bt[bo[b]:bo[b + 1]].tolist(), bv[bo[b]:bo[b + 1]].tolist())
        for i in range(o1 - o0):
            path = ol.path_drafts(w.parents[b], w.draft_tokens[o0:o1], i)
            want = ol.process_row(raw[o0 + i].double().cpu().numpy(), counts[b], pen[b].tolist(), bias,
                                  mask[o0 + i].numpy().view(np.uint32), path)
            fin = np.isfinite(want)
            assert np.array_equal(fin, np.isfinite(got[o0 + i]))
            assert (np.abs(got[o0 + i][fin] - want[fin]) <= half * np.abs(want[fin]) + 2.0 ** -19).all()
    # the verify step on that cache and those logits
    w.k_cache, w.v_cache, w.logits = st.k_cache.cpu(), st.v_cache.cpu(), st.logits.cpu()
    ref = oracle.verify_step(w)
    st.attn()
    st.accept_commit()
    ctl.emitted()
    torch.cuda.synchronize()
    check_step(w, st, ref)
    for b, (k, _, tokens) in enumerate(ref["accepted"]):
        want = ol.add_counts(counts[b], tokens, False)
        assert np.array_equal(ctl.counts[b, :V].cpu().numpy().view(np.uint16).astype(np.int64), want)


def test_a_chunk_is_a_chain_of_tree_rows():
    """The prompt attention of 60 rows equals the verify attention of a chain, within both kernels' roundings."""
    w = workload(wl.small_variant(5, batch=1, hq=4, hkv=2, d=128, prefix=(300, 300), tree="chain:60", vocab=64,
                                  paged=True, seed=3))
    st = runner.DeviceStep(w)
    st.mask()
    st.attn()
    pr = runner.DevicePrompt(st, [60], max_prefix=300)
    pr.q.copy_(st.q)
    pr.k_rows.copy_(st.k_tree)
    pr.v_rows.copy_(st.v_tree)
    pr.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    # two kernels' weights and results rounded to bf16 (2^-8 each), of values whose weighted magnitudes are below 4
    assert float((pr.out.float() - st.out.float()).abs().max()) <= 4 * 2.0 ** -8 * 4


def test_prompt_into_the_4_bit_cache():
    """A prompt without a prefix needs no cache of the plain kind: the same rows go to the 4-bit append."""
    w = workload(wl.small_variant(5, batch=2, hq=4, hkv=2, d=128, prefix=(40, 90), tree="random:3,9,4", vocab=64,
                                  paged=True, seed=4))
    st = runner.DeviceKv4Step(w)
    st.prefix_len.zero_()
    lens = w.prefix_len.tolist()
    offs = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32).cuda()
    R = sum(lens)
    q, k, v = rows_of(R, st, 9)
    desc = tv.make_desc(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=128, dtype=tv.BF16, max_nodes=1, total_rows=2,
                        capacity=st.desc.capacity, max_prefix=0, page_size=16, num_pages=st.desc.num_pages)
    kr, vr = (torch.empty(2, R, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tv.tv_prompt_rope_store(desc, R, max(lens), 1e4, q, k, v, st.prefix_len, offs, q, kr, vr, None, None, None, None,
                            st.status)
    out = torch.empty_like(q)
    n = tv.tv_prompt_workspace_size(desc, R, max(lens))
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    tv.tv_prompt_attn(desc, R, max(lens), q, None, None, None, st.prefix_len, offs, kr, vr, out, ws, n, st.status)
    tv.tv_kv4_append(st.desc, R, max(lens), kr, vr, offs, st.prefix_len, st.k4, st.v4, st.page_table, st.status)
    st.prefix_len.copy_(torch.tensor(lens, dtype=torch.int32))
    st.mask()
    st.attn()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0 and torch.isfinite(out).all() and torch.isfinite(st.out).all()
    for b in range(2):
        sl = slice(*offs[b:b + 2].tolist())
        f = lambda x: x.double().cpu().numpy()
        ref, lim = reference(f(q[sl]), np.zeros((2, 0, 128)), np.zeros((2, 0, 128)), f(kr[:, sl]), f(vr[:, sl]),
                             128 ** -0.5, True, False)
        assert (np.abs(f(out[sl]) - ref) <= lim).all()


def test_captured_loop():
    """Chunk, steering and step in one graph, replayed on new inputs."""
    w = workload(spec("bf16", True))
    st = runner.DeviceStep(w)
    st.prefix_len.zero_()
    lens = [n // 2 for n in w.prefix_len.tolist()]
    pr = runner.DevicePrompt(st, lens)
    q, k, v = rows_of(pr.rows, st, 1)
    ctl = runner.LogitControl(st, torch.tensor([[1.2, 0.1, 0.1]] * 3).cuda())
    logits = st.logits.clone()

    def loop():
        st.prefix_len.zero_()
        st.logits.copy_(logits)
        ctl.counts.zero_()
        pr.run(q, k, v)
        st.mask()
        ctl.process()
        st.attn()
        st.accept_commit()
        ctl.emitted()

    loop()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        loop()
    q2, k2, v2 = rows_of(pr.rows, st, 2)
    for a, b in ((q, q2), (k, k2), (v, v2)):
        a.copy_(b)
    loop()
    torch.cuda.synchronize()
    want = [x.clone() for x in (pr.out, st.out, st.tokens, st.prefix_len, ctl.counts, st.logits)]
    for x in (pr.out, st.out):
        x.zero_()
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    for x, y in zip(want, (pr.out, st.out, st.tokens, st.prefix_len, ctl.counts, st.logits)):
        assert torch.equal(x, y)


def test_command():
    assert runner.main(["--config", "1", "--steps", "2", "--prompt", "20", "--steer"]) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_beyond_32_bit_offsets(dtype):
    """The sequence's pages lie behind 2^31 values of a pool."""
    pages, hkv, d, P, n = 140000, 8, 128, 100, 60
    k_cache, v_cache = (torch.empty(pages, hkv, 16, d, dtype=dtype, device="cuda") for _ in range(2))
    assert k_cache.numel() > 2 ** 31
    table = torch.arange(pages - 1, pages - 12, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    past = [torch.randn(hkv, 112, d, generator=torch.Generator().manual_seed(i)).to(dtype).cuda() for i in range(2)]
    for x, y in ((k_cache, past[0]), (v_cache, past[1])):
        x[table[0, :7].long()] = y.reshape(hkv, 7, 16, d).transpose(0, 1)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(n, h, d, generator=g).to(dtype).cuda() for h in (hkv, hkv, hkv))
    i32 = dict(dtype=torch.int32, device="cuda")
    prefix, offs, new, status = torch.tensor([P], **i32), torch.tensor([0, n], **i32), torch.zeros(1, **i32), torch.zeros(4, **i32)
    desc = tv.make_desc(batch=1, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, max_nodes=1, total_rows=1, capacity=176,
                        dtype=tv.BF16 if dtype == torch.bfloat16 else tv.F32, max_prefix=P, page_size=16, num_pages=pages)
    kr, vr = (torch.empty(hkv, n, d, dtype=dtype, device="cuda") for _ in range(2))
    tv.tv_prompt_rope_store(desc, n, n, 1e4, q, k, v, prefix, offs, q, kr, vr, k_cache, v_cache, table, new, status)
    out = torch.empty_like(q)
    size = tv.tv_prompt_workspace_size(desc, n, n)
    ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    tv.tv_prompt_attn(desc, n, n, q, k_cache, v_cache, table, prefix, offs, kr, vr, out, ws, size, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0 and int(new[0]) == P + n
    for x, rows in ((k_cache, kr), (v_cache, vr)):
        assert torch.equal(x[table[0].long()].transpose(0, 1).flatten(1, 2)[:, P:P + n], rows)
    f = lambda x: x.double().cpu().numpy()
    bf16 = dtype == torch.bfloat16
    ref, lim = reference(f(q), f(past[0][:, :P]), f(past[1][:, :P]), f(kr), f(vr), d ** -0.5, bf16, not bf16)
    assert (np.abs(f(out) - ref) <= lim).all()
