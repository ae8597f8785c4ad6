"""Prompts and the control of logits at their edges: no rows, infinities, roots
(GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from gpu_helpers import workload
from oracle import logits as ol, prompt as op
from prompt_helpers import Prompts, reference
from speculative_decoding_tree_gb300 import runner, workloads as wl

pytestmark = pytest.mark.gpu


def tree_step(**kw):
    base = dict(batch=3, hq=4, hkv=2, d=128, dtype="bf16", prefix=(20, 190), tree="random:3,17,5", vocab=501, seed=31)
    w = workload(wl.small_variant(5, **{**base, **kw}))
    return w, runner.DeviceStep(w)


def test_empty_prompts_leave_the_lengths():
    w, st = tree_step(paged=True)
    pr = runner.DevicePrompt(st, [0, 0, 0])
    pr.new_prefix.fill_(-77)
    none = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    pr.run(none, none[:, :2], none[:, :2])
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0 and st.prefix_len.tolist() == w.prefix_len.tolist()


@pytest.mark.parametrize("side", [False, True])
def test_a_trees_first_row_is_steered_like_plain_decoding(side):
    """A sequence's first root, counted by started(), weighs on every row as any emitted token does."""
    w, st = tree_step()
    V = st.vocab
    ctl = runner.LogitControl(st, torch.tensor([[1.3, 0.2, 0.1]] * 3).cuda())
    stream = None
    if side:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
    ctl.started(stream)
    if side:
        torch.cuda.current_stream().wait_stream(stream)
    st.mask()
    raw = st.logits.double().cpu().numpy()
    ctl.process()
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    half = 2.0 ** -8 if st.logits.dtype == torch.bfloat16 else 2.0 ** -24
    for b in range(3):
        o0, o1 = w.seq_rows(b)
        said = ol.add_counts(np.zeros(V, np.int64), [int(w.draft_tokens[o0])], False)
        assert np.array_equal(ctl.counts[b, :V].cpu().numpy(), said)
        for i in range(o1 - o0):
            path = ol.path_drafts(w.parents[b], w.draft_tokens[o0:o1], i)
            want = ol.process_row(raw[o0 + i], said, (1.3, 0.2, 0.1), None, None, path)
            got = st.logits[o0 + i].double().cpu().numpy()
            # five fp32 roundings of values below 2^5, then the type's half step
            assert (np.abs(got - want) <= half * np.abs(want) + 5 * 2.0 ** -19).all()


def busy():
    """Allocations of every small size on the current stream, filled: memory that was given back is written again."""
    keep = [torch.full((n,), 2 ** 30 + 7, dtype=torch.int32, device="cuda") for n in [5] * 64 + [128] * 64]
    return keep + [torch.full((60, h, 128), 9.0, dtype=torch.bfloat16, device="cuda") for h in [4] * 16 + [2] * 16]


@pytest.mark.parametrize("kind", ["stream", "address"])
def test_chunks_on_a_side_stream(kind):
    """Prompts, their rows and their tokens are let go of while the stream has yet to read them."""
    lens = [20, 31, 9]

    def chunk(st, ctl, arg):
        g = torch.Generator("cuda").manual_seed(4)
        rows = [torch.randn(60, h, 128, generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2)]
        said = torch.randint(0, st.vocab, (60,), generator=g, device="cuda").int()
        offs = torch.tensor([0, 20, 51, 60], dtype=torch.int32, device="cuda")
        pr = runner.DevicePrompt(st, lens, max_prefix=0)
        if arg is not None:
            side.wait_stream(torch.cuda.current_stream())
        pr.run(*rows, arg)
        ctl.read(said, offs, arg)
        return pr.out

    results = []
    side = torch.cuda.Stream()
    for arg in (None, side if kind == "stream" else side.cuda_stream):
        w, st = tree_step(paged=True)
        ctl = runner.LogitControl(st, torch.ones(3, 3, device="cuda"))
        st.prefix_len.zero_()
        torch.cuda.synchronize()
        if arg is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)            # the calls run well after they were made
        out = chunk(st, ctl, arg)
        keep = busy()
        torch.cuda.synchronize()
        assert int(st.status[0]) == 0 and st.prefix_len.tolist() == lens
        caches = [torch.cat([x[st.page_table[b].long()].transpose(0, 1).flatten(1, 2)[:, :n] for b, n in enumerate(lens)], 1)
                  for x in (st.k_cache, st.v_cache)]
        results.append([out.clone(), ctl.counts.clone(), *caches])
        del keep
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 2, 1), (512, 2, 1)])
def test_a_score_of_minus_infinity_has_no_weight(d, hq, hkv):
    """bf16: a key of -inf against queries above 0 is seen and weighs nothing, in the prefix and among the rows."""
    c = Prompts([150], [200], hq, hkv, d, "bf16", seed=12)
    c.q.abs_()
    c.q[c.q == 0] = 1
    inf = float("-inf")
    c.k_rows[:, 60] = c.k_rows[:, 130] = inf
    c.past[0][0][:, 7] = inf
    c.k_cache[0, :, 7] = inf
    for x, y in zip(c.gpu, (c.q, c.k_rows, c.v_rows)):
        x.copy_(y)
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0
    q, kp, vp, kr, vr = c.seq(0)
    got = c.out.double().cpu().numpy()
    gone = [60, 130]
    for a, b in ((0, 60), (60, 130), (130, 200)):            # rows a .. b - 1 see the same rows of -inf
        keep = np.array([i for i in range(b) if i not in gone])
        live = np.array([i for i in range(a, b) if i not in gone])
        rows = np.concatenate([np.searchsorted(keep, live)])
        ref, lim = reference(q[keep], np.delete(kp, 7, 1), np.delete(vp, 7, 1), kr[:, keep], vr[:, keep], c.scale, True, False)
        assert (np.abs(got[live] - ref[rows]) <= lim[rows]).all()
    # the rows of -inf themselves see the others
    for i in gone:
        keep = np.array([j for j in range(i) if j not in gone])
        one = op.attention(q[i:i + 1], np.concatenate([np.delete(kp, 7, 1), kr[:, keep[:-1]]], 1),
                           np.concatenate([np.delete(vp, 7, 1), vr[:, keep[:-1]]], 1), kr[:, keep[-1:]], vr[:, keep[-1:]], c.scale)
        assert np.abs(got[i] - one[0]).max() <= 3 * 2.0 ** -8 * np.abs(vr).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 2, 1), (512, 2, 1)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_infinite_keys_of_later_rows(d, hq, hkv, dtype, bad):
    c = Prompts([30], [200], hq, hkv, d, dtype, seed=13)
    c.k_rows[:, 150:] = bad
    c.gpu[1].copy_(c.k_rows)
    c.attn()
    torch.cuda.synchronize()
    q, kp, vp, kr, vr = c.seq(0)
    ref, lim = reference(q[:150], kp, vp, kr[:, :150], vr[:, :150], c.scale, c.bf16, c.out_f32)
    assert (np.abs(c.out[:150].double().cpu().numpy() - ref) <= lim).all()


def steer(x, counts=None, pen=None, bias=None, mask=None, nodes=None):
    """One sequence of rows without drafts on their paths, through the library."""
    R, V = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    T = 0 if bias is None else len(bias[0])
    desc = tv.make_logits_desc(batch=1, vocab=V, max_nodes=R, total_rows=R, biases=T,
                               logits_dtype=tv.BF16 if x.dtype == torch.bfloat16 else tv.F32)
    to = lambda t: None if t is None else t.cuda()
    bo = bt = bv = None
    if T:
        bo, bt, bv = torch.tensor([0, T], **i32), torch.tensor(bias[0], **i32), torch.tensor(bias[1], device="cuda")
    out, status = torch.full_like(x, 5.0).cuda(), torch.zeros(4, **i32)
    keep = [to(x), to(counts), to(pen), to(mask)]
    tv.tv_tree_logits_process(desc, keep[0], keep[1], keep[2], bo, bt, bv, keep[3], None, torch.tensor([0, R], **i32), None,
                              out, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    return out.cpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [64, 4099, 8200])
def test_logits_that_nothing_touches_keep_their_bits(V, dtype):
    """Only counted, biased and masked tokens change; every other one is the input, bit for bit."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(9, V, generator=g) * 3).to(dtype)
    x[0, 1], x[1, 2], x[2, 0], x[3, 4] = float("nan"), float("inf"), float("-inf"), -0.0
    bits = lambda t: t.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
    assert torch.equal(bits(steer(x)), bits(x))
    counts = torch.zeros(1, (V + 7) // 8 * 8, dtype=torch.int16)
    counts[0, 7], counts[0, V - 1] = 3, -32768
    pen = torch.tensor([[1.5, 0.25, 0.5]])
    mask = torch.full((9, (V + 31) // 32), -1, dtype=torch.int32)
    mask[:, 1] = ~(1 << 5)                                   # token 37
    got = steer(x, counts, pen, ([11, 12], [2.0, -1.0]), mask)
    touched = torch.zeros(V, dtype=torch.bool)
    touched[torch.tensor([7, 11, 12, 37, V - 1])] = True
    assert torch.equal(bits(got)[:, ~touched], bits(x)[:, ~touched])
    assert (got[:, 37] == float("-inf")).all() and not torch.equal(got[:, 7], x[:, 7])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinities_and_nan_of_touched_logits(dtype):
    """NaN and +inf stay through penalties and biases, -inf too; forbidden ones become -inf whatever they are."""
    x = torch.zeros(4, 96, dtype=dtype)
    x[0, :], x[1, :], x[2, :], x[3, :] = float("nan"), float("inf"), float("-inf"), 2.0
    counts = torch.zeros(1, 96, dtype=torch.int16)
    counts[0, :32] = 2
    mask = torch.tensor([[-1, -1, 0]] * 4, dtype=torch.int32)
    got = steer(x, counts, torch.tensor([[2.0, 0.25, 0.5]]), (list(range(16, 48)), [1.0] * 32), mask).float()
    assert torch.isnan(got[0, :64]).all() and (got[1, :64] == float("inf")).all()
    assert (got[2] == float("-inf")).all() and (got[:, 64:] == float("-inf")).all()
    assert got[3, :64].tolist() == [0.0] * 16 + [1.0] * 16 + [3.0] * 16 + [2.0] * 16


def test_a_length_beyond_its_type_is_reported():
    """Rows up to position 2^31 + 19 are rotated (no cache); the new length does not fit and stays."""
    from test_gpu_prompt_rope import Rows
    c = Rows([2 ** 31 - 100, 5], [120, 3], 2, 1, 128, "f32", cache=False, cap=2 ** 31 - 16, seed=2)
    c.run(1e4)
    assert int(c.status[0]) == 16 and c.new.tolist() == [2 ** 31 - 100, 8]
    want = op.rotate(c.q.double().cpu().numpy(), op.positions(c.p, c.offs), 1e4)
    # the fraction of a turn a position times is off by at most 2^-52 relative: 2^31 * 0.16 * 2^-52 turns
    assert np.abs(c.q_out.double().cpu().numpy() - want).max() < 5e-6


@pytest.mark.parametrize("p,n", [(0, 140), (2000, 3)])
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 2, 1), (512, 2, 1)])
def test_rows_of_minus_infinity_alone_are_zeros(d, hq, hkv, p, n):
    """bf16, one key chunk and several: the rows before row 2 see scores of -inf alone."""
    c = Prompts([p], [n], hq, hkv, d, "bf16", seed=14)
    assert (c.plan()["num_splits"] > 1) == (p > 0)
    c.gpu[0].fill_(1.0)
    c.gpu[1][:, :2] = float("-inf")
    c.k_cache[:, :, :p] = float("-inf")
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0 and (c.out[:2] == 0).all()
    # row 2 sees one key besides: its value, weight 1, rounded to bf16 from the product with 1 / 1
    assert torch.equal(c.out[2], c.gpu[2][:, 2].repeat_interleave(hq // hkv, 0))


@pytest.mark.parametrize("d", [128, 256, 512])
def test_wide_groups_of_bf16_heads(d):
    """More than 128 query heads a KV head: bf16 on the kernel of three parts, paged, behind a prefix, split and not."""
    for p, n in (([300, 0, 17], [9, 20, 1]), ([0] * 4, [160] * 4)):
        c = Prompts(p, n, 130, 1, d, "bf16", paged=True, pad=2, seed=15)
        assert c.plan()["kernel"] == 8
        c.attn()
        c.check()


@pytest.mark.parametrize("args", [("--kv4", "--steer"), ("--window", "512,4", "--steer"), ("--sampled", "0.7", "--steer"),
                                  ("--attn-only", "--steer"), ("--prompt", "70")])
def test_command_forms(args):
    assert runner.main(["--config", "3", "--steps", "2", *args]) == 0


def test_command_steers_before_the_4_bit_step_accepts(monkeypatch):
    """The argmax that the 4-bit step walks on is that of the logits as steered once."""
    seen = []

    class Step(runner.DeviceKv4Step):
        def step(self, argmax, stream=None):
            seen.append((argmax.clone(), self.logits.clone()))
            super().step(argmax, stream)

    monkeypatch.setattr(runner, "DeviceKv4Step", Step)
    assert runner.main(["--config", "3", "--steps", "2", "--kv4", "--steer"]) == 0
    w = wl.make_workload(wl.CONFIGS[3], canary=0.0, argmax_fn=lambda x: torch.argmax(x.float(), dim=1))
    st = Step(w)
    ctl = runner.LogitControl(st, torch.tensor([[1.1, 0.1, 0.1]] * st.desc.batch, device="cuda"))
    ctl.started()
    raw = st.logits.clone()
    for argmax, logits in seen:
        st.logits.copy_(raw)
        st.mask()
        ctl.process()
        assert torch.equal(logits, st.logits) and not torch.equal(logits, raw)
        assert torch.equal(argmax, st.logits.float().argmax(1).to(torch.int32))
        st.accept_commit_argmax(argmax)
        ctl.emitted()
