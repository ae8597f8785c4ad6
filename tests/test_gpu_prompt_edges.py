"""Prompts and the control of logits at their edges: no rows, infinities, roots
(GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from gpu_helpers import workload
from oracle import logits as ol
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
