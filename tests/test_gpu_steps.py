"""Whole steps over a window and on the 4-bit cache, and the package's command
that runs them (GPU)."""
import pytest
import torch

import oracle
import speculative_decoding_tree_gb300 as tv
from oracle import kv4
from speculative_decoding_tree_gb300 import runner, workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step, DeviceStep, DeviceWindowStep
from gpu_helpers import workload
from kv4_helpers import bits, check_attn

pytestmark = pytest.mark.gpu


def small(**kw):
    return workload(wl.small_variant(5, batch=3, hq=8, hkv=2, prefix=(200, 300), vocab=97, seed=9, **kw))


@pytest.mark.parametrize("win", [None, (50, 4)])
@pytest.mark.parametrize("paged", [False, True])
def test_a_4_bit_step_is_its_three_calls(win, paged):
    w = small(paged=paged)
    argmax = torch.tensor(oracle.argmax_rows(w.logits), dtype=torch.int32, device="cuda")
    st = DeviceKv4Step(w, win)
    st.step(argmax)
    torch.cuda.synchronize()
    check_attn(w, st, True, win)
    one = DeviceKv4Step(w, win)
    one.mask()
    one.attn()
    one.accept_commit_argmax(argmax)
    torch.cuda.synchronize()
    assert int(st.status[0]) == int(one.status[0]) == 0
    assert torch.equal(bits(st.out), bits(one.out)) and torch.equal(st.prefix_len, one.prefix_len)
    assert torch.equal(st.k4, one.k4) and torch.equal(st.v4, one.v4) and torch.equal(st.path, one.path)
    # the accepted rows read back as what the format holds of them
    counts = (st.accept_len + 1).tolist()
    k, v = st.read(counts, w.prefix_len.cuda())
    at = 0
    for b, n in enumerate(counts):
        rows = w.seq_rows(b)[0] + st.path[b, :n].cpu().long()
        for got, src, groups in ((k, w.k_tree, 4), (v, w.v_tree, 1)):
            want = torch.from_numpy(kv4.stored(src[:, rows], groups))
            assert torch.equal(got[:, at:at + n].double().cpu(), want)
        at += n


def test_a_window_step_commits_like_the_full_one():
    w = small()
    full, st = DeviceStep(w), DeviceWindowStep(w, 50, 4)
    full.step()
    st.step()
    torch.cuda.synchronize()
    check_attn(w, st, False, (50, 4))
    assert torch.equal(st.prefix_len, full.prefix_len) and torch.equal(st.tokens, full.tokens)
    assert torch.equal(bits(st.k_cache), bits(full.k_cache)) and torch.equal(bits(st.v_cache), bits(full.v_cache))


def test_launches_of_a_step_follow_its_own_plan():
    # 5000 keys: several chunks in full, one over a window of 60 positions
    w = workload(wl.small_variant(5, batch=2, hq=8, hkv=2, prefix=(5000, 5000), vocab=97, seed=9))
    assert DeviceStep(w).kernels_per_step() == 5
    st = DeviceWindowStep(w, 60, 4)
    assert tv.tv_window_attn_plan(st.desc, st.win)["num_splits"] == 1 and st.kernels_per_step() == 4
    assert DeviceKv4Step(w).kernels_per_step() == 4
    assert DeviceKv4Step(w, (60, 4)).kernels_per_step() == 3


@pytest.mark.parametrize("args", [["--kv4"], ["--window", "100,4"], ["--kv4", "--window", "100,4"], ["--kv4", "--attn-only"]])
def test_the_command_runs_whole_steps(args):
    assert runner.main(["--config", "2", "--steps", "2", *args]) == 0
