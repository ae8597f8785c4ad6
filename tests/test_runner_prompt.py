"""What DevicePrompt, LogitControl and the command do around the library's calls
(CPU: the calls enqueue nothing, or stand-ins record them)."""
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import _build, runner

P0 = [3, 0, 17]


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    _build.build()
    monkeypatch.setattr(tv, "_current_stream", lambda: 0)


def step(**kw):
    """What DevicePrompt and LogitControl look at of a step, on the CPU."""
    B = len(P0)
    desc = tv.make_desc(batch=B, num_q_heads=4, num_kv_heads=2, head_dim=128, dtype=tv.BF16, max_nodes=4, total_rows=6,
                        capacity=64, max_prefix=20)
    bf = dict(dtype=torch.bfloat16)
    base = dict(desc=desc, device=torch.device("cpu"), vocab=50, logits_dtype=tv.F32, page_table=None,
                q=torch.zeros(6, 4, 128, **bf), out=torch.zeros(6, 4, 128, **bf), k_cache=torch.zeros(B, 2, 64, 128, **bf),
                v_cache=torch.zeros(B, 2, 64, 128, **bf), prefix_len=torch.tensor(P0, dtype=torch.int32),
                status=torch.zeros(4, dtype=torch.int32), tokens=torch.zeros(B, 4, dtype=torch.int32),
                logits=torch.zeros(6, 50))
    return SimpleNamespace(**{**base, **kw})


def test_empty_prompts_leave_the_lengths():
    st = step()
    pr = runner.DevicePrompt(st, [0, 0, 0])
    pr.new_prefix.fill_(-77)                             # as uninitialised memory may be
    none = torch.zeros(0, 4, 128, dtype=torch.bfloat16)
    pr.run(none, none[:, :2], none[:, :2])
    assert st.prefix_len.tolist() == P0 and pr.new_prefix.tolist() == P0


class Recorder(SimpleNamespace):
    """A step of the command on the CPU: `seen` has the logits that acceptance went by, step by step."""

    def __init__(self, w, *_):
        super().__init__(**vars(step()), seen=[])
        self.logits = torch.arange(300.0).reshape(6, 50) % 7
        self.mask = self.attn = lambda *_: None
        made.append(self)

    def step(self, argmax=None):
        self.seen.append(self.logits.clone() if argmax is None else argmax)


class AddOne:
    """A control that adds 10 to token 3 of every row."""

    def __init__(self, st, *_, **__):
        self.st = st
        self.process = lambda: st.logits[:, 3].add_(10)

    def __getattr__(self, name):
        return lambda *_: None


made = []


@pytest.fixture
def command(monkeypatch):
    for name in ("DeviceStep", "DeviceKv4Step"):
        monkeypatch.setattr(runner, name, Recorder)
    monkeypatch.setattr(runner, "LogitControl", AddOne)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda: None)

    def run(*args):
        made.clear()
        assert runner.main(["--config", "1", *args]) == 0
        return made[0]
    return run


def test_the_4_bit_step_accepts_on_steered_logits(command):
    raw = torch.arange(300.0).reshape(6, 50) % 7
    steered = raw.clone()
    steered[:, 3] += 10
    st = command("--kv4", "--steps", "1", "--steer")
    assert st.seen[0].dtype == torch.int32 and st.seen[0].tolist() == [3] * 6
    assert command("--kv4", "--steps", "1").seen[0].tolist() == raw.argmax(1).tolist()


@pytest.mark.parametrize("kind", [(), ("--kv4",)])
def test_every_step_steers_the_targets_logits(command, kind):
    raw = torch.arange(300.0).reshape(6, 50) % 7
    raw[:, 3] += 10
    st = command(*kind, "--steps", "3", "--steer")
    want = torch.full((6,), 3, dtype=torch.int32) if kind else raw
    assert len(st.seen) == 3 and all(torch.equal(x, want) for x in st.seen) and torch.equal(st.logits, raw)


def test_first_roots_are_counted_as_emitted(monkeypatch):
    calls = []
    monkeypatch.setattr(runner, "tv_token_counts_add", lambda d, t, o, n, prompt, *_: calls.append((t.tolist(), o, n, prompt)))
    st = step(draft=torch.tensor([9, 1, 4, 30, 31, 8], dtype=torch.int32), node_offsets=torch.tensor([0, 2, 3, 6], dtype=torch.int32))
    runner.LogitControl(st, torch.ones(3, 3)).started()
    assert calls == [([9, 4, 30], None, 1, False)]


def test_windowed_prompts_are_refused():
    st = runner.DeviceWindowStep.__new__(runner.DeviceWindowStep)
    vars(st).update(vars(step()), win=tv.make_window(30, 4))
    with pytest.raises(NotImplementedError, match="window"):
        runner.DevicePrompt(st, [5, 11, 0])                  # positions up to 20 + 10
    assert runner.DevicePrompt(st, [5, 10, 0]).rows == 15   # 29 is the last that sees everything
    assert runner.DevicePrompt(st, [30, 1, 0], max_prefix=0).rows == 31


def test_prompts_of_4_bit_steps_are_refused():
    with pytest.raises(NotImplementedError, match="append"):
        runner.DevicePrompt(runner.DeviceKv4Step.__new__(runner.DeviceKv4Step), [5])


def test_command_refuses_windowed_prompts(capsys):
    with pytest.raises(SystemExit) as e:
        runner.main(["--window", "64,4", "--prompt", "5"])
    assert e.value.code == 2 and "--prompt" in capsys.readouterr().err


def test_calls_on_a_stream_keep_what_they_use(monkeypatch):
    """Every tensor a call hands to the library that is not the step's own is kept until the stream has passed."""
    step_own, handed, kept = set(), set(), set()
    ids = lambda xs: {x.data_ptr() for x in xs if isinstance(x, torch.Tensor) and x.numel()}
    for name in ("tv_prompt_rope_store", "tv_prompt_attn", "tv_token_counts_add", "tv_tree_logits_process"):
        monkeypatch.setattr(runner, name, lambda *a: handed.update(ids(a)))
    monkeypatch.setattr(runner, "_keep", lambda stream, *t: kept.update(ids(t)) if stream is not None else None)
    monkeypatch.setattr(runner, "_on", lambda stream: runner.contextlib.nullcontext())
    i32 = dict(dtype=torch.int32)
    st = step(draft=torch.zeros(6, **i32), node_offsets=torch.tensor([0, 2, 3, 6], **i32), anc=torch.zeros(6, dtype=torch.int64))
    step_own = ids(vars(st).values())
    pr = runner.DevicePrompt(st, [5, 3, 0])
    bias = (torch.zeros(4, **i32), torch.zeros(2, **i32), torch.zeros(2))
    ctl = runner.LogitControl(st, torch.ones(3, 3), bias, torch.zeros(6, 2, **i32))
    tokens, offsets = torch.zeros(8, **i32), torch.tensor([0, 5, 8, 8], **i32)
    rows = [torch.zeros(8, h, 128, dtype=torch.bfloat16) for h in (4, 2, 2)]
    calls = [lambda: pr.rope_store(*rows, 7), lambda: pr.attn(7), lambda: pr.run(*rows, 7), lambda: ctl.process(7),
             lambda: ctl.read(tokens, offsets, 7), lambda: ctl.emitted(7)]
    for call in calls:
        handed.clear()
        kept.clear()
        call()
        assert handed - step_own and not handed - step_own - kept


@pytest.mark.parametrize("lens", [[], [4, 5], [1, 2, 3, 4], [3, -1, 2]])
def test_one_length_a_sequence(lens):
    """Fewer lengths would make offsets that end before the last sequence's."""
    with pytest.raises(ValueError, match="lens"):
        runner.DevicePrompt(step(), lens)


def test_an_empty_bias_list_is_no_bias(monkeypatch):
    calls = []
    monkeypatch.setattr(runner, "tv_tree_logits_process", lambda *a: calls.append(a))
    i32 = dict(dtype=torch.int32)
    st = step(draft=torch.zeros(6, **i32), node_offsets=torch.tensor([0, 2, 3, 6], **i32), anc=torch.zeros(6, dtype=torch.int64))
    ctl = runner.LogitControl(st, torch.ones(3, 3), (torch.zeros(4, **i32), torch.zeros(0, **i32), torch.zeros(0)))
    ctl.process()
    assert ctl.desc.biases == 0 and calls[0][4:7] == (None, None, None)
