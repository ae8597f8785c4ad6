"""What the windowed and the 4-bit steps refuse (CPU: no call reaches the
library)."""
import pytest

from speculative_decoding_tree_gb300 import runner


def bare(kind):
    return kind.__new__(kind)


@pytest.mark.parametrize("kind,calls", [
    (runner.DeviceWindowStep, [("partials", ()), ("merge", ())]),
    (runner.DeviceKv4Step, [("partials", ()), ("merge", ()), ("accept_commit", ()),
                            ("accept_commit_sampled", (1.0, 1, 0))]),
])
def test_calls_without_a_form_say_so(kind, calls):
    for name, args in calls:
        with pytest.raises(NotImplementedError, match="use "):
            getattr(bare(kind), name)(*args)


def test_a_4_bit_step_wants_the_argmax():
    with pytest.raises(TypeError):
        bare(runner.DeviceKv4Step).step()


def test_command_refuses_draws_on_the_4_bit_cache(capsys):
    with pytest.raises(SystemExit) as e:
        runner.main(["--kv4", "--sampled", "0.7"])
    assert e.value.code == 2 and "--sampled" in capsys.readouterr().err
