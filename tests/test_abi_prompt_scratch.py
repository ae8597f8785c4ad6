"""The prompt attention's scratch is a call's own: a smaller call may need more
(CPU: refused before any launch)."""
import ctypes

import pytest

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import _build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return tv.lib()


def test_the_size_of_a_longer_prompt_does_not_do_for_a_shorter_one(L):
    d = tv.make_desc(batch=1, num_q_heads=16, num_kv_heads=4, head_dim=256, dtype=tv.BF16, max_nodes=0, total_rows=0,
                     capacity=65536, max_prefix=32768)
    size = {n: tv.tv_prompt_workspace_size(d, n, n) for n in (50, 16384)}
    assert size[50] > size[16384]
    call = lambda n, ws: L.tv_prompt_attn(ctypes.byref(d), n, n, *[FAKE] * 10, ws, FAKE, None)
    assert call(50, size[16384]) == -10 and call(50, size[50] - 1) == -10
