"""The 4-bit cache's own calls take no tree: max_nodes and total_rows of their
descriptor are not looked at (CPU: no call reaches a kernel)."""
import ctypes

import pytest

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import _build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return tv.lib()


def desc(**kw):
    base = dict(batch=3, num_q_heads=8, num_kv_heads=8, head_dim=128, dtype=tv.BF16, max_nodes=0, total_rows=0,
                capacity=4176, max_prefix=4096)
    base.update(kw)
    return tv.make_desc(**base)


@pytest.mark.parametrize("nodes,rows", [(0, 0), (1, 3), (64, 100000), (4099, 4099), (-1, -5)])
def test_any_tree_is_taken(L, nodes, rows):
    d = desc(max_nodes=nodes, total_rows=rows)
    assert tv.tv_kv4_cache_bytes(d) == (3 * 8 * 261 * 1088, 3 * 8 * 261 * 1040)
    for f in (L.tv_kv4_append, L.tv_kv4_read):
        # nothing to do: the checks pass, and nothing is launched
        assert f(ctypes.byref(d), 0, 10, *[FAKE] * 8, None) == 0
        assert f(ctypes.byref(d), 10, 10, *[FAKE + 4] * 8, None) == -11


@pytest.mark.parametrize("kw,code", [(dict(batch=0), -6), (dict(num_kv_heads=0), -4), (dict(head_dim=64), -3),
                                     (dict(dtype=7), -2), (dict(capacity=4177), -6), (dict(page_size=16), -8),
                                     (dict(max_prefix=5000), -6)])
def test_the_rest_is_checked(L, kw, code):
    d = desc(**kw)
    n = [ctypes.c_int64(0), ctypes.c_int64(0)]
    assert L.tv_kv4_cache_bytes(ctypes.byref(d), *[ctypes.byref(x) for x in n]) == code
    for f in (L.tv_kv4_append, L.tv_kv4_read):
        assert f(ctypes.byref(d), 0, 10, *[FAKE] * 8, None) == code


def test_the_tree_is_checked_where_there_is_one(L):
    for kw in (dict(max_nodes=0, total_rows=3), dict(max_nodes=65, total_rows=65), dict(max_nodes=2, total_rows=7)):
        d = desc(**kw)
        n = ctypes.c_size_t(0)
        assert L.tv_kv4_workspace_size(ctypes.byref(d), None, ctypes.byref(n)) == -7
        assert L.tree_accept_commit_argmax_kv4(ctypes.byref(d), *[FAKE] * 14, None) == -7
