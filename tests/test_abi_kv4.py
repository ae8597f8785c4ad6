"""Host checks of the windowed attention and of the 4-bit cache: every bad
argument is refused before any launch.  CPU only: no call reaches a kernel."""
import ctypes

import pytest

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import _build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    _build.build()
    return tv.lib()


def _desc(**kw):
    base = dict(batch=1, num_q_heads=32, num_kv_heads=8, head_dim=256, dtype=tv.BF16, max_nodes=64, total_rows=64,
                capacity=4176, max_prefix=4096)
    base.update(kw)
    return tv.make_desc(**base)


def _attn(L, name, d, win, ptrs=None, ws=1 << 40, status=FAKE):
    p = [FAKE] * 12 if ptrs is None else ptrs
    return getattr(L, name)(None if d is None else ctypes.byref(d), None if win is None else ctypes.byref(win), *p,
                            ws, status, None)


NAMES = ["tree_verify_attn_window", "tree_verify_attn_kv4"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,code", [
    (dict(num_kv_heads=0), -4), (dict(num_q_heads=30), -5), (dict(head_dim=64), -3), (dict(dtype=7), -2),
    (dict(max_nodes=65, total_rows=65), -7), (dict(batch=0), -6), (dict(max_prefix=5000), -6),
    (dict(page_size=8), -8), (dict(page_size=16, num_pages=0), -8), (dict(capacity=2 ** 62, max_prefix=4096), -9),
    (dict(batch=70000, total_rows=70000, max_nodes=1, capacity=64, max_prefix=64), -6),
])
def test_descriptor_refused(L, name, kw, code):
    assert _attn(L, name, _desc(**kw), tv.make_window(64, 4)) == code


@pytest.mark.parametrize("name", NAMES)
def test_window_pointer_and_workspace_refused(L, name):
    d = _desc()
    for win in ((0, 0), (-5, 0), (8, -1)):
        assert _attn(L, name, d, tv.make_window(*win)) == -6
    ok = tv.make_window(100, 4)
    assert _attn(L, name, None, ok) == -1
    for i in range(12):
        if i == 3:                                       # the page table of a contiguous cache may be NULL
            continue
        assert _attn(L, name, d, ok, [None if j == i else FAKE for j in range(12)]) == -1, i
        assert _attn(L, name, d, ok, [FAKE + 8 if j == i else FAKE for j in range(12)]) == -11, i
    assert _attn(L, name, d, ok, status=None) == -1
    assert _attn(L, name, d, ok, ws=16) == -10
    paged = _desc(page_size=16, num_pages=300)
    assert _attn(L, name, paged, ok, [None if j == 3 else FAKE for j in range(12)]) == -1


def test_window_is_required_only_where_it_defines_the_call(L):
    d = _desc()
    n = ctypes.c_size_t(0)
    assert _attn(L, "tree_verify_attn_window", d, None) == -1
    assert L.tv_window_workspace_size(ctypes.byref(d), None, ctypes.byref(n)) == -1
    assert L.tv_kv4_workspace_size(ctypes.byref(d), None, ctypes.byref(n)) == 0 and n.value > 0
    assert L.tv_kv4_workspace_size(ctypes.byref(d), None, None) == -1
    with pytest.raises(tv.TreeVerifyError):
        tv.tv_window_workspace_size(d, tv.make_window(0))


def test_capacity_in_whole_blocks(L):
    odd = _desc(capacity=4177)
    k, v = ctypes.c_int64(0), ctypes.c_int64(0)
    assert L.tv_kv4_cache_bytes(ctypes.byref(odd), ctypes.byref(k), ctypes.byref(v)) == -6
    assert _attn(L, "tree_verify_attn_kv4", odd, None) == -6
    assert tv.tv_kv4_cache_bytes(_desc()) == (8 * 261 * 8.5 * 256, 8 * 261 * (8 * 256 + 16))
    assert tv.tv_kv4_cache_bytes(_desc(page_size=16, num_pages=7)) == (7 * 8 * 2176, 7 * 8 * 2064)


def test_window_bounds_the_keys_of_a_plan(L):
    d = _desc(capacity=32784, max_prefix=32768)
    full = tv.tv_attn_plan(d)
    small = tv.tv_window_attn_plan(d, tv.make_window(1024, 4))
    assert small["chunk"] * small["num_splits"] <= 2048 < full["chunk"] * full["num_splits"]
    wide = tv.tv_window_attn_plan(d, tv.make_window(2 ** 62, 2 ** 62))
    assert wide["chunk"] * wide["num_splits"] >= 32768
    assert tv.tv_window_attn_plan(_desc(dtype=tv.F32), tv.make_window(9))["kernel"] == 0


@pytest.mark.parametrize("name", ["tv_kv4_append", "tv_kv4_read"])
def test_rows_refused(L, name):
    f = getattr(L, name)
    d = ctypes.byref(_desc())
    ptrs = [FAKE] * 8
    assert f(None, 10, 10, *ptrs, None) == -1
    assert f(d, -1, 10, *ptrs, None) == -6 and f(d, 10, -1, *ptrs, None) == -6
    assert f(d, 2 ** 31, 10, *ptrs, None) == -6
    table = 6 if name == "tv_kv4_append" else 2
    for i in range(8):
        if i == table:
            continue
        assert f(d, 10, 10, *[None if j == i else FAKE for j in range(8)], None) == -1, i
        assert f(d, 10, 10, *[FAKE + 4 if j == i else FAKE for j in range(8)], None) == -11, i
    paged = ctypes.byref(_desc(page_size=16, num_pages=300))
    assert f(paged, 10, 10, *[None if j == table else FAKE for j in range(8)], None) == -1
    assert f(ctypes.byref(_desc(capacity=4177)), 10, 10, *ptrs, None) == -6
    assert f(d, 0, 10, *ptrs, None) == 0 and f(d, 10, 0, *ptrs, None) == 0       # nothing to do, nothing launched


def test_commit_refused(L):
    f = L.tree_accept_commit_argmax_kv4
    d = ctypes.byref(_desc())
    assert f(None, *[FAKE] * 14, None) == -1
    for i in range(14):
        if i == 8:
            continue
        assert f(d, *[None if j == i else FAKE for j in range(14)], None) == -1, i
        assert f(d, *[FAKE + 2 if j == i else FAKE for j in range(14)], None) == -11, i
    assert f(ctypes.byref(_desc(capacity=4177)), *[FAKE] * 14, None) == -6
    assert f(ctypes.byref(_desc(page_size=16, num_pages=9)), *[None if j == 8 else FAKE for j in range(14)],
             None) == -1
