"""Host checks of the prompt's calls and of the logits' control: every bad
argument is refused before any launch.  CPU only: no call reaches a kernel."""
import ctypes

import pytest

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import _build

FAKE = 1 << 20
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return tv.lib()


def _desc(**kw):
    base = dict(batch=2, num_q_heads=32, num_kv_heads=8, head_dim=128, dtype=tv.BF16, max_nodes=0, total_rows=0,
                capacity=4176, max_prefix=4096)
    base.update(kw)
    return tv.make_desc(**base)


def _attn(L, d, rows=100, max_rows=60, ptrs=None, ws=1 << 50, status=FAKE):
    p = [FAKE] * 10 if ptrs is None else ptrs
    return L.tv_prompt_attn(None if d is None else ctypes.byref(d), rows, max_rows, *p, ws, status, None)


def _rope(L, d, rows=100, max_rows=60, theta=1e4, ptrs=None):
    p = [FAKE] * 13 if ptrs is None else ptrs
    return L.tv_prompt_rope_store(None if d is None else ctypes.byref(d), rows, max_rows, theta, *p, None)


def but(n, i, x):
    return [x if j == i else FAKE for j in range(n)]


@pytest.mark.parametrize("call", [_attn, _rope])
@pytest.mark.parametrize("kw,code", [
    (dict(num_kv_heads=0), -4), (dict(num_q_heads=30), -5), (dict(head_dim=64), -3), (dict(dtype=7), -2),
    (dict(batch=0), -6), (dict(max_prefix=5000), -6), (dict(page_size=8), -8), (dict(page_size=16, num_pages=0), -8),
    (dict(capacity=2 ** 62, max_prefix=4096), -9), (dict(scale=NAN), -6),
])
def test_descriptor_refused(L, call, kw, code):
    assert call(L, _desc(**kw)) == code


@pytest.mark.parametrize("call", [_attn, _rope])
def test_rows(L, call):
    d = _desc()
    assert call(L, None) == -1
    assert call(L, d, rows=-1) == -6 and call(L, d, max_rows=-1) == -6 and call(L, d, rows=2 ** 31) == -6
    nothing = [None] * (10 if call is _attn else 13)
    assert call(L, d, rows=0, ptrs=nothing) == 0 and call(L, d, max_rows=0, ptrs=nothing) == 0


def test_attention_pointers(L):
    d = _desc()
    for i in range(10):
        if i not in (3, 9):                              # the page table of a contiguous cache, the unsplit call's scratch
            assert _attn(L, d, ptrs=but(10, i, None)) == -1, i
        assert _attn(L, d, ptrs=but(10, i, FAKE + 8)) == -11, i
    assert _attn(L, d, status=None) == -1
    paged = _desc(page_size=16, num_pages=300)
    assert _attn(L, paged, ptrs=but(10, 3, None)) == -1
    # a prefix's split needs its scratch, and so does fp32
    assert tv.tv_prompt_attn_plan(d, 100, 60)["num_splits"] > 1
    assert _attn(L, d, ptrs=but(10, 9, None)) == -1 and _attn(L, d, ws=16) == -10
    fresh = _desc(dtype=tv.F32, max_prefix=0)
    assert _attn(L, fresh, ptrs=but(10, 9, None)) == -1 and _attn(L, fresh, ws=16) == -10


def test_plans(L):
    plan = lambda rows=5000, most=5000, **kw: tv.tv_prompt_attn_plan(_desc(**kw), rows, most)
    assert plan()["kernel"] == 6 and plan(head_dim=256)["kernel"] == 7 and plan(head_dim=512)["kernel"] == 7
    assert plan(dtype=tv.F32)["kernel"] == 8
    assert plan(num_q_heads=130, num_kv_heads=1)["kernel"] == 8              # more heads a group than a tile has rows
    assert plan(page_size=16, num_pages=2 ** 25)["kernel"] == 8              # a cache of 2^32 rows
    assert plan(max_prefix=0, page_size=16, num_pages=2 ** 25)["kernel"] == 6   # which no prefix reads
    assert tv.tv_prompt_workspace_size(_desc(max_prefix=0), 5000, 5000) == 0
    assert tv.tv_prompt_workspace_size(_desc(), 0, 0) >= 0
    n = ctypes.c_size_t(0)
    assert L.tv_prompt_workspace_size(ctypes.byref(_desc()), 5, 5, None) == -1
    assert L.tv_prompt_attn_plan(ctypes.byref(_desc()), 5, 5, None) == -1
    big = _desc(num_q_heads=512, num_kv_heads=512, batch=2 ** 20, capacity=16, max_prefix=16, dtype=tv.F32)
    assert L.tv_prompt_workspace_size(ctypes.byref(big), 2 ** 31 - 1, 2 ** 31 - 1, ctypes.byref(n)) == -9


def test_rope_arguments(L):
    d = _desc()
    for theta in (1.0, 0.0, -5.0, NAN, INF):
        assert _rope(L, d, theta=theta) == -6
    for i in range(13):
        if i not in (10, 11):                            # page table, new lengths
            assert _rope(L, d, ptrs=but(13, i, None)) == -1, i
        assert _rope(L, d, ptrs=but(13, i, FAKE + 4)) == -11, i
    assert _rope(L, _desc(page_size=16, num_pages=300), ptrs=but(13, 10, None)) == -1
    assert _rope(L, d) == -6                             # the new lengths over the old ones


def test_grids_that_do_not_fit(L):
    n = ctypes.c_size_t(0)
    wide = _desc(num_q_heads=2 ** 30, num_kv_heads=2 ** 30, batch=2 ** 31 - 1, page_size=16, num_pages=1, capacity=16,
                 max_prefix=0)
    assert L.tv_prompt_workspace_size(ctypes.byref(wide), 2 ** 20, 2 ** 20, ctypes.byref(n)) == -9


def _logits(**kw):
    base = dict(batch=2, vocab=1000, max_nodes=8, total_rows=10, logits_dtype=tv.F32, biases=3)
    base.update(kw)
    return tv.make_logits_desc(**base)


def _process(L, d, ptrs=None):
    return L.tv_tree_logits_process(None if d is None else ctypes.byref(d), *([FAKE] * 12 if ptrs is None else ptrs),
                                    None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -6), (dict(vocab=0), -6), (dict(vocab=2 ** 30 + 1), -6), (dict(logits_dtype=9), -2),
    (dict(max_nodes=65, total_rows=65), -7), (dict(max_nodes=0), -7), (dict(total_rows=1), -7),
    (dict(total_rows=17), -7), (dict(biases=-1), -6),
])
def test_logits_descriptor_refused(L, kw, code):
    assert _process(L, _logits(**kw)) == code


def test_logits_pointers(L):
    d = _logits()
    assert _process(L, None) == -1
    for i in range(12):
        if i != 6:                                       # the mask; the others are required, or go in pairs and threes
            assert _process(L, d, but(12, i, None)) == -1, i
        assert _process(L, d, but(12, i, FAKE + 2)) == -11, i


def test_counts_arguments(L):
    d = ctypes.byref(_logits(max_nodes=0, total_rows=0, logits_dtype=9))     # not looked at
    f = L.tv_token_counts_add
    assert f(None, FAKE, FAKE, 5, 1, FAKE, FAKE, None) == -1
    assert f(d, FAKE, FAKE, -1, 1, FAKE, FAKE, None) == -6 and f(d, FAKE, FAKE, 2 ** 31, 1, FAKE, FAKE, None) == -6
    assert f(d, None, None, 0, 1, None, None, None) == 0
    for i in (0, 4, 5):
        p = [FAKE, FAKE, 5, 1, FAKE, FAKE]
        p[i] = None
        assert f(d, *p, None) == -1
    for i in (0, 1, 4, 5):
        p = [FAKE, FAKE, 5, 1, FAKE, FAKE]
        p[i] = FAKE + 4
        assert f(d, *p, None) == -11
    assert f(ctypes.byref(_logits(batch=0)), FAKE, FAKE, 5, 1, FAKE, FAKE, None) == -6


def test_status_names(L):
    assert "vocabulary" in tv.tv_status_string(256) and tv.DEV_BITS[256] == "BAD_TOKEN"


def test_command_refuses_prompts_on_the_4_bit_cache(capsys):
    from speculative_decoding_tree_gb300 import runner
    with pytest.raises(SystemExit):
        runner.main(["--kv4", "--prompt", "5"])
    assert "--prompt" in capsys.readouterr().err
