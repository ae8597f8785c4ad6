"""Rows of the 4-bit cache at the edges of tv_kv4_append and tv_kv4_read:
sequences without rows beside ones with rows (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from speculative_decoding_tree_gb300 import workloads as wl
from speculative_decoding_tree_gb300.runner import DeviceKv4Step
from gpu_helpers import workload
from kv4_helpers import bits

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows_of(st, counts, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    shape = (st.desc.num_kv_heads, sum(counts), st.desc.head_dim)
    return [torch.randn(shape, generator=g, device="cuda").to(st.q.dtype) for _ in range(2)]


def offsets(counts):
    return i32([0] + torch.tensor(counts).cumsum(0).tolist())


def four_sequences(d, dtype, paged):
    return DeviceKv4Step(workload(wl.small_variant(5, batch=4, hq=4, hkv=2, d=d, dtype=dtype, prefix=(40, 60), vocab=64,
                                                   paged=paged, seed=d)))


# Counts and starts: no start is a multiple of 16, the last sequence is empty
# (its first row would be row 8 of 8).
COUNTS, STARTS = [5, 0, 3, 0], [7, 21, 33, 13]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("bf16", 256), ("bf16", 512)])
@pytest.mark.parametrize("paged", [False, True])
def test_sequences_without_rows_touch_nothing(dtype, d, paged):
    st = four_sequences(d, dtype, paged)
    k, v = rows_of(st, COUNTS, 1)
    table = st.page_table
    if paged:
        table = table.clone()
        table[1, 21 // 16] = -1                          # an empty sequence whose page is gone
        table[3, 13 // 16] = table[0, 7 // 16]           # and one whose page another sequence now writes
    want_k, want_v = st.k4.clone(), st.v4.clone()
    for b in (0, 2):                                     # the two sequences with rows, each by itself
        a = sum(COUNTS[:b])
        one = [COUNTS[b] if x == b else 0 for x in range(4)]
        tv.tv_kv4_append(st.desc, COUNTS[b], COUNTS[b], k[:, a:a + COUNTS[b]].contiguous(),
                         v[:, a:a + COUNTS[b]].contiguous(), offsets(one), i32([STARTS[b] if x == b else 0 for x in range(4)]),
                         want_k, want_v, st.page_table, st.status)
    for _ in range(20):
        k4, v4 = st.k4.clone(), st.v4.clone()
        tv.tv_kv4_append(st.desc, 8, 5, k, v, offsets(COUNTS), i32(STARTS), k4, v4, table, st.status)
        torch.cuda.synchronize()
        assert int(st.status[0]) == 0
        assert torch.equal(k4, want_k) and torch.equal(v4, want_v)
    # read back: the rows that were written, and no fault for the missing page
    ko, vo = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    tv.tv_kv4_read(st.desc, 8, 5, k4, v4, table, offsets(COUNTS), i32(STARTS), ko, vo, st.status)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    one = torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    tv.tv_kv4_read(st.desc, 8, 5, want_k, want_v, st.page_table, offsets(COUNTS), i32([7, 0, 33, 0]), *one, st.status)
    assert torch.equal(bits(ko), bits(one[0])) and torch.equal(bits(vo), bits(one[1]))
    assert bool(torch.isfinite(ko).all()) and bool(torch.isfinite(vo).all())


def test_a_batch_of_empty_sequences():
    st = four_sequences(128, "bf16", True)
    k, v = rows_of(st, [1], 2)
    k4, v4 = st.k4.clone(), st.v4.clone()
    out = k.clone(), v.clone()
    none = i32([1, 1, 1, 1, 1])                          # all empty, behind the last of the rows
    table = torch.full_like(st.page_table, -1)
    tv.tv_kv4_append(st.desc, 1, 1, k, v, none, i32(STARTS), st.k4, st.v4, table, st.status)
    tv.tv_kv4_read(st.desc, 1, 1, st.k4, st.v4, table, none, i32(STARTS), k, v, st.status)
    torch.cuda.synchronize()
    assert int(st.status[0]) == 0
    assert torch.equal(st.k4, k4) and torch.equal(st.v4, v4)
    assert torch.equal(bits(k), bits(out[0])) and torch.equal(bits(v), bits(out[1]))
