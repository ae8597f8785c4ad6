"""Prompt attention against the float64 oracle (GPU)."""
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from prompt_helpers import Prompts

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f32"]
# lengths around the tiles of 16 (pages), 64 and 128 keys and of 128 / G rows
ROWS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257, 300]
PREFIX = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 256, 300, 511]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (256, 4, 2), (512, 4, 1)])
def test_lengths(d, hq, hkv, dtype, paged):
    """Every row count of ROWS, each behind some prefix of PREFIX, in one packed batch."""
    pre = [PREFIX[(3 * i + 1) % len(PREFIX)] for i in range(len(ROWS))]
    c = Prompts(pre, ROWS, hq, hkv, d, dtype, paged, pad=5, seed=d)
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", PREFIX)
def test_prefixes(p, dtype):
    c = Prompts([p, p], [40, 1], 4, 1, 128, dtype, paged=True, seed=p)
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (5, 1), (7, 7), (16, 1), (48, 1), (130, 1)])
def test_heads(hq, hkv, d, dtype):
    n = 70 if hq < 100 else 9
    c = Prompts([37, 0], [n, 20], hq, hkv, d, dtype, seed=hq)
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_empty_sequences_and_padding(dtype):
    c = Prompts([5, 0, 200, 7, 0], [0, 33, 0, 1, 0], 4, 2, 128, dtype, paged=True, pad=200)
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 4, 2), (512, 2, 1)])
@pytest.mark.parametrize("p,n", [(4000, 3), (2047, 130), (2049, 64), (0, 1500), (1029, 700)])
def test_split_over_the_keys(p, n, d, hq, hkv, dtype):
    """Few rows over many keys: split, and joined from partials; rows of one chunk and of several in one call."""
    c = Prompts([p], [n], hq, hkv, d, dtype, paged=p % 2 == 0, pad=3, seed=n)
    assert c.plan()["num_splits"] > 1
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_split_of_a_ragged_batch(dtype):
    c = Prompts([3000, 0, 130, 2999], [5, 90, 0, 200], 4, 1, 128, dtype, seed=3)
    assert c.plan()["num_splits"] > 1
    c.attn()
    c.check()


@pytest.mark.parametrize("amp", [0.0, 8.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 4, 2), (512, 4, 1)])
def test_flat_and_steep_scores(d, hq, hkv, dtype, amp):
    """All scores equal; and scores whose maximum moves by hundreds from tile to tile."""
    c = Prompts([600, 0], [150, 260], hq, hkv, d, dtype, amp=amp, seed=9)
    c.attn()
    c.check()


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 4, 2), (512, 2, 1)])
def test_fp32_output_and_scale(d, hq, hkv):
    c = Prompts([100], [200], hq, hkv, d, "bf16", out_f32=True, scale=0.02)
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_no_prefix_without_a_cache(dtype):
    c = Prompts([0, 0], [100, 33], 4, 2, 128, dtype)
    c.k_cache = c.v_cache = None
    c.attn()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 4, 2), (512, 2, 1)])
def test_wider_bounds_give_the_same_rows(d, hq, hkv, dtype):
    """max_rows and max_prefix above the true ones."""
    a = Prompts([70, 300], [90, 20], hq, hkv, d, dtype, seed=4)
    b = Prompts([70, 300], [90, 20], hq, hkv, d, dtype, seed=4, max_rows=500, max_prefix=310)
    for c in (a, b):
        c.attn()
        c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 1), (256, 4, 1), (512, 4, 1)])
def test_same_bytes_every_time(d, hq, hkv, dtype):
    c = Prompts([900, 30], [70, 300], hq, hkv, d, dtype, seed=5)
    c.attn()
    first = c.out.clone()
    c.ws.fill_(0)
    for _ in range(3):
        c.out.zero_()
        c.attn()
        torch.cuda.synchronize()
        n = int(c.offsets_cpu[-1])
        assert torch.equal(c.out[:n].view(torch.uint8), first[:n].view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 2, 1), (512, 2, 1)])
def test_neighbours_do_not_reach_a_row(d, hq, hkv, dtype):
    """Another sequence's rows (NaN and infinity in all of them) leave a sequence's answer as it was."""
    c = Prompts([20, 50, 20], [37, 70, 37], hq, hkv, d, dtype, seed=6)
    c.attn()
    torch.cuda.synchronize()
    first = c.out.clone()
    o, e = c.offsets_cpu[1], c.offsets_cpu[2]
    q, k, v = c.gpu
    for bad in (float("nan"), float("inf")):
        q[o:e], k[:, o:e], v[:, o:e] = bad, bad, bad
        c.attn()
        torch.cuda.synchronize()
        assert torch.equal(c.out[:o], first[:o]) and torch.equal(c.out[e:], first[e:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 2, 1), (512, 2, 1)])
def test_infinite_keys_that_no_row_sees(d, hq, hkv, dtype):
    """K of later rows may be anything; a seen -inf score takes no part."""
    c = Prompts([0], [200], hq, hkv, d, dtype, seed=7)
    c.k_rows[:, 150:] = float("nan")
    c.gpu[1].copy_(c.k_rows)
    c.attn()
    torch.cuda.synchronize()
    got = c.out[:150].double().cpu().numpy()
    from prompt_helpers import reference
    q, kp, vp, kr, vr = c.seq(0)
    ref, lim = reference(q[:150], kp, vp, kr[:, :150], vr[:, :150], c.scale, c.bf16, c.out_f32)
    assert (abs(got - ref) <= lim).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_device_faults(dtype):
    # a prefix length out of range is clamped and reported
    c = Prompts([40], [20], 4, 2, 128, dtype)
    c.prefix.fill_(1000)
    c.attn()
    c.check(status=4)
    # offsets that run backwards or past the rows leave their sequences out
    c = Prompts([10, 10, 10], [20, 20, 20], 4, 2, 128, dtype)
    c.offsets.copy_(torch.tensor([0, 30, 20, 70], dtype=torch.int32))
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 2 and (c.out == 7.0).all()
    # a page out of range reads as zeros
    c = Prompts([40], [20], 4, 2, 128, dtype, paged=True)
    c.table[0, 1] = -5
    for x in c.past[0]:
        x[:, 16:32] = 0
    c.attn()
    c.check(status=8)
    c.table[0, 1] = 2 ** 31 - 1
    c.status.zero_()
    c.attn()
    c.check(status=8)


def test_more_sequences_than_a_warp():
    n = [(7 * i) % 23 for i in range(75)]
    p = [(5 * i) % 40 for i in range(75)]
    for dtype in TYPES:
        c = Prompts(p, n, 4, 2, 128, dtype, paged=True, seed=8)
        c.attn()
        c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (256, 4, 2), (512, 2, 1)])
def test_streams_and_graphs(d, hq, hkv, dtype):
    """Two calls on two streams, and two graphs replayed after new inputs and lengths."""
    a = Prompts([700], [90], hq, hkv, d, dtype, seed=10, max_prefix=700)
    b = Prompts([0, 64], [300, 5], hq, hkv, d, dtype, seed=11)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a.attn(s1.cuda_stream)
    b.attn(s2.cuda_stream)
    torch.cuda.synchronize()
    a.check()
    b.check()
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        a.attn()
    with torch.cuda.graph(gb):
        b.attn()
    for x in (a, b):
        x.q.mul_(0.5)
        x.gpu[0].copy_(x.q)
        x.out.fill_(7.0)
    a.prefix.fill_(333)
    a.past[0] = tuple(t[:, :333] for t in a.past[0])
    torch.cuda.synchronize()
    for _ in range(2):
        ga.replay()
        gb.replay()
    a.check()
    b.check()
