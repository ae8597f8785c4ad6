"""The fp32 prompt attention to the accuracy its six products give, not the one
three of them would (GPU; the bounds' meaning: test_fp32_parts.py)."""
import numpy as np
import pytest
import torch

from fp32_parts import RMS_BOUND, relative_rms, scores_from, values_from_third_parts
from oracle import prompt as op
from prompt_helpers import Prompts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_relative_error(d, split):
    c = Prompts([900, 20], [200, 61], 4, 2, d, "f32", paged=True, seed=d) if split else \
        Prompts([40] * 20, [130] * 20, 4, 4, d, "f32", seed=d)
    assert (c.plan()["num_splits"] > 1) == split and c.plan()["kernel"] == 8
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0
    want = np.concatenate([op.attention(*c.seq(b), c.scale) for b in range(len(c.n))])
    assert relative_rms(c.out.double().cpu().numpy(), want) <= RMS_BOUND


@pytest.mark.parametrize("product", [(1, 1), (0, 2), (2, 0)])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_scores_from_one_small_product(d, product):
    """Scores of order 1 that are one product of parts, scaled up; without it all weights would be equal.

    All other products cancel among 16 channels.  Beside those of magnitude 2^-7 (large ones among the small products)
    the adder keeps bits down to 2^-31, so 3 d / 16 steps drop at most 2^-24.4 of scores of root mean square 2^-14 (d =
    128: 24 steps, 2^-15): 2^-10 relative.  Twice that in a weight, with scores up to 5, is below 2^-6."""
    P, n = 64, 100
    q, k = scores_from(product, n, P + n, d, seed=d)
    scale = float(np.float32(1 / (q.astype(np.float64) @ k.astype(np.float64).T).std()))
    c = Prompts([P], [n], 1, 1, d, "f32", seed=d, scale=scale)
    c.q[:, 0], c.k_rows[0] = torch.tensor(q), torch.tensor(k[P:])
    c.past[0] = (torch.tensor(k[None, :P]), c.past[0][1])
    c.k_cache[0, 0, :P] = c.past[0][0][0].cuda()
    c.gpu[0].copy_(c.q)
    c.gpu[1].copy_(c.k_rows)
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0
    qs, kp, vp, kr, vr = c.seq(0)
    want = op.attention(qs, kp, vp, kr, vr, scale)
    size = op.attention(qs, kp, np.abs(vp), kr, np.abs(vr), scale)
    err = np.abs(c.out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -6 * size).all()
    flat = np.abs(op.attention(0 * qs, kp, vp, kr, vr, scale) - want)
    assert (flat > 2.0 ** -6 * size).mean() > 0.5             # equal weights would not do


@pytest.mark.parametrize("d", [128, 256, 512])
def test_values_from_third_parts(d):
    """Equal weights (exactly 1) over pairs of rows of V whose first two parts cancel: the sums are third parts.

    A tile adds 8 steps of first parts of magnitude 1 to 2 to sums of up to 64 third parts (multiples of 2^-23, root mean
    square 2^-19.5 each, 2^-16.5 in all); a step drops what is below 2^-23 at most: 2^-20 of them at worst."""
    n = 256
    c = Prompts([0], [n], 1, 1, d, "f32", seed=d)
    c.k_rows.zero_()
    c.v_rows[0] = torch.tensor(values_from_third_parts(n, d, seed=d))
    c.gpu[1].copy_(c.k_rows)
    c.gpu[2].copy_(c.v_rows)
    c.attn()
    torch.cuda.synchronize()
    assert int(c.status[0]) == 0
    even = slice(1, None, 2)                                 # rows that see whole pairs
    want = op.attention(*c.seq(0), c.scale)[even]
    assert np.abs(want).max() < 2.0 ** -16
    assert relative_rms(c.out.double().cpu().numpy()[even], want) <= 0.25
