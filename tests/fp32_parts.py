"""fp32 numbers in three bf16 parts: a float64 restatement of the six products,
inputs whose answer comes from one of the small ones, and how large an error
says that one is missing."""
import numpy as np
import torch

PRODUCTS = [(0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)]      # parts of the left and of the right factor

# Relative rms error of attention on values from a unit normal, scale d^-1/2.
#
# A correct kernel.  The adder of a step of 16 products keeps 24 bits of the running score and drops the rest, on
# average half a last place: 2^-24.5 of a running score of about sqrt(16 j) after j steps, always to the same side, in all
# 2^-24.5 * 4 * 2/3 * (d / 16)^1.5, times the scale: 2.2e-7, 4.5e-7 and 9e-7 at head_dim 128, 256, 512.  A weight's
# error is the score's; with the softmax's own roundings (numbers up to 2^3 in log2 units, two of them: 2e-7; the
# exponential: 1e-7) and the products with V (8 steps a tile: 2e-7) that makes 3.8e-7, 5.4e-7 and 9.5e-7 of root mean
# square.
#
# One missing product.  The second part of a number is at most 2^-8 of it and the third 2^-16: test_fp32_parts.py takes
# each product out of the float64 restatement and finds 2.1e-6 or more.
RMS_BOUND = 1.5e-6


def parts(x):
    """[3] arrays of bf16 values that sum to the fp32 array x."""
    x = torch.as_tensor(np.asarray(x, np.float32))
    out = []
    for _ in range(3):
        p = x.bfloat16().float()
        out.append(p.double().numpy())
        x = x - p
    return out


def products(a, b, without=()):
    """a @ b as the sum of the products of their parts, in float64."""
    a, b = parts(a), parts(b)
    return sum(a[i] @ b[j] for i, j in PRODUCTS if (i, j) not in without)


def relative_rms(got, want):
    return float(np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean()))


def _spread(g, *shape):
    """Magnitudes from 1 to 2 of both signs, fp32, whose first two parts are those of their sum (a second part of half a
    step of the first may round the other way there: such numbers become their first part)."""
    x = ((1 + torch.rand(*shape, generator=g)) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)).numpy()
    x1, x2, _ = parts(x)
    return np.where(parts(x1 + x2)[0] == x1, x, x1).astype(np.float32)


def scores_from(product, rows, keys, d, seed=0):
    """(q [rows, d], k [keys, d]) fp32 whose scores are the named product of parts alone: groups of channels in which
    every other product cancels, within the 16 channels that are added at once."""
    g = torch.Generator().manual_seed(seed)
    if product == (1, 1):
        x, y = _spread(g, rows, d // 4), _spread(g, keys, d // 4)
        (x1, x2, _), (y1, y2, _) = parts(x), parts(y)
        q, k = (x1 + x2, x1, x1 + x2, x1), (y1 + y2, -y1 - y2, -y1, y1)      # (x - x1) (y - y1)
    else:
        x, y = _spread(g, rows, d // 2), _spread(g, keys, d // 2)
        (x1, x2, x3), (y1, y2, y3) = parts(x), parts(y)
        if product == (0, 2):
            q, k = (x1, x1), (y, -y1 - y2)                                   # x1 (y - y1 - y2)
        else:
            q, k = (x, -x1 - x2), (y1, y1)
    flat = lambda t: np.stack([np.asarray(c, np.float64) for c in t], -1).reshape(t[0].shape[0], d).astype(np.float32)
    return flat(q), flat(k)


def values_from_third_parts(keys, d, seed=0):
    """v [keys, d] fp32, keys even: the first and second parts of neighbours cancel, what is left are third parts."""
    g = torch.Generator().manual_seed(seed)
    w = _spread(g, keys // 2, d)
    w1, w2, _ = parts(w)
    return np.stack([w.astype(np.float64), -w1 - w2], 1).reshape(keys, d).astype(np.float32)
