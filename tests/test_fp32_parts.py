"""What the bounds of the fp32 attention tests tell apart, on the float64
restatement of its arithmetic (CPU)."""
import numpy as np
import pytest

from fp32_parts import PRODUCTS, RMS_BOUND, products, relative_rms, scores_from, values_from_third_parts
from oracle import prompt as op


def attention(q, k, v, first, scale, without_qk=(), without_pv=()):
    """Rows at positions first, first + 1, ...; fp32 scores and weights, products of parts."""
    f32 = lambda x: x.astype(np.float32).astype(np.float64)
    x = f32(f32(products(q, k.T, without_qk)) * (scale * np.log2(np.e)))
    x = np.where(np.arange(len(k)) <= first + np.arange(len(q))[:, None], x, -np.inf)
    p = f32(np.exp2(f32(x - x.max(1, keepdims=True))))
    return products(p, v, without_pv) / p.sum(1, keepdims=True)


def exact(q, k, v, first, scale):
    return op.attention(q[:, None], k[None, :first], v[None, :first], k[None, first:], v[None, first:], scale)[:, 0]


@pytest.mark.parametrize("d", [128, 256, 512])
def test_a_missing_product_is_outside_the_bound(d):
    g = np.random.default_rng(d)
    q, k, v = (g.standard_normal((n, d)).astype(np.float32) for n in (150, 450, 450))
    want = exact(q, k, v, 300, d ** -0.5)
    err = lambda **kw: relative_rms(attention(q, k, v, 300, d ** -0.5, **kw), want)
    assert err() < 0.2 * RMS_BOUND
    for missing in PRODUCTS:
        assert err(without_qk=[missing]) > 1.3 * RMS_BOUND and err(without_pv=[missing]) > 1.3 * RMS_BOUND, missing


@pytest.mark.parametrize("product", [(1, 1), (0, 2), (2, 0)])
@pytest.mark.parametrize("d", [128, 512])
def test_scores_of_one_product(d, product):
    q, k = scores_from(product, 40, 100, d)
    s = q.astype(np.float64) @ k.astype(np.float64).T
    assert np.abs(products(q, k.T) - s).max() <= 2.0 ** -8 * s.std()
    without = products(q, k.T, [product])
    assert np.abs(without).max() <= 2.0 ** -6 * s.std()
    assert 2.0 ** -20 < s.std() < 2.0 ** -11                 # of products of magnitude 1 to 4


def test_values_of_third_parts():
    v = values_from_third_parts(200, 128)
    p = np.ones((1, 200))
    want = p @ v.astype(np.float64)
    assert np.abs(want).max() < 2.0 ** -11 and np.array_equal(products(p, v), want)
    assert (products(p, v, [(0, 2)]) == 0).all()
