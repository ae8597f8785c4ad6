"""Pins of the prompt oracle and of the logits oracle (CPU)."""
import numpy as np
import pytest

from oracle import kv4, logits as ol, prompt as op


def _case(P, n, hq, hkv, d, seed=0):
    g = np.random.default_rng(seed)
    return [g.standard_normal(s) for s in ((n, hq, d), (hkv, P, d), (hkv, P, d), (hkv, n, d), (hkv, n, d))]


@pytest.mark.parametrize("P,n,hq,hkv", [(0, 7, 4, 2), (9, 5, 3, 1), (16, 1, 2, 2)])
def test_attention_is_a_chain_of_tree_rows(P, n, hq, hkv):
    q, kp, vp, kr, vr = _case(P, n, hq, hkv, 8)
    chain = kv4.attention(q, kp, vp, kr, vr, [-1] + list(range(n - 1)), 0.3)
    np.testing.assert_allclose(op.attention(q, kp, vp, kr, vr, 0.3), chain, rtol=0, atol=1e-13)


def test_chunks_equal_the_whole():
    q, kp, vp, kr, vr = _case(5, 12, 4, 2, 8, 1)
    whole = op.attention(q, kp, vp, kr, vr, 0.4)
    second = op.attention(q[7:], np.concatenate([kp, kr[:, :7]], 1), np.concatenate([vp, vr[:, :7]], 1), kr[:, 7:],
                          vr[:, 7:], 0.4)
    np.testing.assert_allclose(whole[7:], second, rtol=0, atol=1e-13)


def test_first_row_without_a_prefix_is_its_own_value():
    q, kp, vp, kr, vr = _case(0, 3, 4, 2, 8, 2)
    np.testing.assert_allclose(op.attention(q, kp, vp, kr, vr, 1.0)[0], vr[[0, 0, 1, 1], 0], atol=1e-15)


def test_rotation_and_positions():
    pos = op.positions([5, 0, 100], [0, 3, 3, 5])
    assert pos.tolist() == [5, 6, 7, 100, 101]
    x = np.random.default_rng(3).standard_normal((5, 2, 8))
    y = op.rotate(x, pos, 1e4)
    z = (x[..., :4] + 1j * x[..., 4:]) * np.exp(1j * pos[:, None, None] * 1e4 ** (-np.arange(4) / 4))
    np.testing.assert_allclose(y, np.concatenate([z.real, z.imag], -1), atol=1e-12)
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))


def test_counts():
    c = np.zeros(6, np.int64)
    c = ol.add_counts(c, [1, 1, 4, -1, 9], True)
    c = ol.add_counts(c, [1, 2, 2, -1], False)
    assert c.tolist() == [0, 0x8001, 2, 0, 0x8000, 0]
    c[3] = ol.MOST - 1
    assert ol.add_counts(c, [3, 3, 3], False)[3] == ol.MOST


def test_every_rule_by_hand():
    x = np.array([2.0, -2.0, 3.0, 0.5, 1.0, -1.0])
    counts = np.array([0, 0x8000, 2, 0x8003, 0, 0])
    y = ol.process_row(x, counts, (2.0, 0.25, 0.5), ([4, 4, 9, 0], [5.0, 7.0, 1.0, -1.0]), None, [5, 5, 2])
    assert y.tolist() == [1.0, -4.0, 1.5 - 0.75 - 0.5, 0.25 - 0.75 - 0.5, 8.0, -2.0 - 0.5 - 0.5]
    z = ol.process_row(x, counts, None, None, np.array([0b010110], np.uint32), [])
    assert z.tolist() == [-np.inf, -2.0, 3.0, -np.inf, 1.0, -np.inf]


def test_a_tree_row_is_plain_decoding_after_its_path():
    g = np.random.default_rng(4)
    parents, draft = [-1, 0, 0, 1, 3, 2], [8, 3, 5, 3, 1, 0]
    base = ol.add_counts(np.zeros(10, np.int64), [8, 2], False)
    x = g.standard_normal(10)
    for row in range(6):
        path = ol.path_drafts(parents, draft, row)
        after = ol.add_counts(base, path, False)
        np.testing.assert_array_equal(ol.process_row(x, base, (1.3, 0.1, 0.2), None, None, path),
                                      ol.process_row(x, after, (1.3, 0.1, 0.2), None, None, []))
    assert ol.path_drafts(parents, draft, 4) == [1, 3, 3] and ol.path_drafts(parents, draft, 0) == []
