"""What pins the oracle of the 4-bit cache and of the windowed attention (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import kv4


def test_every_scale_and_code():
    assert kv4.SCALES[0] == 2.0 ** -15 and kv4.SCALES[255] == 2.0 ** 16 * 1.875
    assert (np.diff(kv4.SCALES) > 0).all()
    for c in (0, 1, 77, 128, 255):
        u = np.arange(16, dtype=np.uint8)
        assert kv4.values(u[None], np.array([[c]], dtype=np.uint8))[0].tolist() == [(x - 8) * kv4.SCALES[c]
                                                                                   for x in range(16)]
    # 3-bit steps times 4-bit significands fit bf16's 8 bits: no value is rounded
    q, m = np.meshgrid(np.arange(-8, 8), np.arange(8, 16))
    assert np.abs(q * m).max() <= 128


@pytest.mark.parametrize("scale", [1.0, 1e-3, 300.0])
def test_rounding_is_within_half_a_step(scale):
    x = np.random.default_rng(1).standard_normal((40, 128)) * scale
    u, c = kv4.quantise(x, 4)
    err = np.abs(kv4.values(u, c) - x).reshape(40, 4, 32)
    s = kv4.SCALES[c]
    assert (err <= s[..., None] / 2).all()
    amax = np.abs(x).reshape(40, 4, 32).max(-1)
    assert (7 * s >= amax).all() and (7 * kv4.SCALES[np.maximum(c, 1) - 1] < amax)[c > 0].all()


def test_ties_specials_and_borders():
    s = kv4.SCALES[120]                                    # 1.0
    x = np.zeros((1, 32))
    x[0, :8] = [7, 0.5, 1.5, 2.5, -0.5, -3.5, np.nan, 0]
    u, c = kv4.quantise(x, 1)
    assert s == 1.0 and c[0, 0] == 120
    assert (u[0, :8].astype(int) - 8).tolist() == [7, 0, 2, 2, 0, -4, 0, 0]
    assert kv4.scale_code(7.0) == 120 and kv4.scale_code(np.nextafter(7.0, 8)) == 121
    assert kv4.scale_code(0.0) == 0 and kv4.scale_code(np.inf) == 255
    x[0, 1] = -np.inf
    u, c = kv4.quantise(x, 1)
    assert c[0, 0] == 255 and u[0, 1] == 1 and u[0, 0] == 8


def test_block_bytes_by_hand():
    k, v = np.zeros((16, 32)), np.zeros((16, 32))
    k[3, 9] = 7.0                                          # group 0, word 1, value 1 of position 3
    v[9, 5] = -7.0                                         # channel 5, word 1, value 1; position 9's scale
    kb, vb = kv4.pack_block(k, v)
    assert len(kb) == 272 and len(vb) == 272
    assert kb[3 * 16 + 4 + 2] == 0x8F and kb[256 + 3] == 120
    assert vb[5 * 8 + 4 + 2] == 0x81 and vb[256 + 9] == 120
    assert (np.delete(kb[:256], 54) == 0x88).all() and (np.delete(kb[256:], 3) == 0).all()
    k2, v2 = kv4.unpack_block(kb, vb, 32)
    assert (k2 == k).all() and (v2 == v).all()


def test_pack_unpack_round_trip():
    g = np.random.default_rng(3)
    k, v = g.standard_normal((48, 64)), g.standard_normal((48, 64)) * 5
    kb, vb = kv4.pack_rows(k, v)
    for n in range(3):
        k2, v2 = kv4.unpack_block(kb[n], vb[n], 64)
        assert (k2 == kv4.stored(k, 2)[16 * n:16 * n + 16]).all()
        assert (v2 == kv4.stored(v, 1)[16 * n:16 * n + 16]).all()


PARENTS = [-1, 0, 0, 1, 1, 2, 3, 5]


def _inputs(P, seed=0):
    g = np.random.default_rng(seed)
    r = lambda *s: g.standard_normal(s)
    return r(8, 4, 32), r(2, P, 32), r(2, P, 32), r(2, 8, 32), r(2, 8, 32)


def test_full_window_is_plain_tree_attention():
    a = _inputs(50)
    want = oracle.attention_one_sequence(*a, PARENTS, 0.2)
    for win in ({}, dict(window=1000), dict(window=54, sinks=0), dict(window=1, sinks=100)):
        assert np.abs(kv4.attention(*a, PARENTS, 0.2, **win) - want).max() < 1e-12


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 0), (3, 1), (10, 4), (20, 45)])
def test_window_equals_dropping_invisible_keys(window, sinks):
    q, kp, vp, kt, vt = _inputs(50, 1)
    got = kv4.attention(q, kp, vp, kt, vt, PARENTS, 0.2, window, sinks)
    dep = oracle.depths(PARENTS)
    for i in range(8):
        p = 50 + dep[i]
        keep = [t for t in range(50) if t < sinks or t > p - window]
        tree = [a for a in oracle.ancestors(PARENTS)[i] if 50 + dep[a] < sinks or dep[a] > dep[i] - window]
        for h in range(4):
            k = np.concatenate([kp[h // 2][keep], kt[h // 2][tree]])
            v = np.concatenate([vp[h // 2][keep], vt[h // 2][tree]])
            e = np.exp(0.2 * k @ q[i, h])
            assert np.abs(got[i, h] - e @ v / e.sum()).max() < 1e-12
    if window == 1 and not sinks:                          # a row that sees itself alone
        assert np.abs(got - np.repeat(vt.transpose(1, 0, 2), 2, axis=1)).max() < 1e-12
