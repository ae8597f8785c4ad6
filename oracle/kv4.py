"""Plain float64 CPU oracle for the 4-bit KV cache and for attention over a
sliding window with sinks.

TEST INFRASTRUCTURE ONLY.  Only the test suite, the package's smoke check and
the benchmark's CPU-baseline / reference leg may import this module.  It
shares no code with the CUDA path and never calls it.

* scale of code e * 8 + m: 2^(e - 15) (1 + m / 8); a value is (u - 8) s with
  u in 0..15.  K: one scale per position and 32 channels; V: one per position.
* writing: NaN counts as 0; the smallest scale with 7 s >= the group's
  largest magnitude (the largest scale if none); u = 8 + clamp(round(x / s),
  -7, 7), ties to even.  All in exact arithmetic (float64 holds it).
* block of 16 positions of one KV head, as bytes: see pack_block.
* attention: the textbook softmax over the visible keys, where a row at
  position p sees a key at t iff t < sinks or p - t < window (window None:
  every key), among the prefix and its ancestors and itself.

Parity status: pinned by the format's closed forms (every scale, every code),
the rounding bound s / 2, byte-level hand-made blocks, and the attention by
the full-window case (= tree_verify.attention_one_sequence) and by dropping
the invisible keys from the inputs.
"""
from __future__ import annotations

import numpy as np

from .tree_verify import _f64, ancestors, depths

GROUP = 32
BLOCK = 16
SCALES = np.array([2.0 ** (c // 8 - 15) * (1 + (c % 8) / 8) for c in range(256)])


def scale_code(amax):
    """Smallest code whose 7 steps reach amax, 255 if none does."""
    for c in range(256):
        if 7 * SCALES[c] >= amax:
            return c
    return 255


def quantise(x, groups):
    """x [..., n] in `groups` groups: (u [..., n] uint8, codes [..., groups] uint8)."""
    x = _f64(x)
    x = np.where(np.isnan(x), 0.0, x)
    g = x.reshape(*x.shape[:-1], groups, x.shape[-1] // groups)
    amax = np.abs(g).max(-1)
    codes = np.minimum(np.searchsorted(7 * SCALES, amax, side="left"), 255)
    q = np.clip(np.rint(g / SCALES[codes][..., None]), -7, 7)      # inf / s is inf: 7 steps
    return (q + 8).astype(np.uint8).reshape(x.shape), codes.astype(np.uint8)


def values(u, codes):
    """The numbers that codes stand for, float64."""
    g = u.astype(np.float64).reshape(*codes.shape, u.shape[-1] // codes.shape[-1]) - 8
    return (g * SCALES[codes][..., None]).reshape(u.shape)


def _word_bytes(u8):
    """Four bytes of eight 4-bit values: value 2 j at bit 4 j, 2 j + 1 at bit 16 + 4 j."""
    w = 0
    for e in range(8):
        w |= int(u8[e]) << (4 * (e // 2) + 16 * (e % 2))
    return [(w >> (8 * i)) & 255 for i in range(4)]


def pack_block(k, v):
    """(K block bytes, V block bytes) of 16 rows [16, d] each."""
    d = k.shape[-1]
    uk, ck = quantise(k, d // GROUP)
    uv, cv = quantise(v, 1)
    kb, vb = [], []
    for c in range(d // GROUP):
        for i in range(BLOCK):
            for w in range(4):
                kb += _word_bytes(uk[i, c * GROUP + w * 8: c * GROUP + w * 8 + 8])
    for c in range(d // GROUP):
        kb += [int(ck[i, c]) for i in range(BLOCK)]
    for ch in range(d):
        vb += _word_bytes(uv[:8, ch]) + _word_bytes(uv[8:, ch])
    vb += [int(x) for x in cv[:, 0]]
    return np.array(kb, dtype=np.uint8), np.array(vb, dtype=np.uint8)


def unpack_block(kb, vb, d):
    """(K [16, d], V [16, d]) float64 of one block's bytes."""
    kb, vb = np.asarray(kb, dtype=np.int64), np.asarray(vb, dtype=np.int64)

    def value(b, at, e, code):
        bit = 4 * (e // 2) + 16 * (e % 2)
        return (((b[at + bit // 8] >> (bit % 8)) & 15) - 8) * SCALES[code]

    k, v = np.zeros((BLOCK, d)), np.zeros((BLOCK, d))
    for i in range(BLOCK):
        for ch in range(d):
            c, e = divmod(ch, GROUP)
            k[i, ch] = value(kb, c * 256 + i * 16 + e // 8 * 4, e % 8, kb[8 * d + c * 16 + i])
            v[i, ch] = value(vb, ch * 8 + i // 8 * 4, i % 8, vb[8 * d + i])
    return k, v


def pack_rows(k, v):
    """[T, d] rows (T a multiple of 16) -> K blocks [T / 16, 8.5 d], V blocks [T / 16, 8 d + 16]."""
    out = [pack_block(k[t:t + BLOCK], v[t:t + BLOCK]) for t in range(0, k.shape[0], BLOCK)]
    return np.stack([a for a, _ in out]), np.stack([b for _, b in out])


def stored(x, groups):
    """x after a write and a read: float64."""
    return values(*quantise(x, groups))


def visible(P, parents, window=None, sinks=0):
    """bool [N, P + N]: what each tree row sees of the prefix positions 0..P-1
    and of the tree's nodes (at positions P + depth)."""
    anc, dep = ancestors(parents), depths(parents)
    N = len(parents)
    vis = np.zeros((N, P + N), dtype=bool)
    for i in range(N):
        for j in list(range(P)) + [P + a for a in anc[i]]:
            t = j if j < P else P + dep[j - P]
            vis[i, j] = window is None or t < sinks or P + dep[i] - t < window
    return vis


def attention(q, k_prefix, v_prefix, k_tree, v_tree, parents, scale, window=None, sinks=0):
    """One sequence: q [N, Hq, d], k/v_prefix [Hkv, P, d], k/v_tree [Hkv, N, d] -> [N, Hq, d] float64."""
    q, kp, vp, kt, vt = (_f64(x) for x in (q, k_prefix, v_prefix, k_tree, v_tree))
    N, Hq, _ = q.shape
    G = Hq // kp.shape[0]
    vis = visible(kp.shape[1], parents, window, sinks)
    out = np.zeros_like(q)
    for h in range(Hq):
        k, v = np.concatenate([kp[h // G], kt[h // G]]), np.concatenate([vp[h // G], vt[h // G]])
        for i in range(N):
            on = vis[i]
            s = scale * (k[on] @ q[i, h])
            w = np.exp(s - s.max())
            out[i, h] = (w @ v[on]) / w.sum()
    return out
