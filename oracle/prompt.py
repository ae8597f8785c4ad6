"""Plain float64 CPU oracle for the prompt's calls: RoPE with the writes of
keys and values, and causal attention of packed rows over a committed prefix.

TEST INFRASTRUCTURE ONLY.  Only the test suite, the package's smoke check and
the benchmark's CPU-baseline / reference leg may import this module.  It
shares no code with the CUDA path and never calls it.

Parity status: pinned by the chain form of the tree oracle (a chain of rows
with the same prefix), by chunking (a prompt in pieces equals the whole), by
one-row closed forms, and the rotation by oracle.rope's complex form.
"""
from __future__ import annotations

import numpy as np


def attention(q, k_past, v_past, k_rows, v_rows, scale):
    """Rows of one sequence: q [n, Hq, d], past [Hkv, P, d], rows [Hkv, n, d].
    Row i sees the past and rows 0 .. i.  [n, Hq, d] float64."""
    q, k_past, v_past, k_rows, v_rows = (np.asarray(x, np.float64) for x in (q, k_past, v_past, k_rows, v_rows))
    n, hq, d = q.shape
    G = hq // k_rows.shape[0]
    P = k_past.shape[1]
    out = np.zeros((n, hq, d))
    hidden = np.arange(P + n) > P + np.arange(n)[:, None]
    for h in range(hq):
        k = np.concatenate([k_past[h // G], k_rows[h // G]])
        v = np.concatenate([v_past[h // G], v_rows[h // G]])
        s = np.where(hidden, -np.inf, q[:, h] @ k.T * scale)
        w = np.exp(s - s.max(1, keepdims=True))
        out[:, h] = w / w.sum(1, keepdims=True) @ v
    return out


def positions(prefix_len, row_offsets):
    """Position of every packed row."""
    return np.concatenate([p + np.arange(b - a) for p, a, b in
                           zip(prefix_len, row_offsets[:-1], row_offsets[1:])] or [np.zeros(0, int)])


def rotate(x, pos, theta):
    """x [rows, heads, d] turned at the rows' positions, float64."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    a = np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)
