"""Plain float64 CPU oracle for the control of tree logits: token counts,
penalties, biases and masks.

TEST INFRASTRUCTURE ONLY.  Only the test suite, the package's smoke check and
the benchmark's CPU-baseline / reference leg may import this module.  It
shares no code with the CUDA path and never calls it.

Parity status: pinned by hand-made cases of every rule and by a step-by-step
decoder (a tree row's steered logits equal those of plain decoding after its
path).
"""
from __future__ import annotations

import numpy as np

PROMPT, MOST = 0x8000, 0x7FFF


def add_counts(counts, tokens, prompt):
    """One sequence's counts [V] (int) after its tokens; negative ones are padding."""
    counts = counts.copy()
    for t in tokens:
        if t < 0 or t >= counts.shape[0]:
            continue
        if prompt:
            counts[t] |= PROMPT
        elif counts[t] & MOST != MOST:
            counts[t] += 1
    return counts


def path_drafts(parents, draft, row):
    """Draft tokens from below the root to `row`."""
    out = []
    while row > 0:
        out.append(int(draft[row]))
        row = int(parents[row])
    return out


def process_row(x, counts, penalties, bias, mask_words, path):
    """x [V]: one row.  penalties (rho, phi, pi) or None; bias: (tokens, values)
    or None; mask_words uint32 or None; path: drafts counted for this row."""
    x = np.array(x, np.float64)
    V = x.shape[0]
    if penalties is not None:
        rho, phi, pi = (float(v) for v in penalties)
        n = (counts & MOST).astype(np.float64)
        for t in path:
            if 0 <= t < V:
                n[t] += 1
        seen = ((counts & PROMPT) != 0) | (n > 0)
        with np.errstate(invalid="ignore"):
            x = np.where(seen, np.where(x > 0, x / rho, x * rho), x) - phi * n - pi * (n > 0)
    if bias is not None:
        last = {int(t): float(v) for t, v in zip(*bias) if 0 <= t < V}
        for t, v in last.items():
            x[t] += v
    if mask_words is not None:
        for v in range(V):
            if not int(mask_words[v // 32]) >> (v % 32) & 1:
                x[v] = -np.inf
    return x
