"""Shared pieces of the 4-bit cache's and the windowed attention's tests:
oracle attention of a workload, error bounds derived from the arithmetic, and
the cache's bytes by sequence."""
import numpy as np
import torch

from oracle import kv4
from oracle.tree_verify import _f64, prefix_kv


def cached_prefix(w, b, four_bits):
    """Sequence b's prefix as the attention reads it, [Hkv, P, d] float64."""
    k, v = prefix_kv(w, b)
    if not four_bits:
        return k, v
    return kv4.stored(k, k.shape[-1] // kv4.GROUP), kv4.stored(v, 1)


def reference(w, four_bits, win=None):
    """(out, bound) [R, Hq, d] float64: the oracle's attention and how far a
    correct kernel may be from it, value by value.

    With A = sum_j p_j |v_j| and S the largest sum_c |q_c k_c| * scale:
    * scores: d products and sums in fp32, u = 2^-24 each (2^-22 on the tensor
      cores, whose adder may drop bits of the smaller operand):
      |ds| <= (d + 4) u S, so each weight is off by 2 |ds| relative;
    * exponentials: 2^-21 relative (two units) plus the rounding of a base-2
      exponent of magnitude up to 2 S: 4 u S;
    * sums over n keys in fp32: 2 (n + 8) u relative, again 2^-22 for u on the
      tensor cores, whose tiles add up at most 128 keys each before the split
      is joined: n keys at most;
    * bf16 kernels: weights rounded to bf16 (2^-8 of each p_j |v_j|), partials
      of a split rounded to bf16 (2^-8 of A at most), the result rounded to
      bf16 (2^-8 of |out|)."""
    win_kw = {} if win is None else dict(window=win[0], sinks=win[1])
    outs, bounds = [], []
    bf16 = w.spec.dtype == "bf16"
    u = 2.0 ** -22 if bf16 else 2.0 ** -24
    for b in range(w.batch):
        o0, o1 = w.seq_rows(b)
        kp, vp = cached_prefix(w, b, four_bits)
        q, kt, vt = _f64(w.q[o0:o1]), _f64(w.k_tree[:, o0:o1]), _f64(w.v_tree[:, o0:o1])
        kp, vp = (np.where(np.isfinite(x), x, 0.0) for x in (kp, vp))   # canaries sit where no row sees them
        args = (w.parents[b], w.scale)
        out = kv4.attention(q, kp, vp, kt, vt, *args, **win_kw)
        A = kv4.attention(q, kp, np.abs(vp), kt, np.abs(vt), *args, **win_kw)
        G = q.shape[1] // kp.shape[0]
        allk = np.abs(np.concatenate([kp, kt], 1))
        S = max(float((np.abs(q[:, g * G:(g + 1) * G]).reshape(-1, q.shape[2]) @ allk[g].T).max())
                for g in range(kp.shape[0])) * w.scale
        n = allk.shape[1]
        rel = 2 * (w.spec.d + 6) * u * S + 2.0 ** -21 + 2 * (n + 8) * u
        if bf16:
            rel += 2 * 2.0 ** -8
        bounds.append(rel * A + (2.0 ** -8 * np.abs(out) if bf16 else 2.0 ** -24 * np.abs(out)) + 1e-30)
        outs.append(out)
    return np.concatenate(outs), np.concatenate(bounds)


def check_attn(w, st, four_bits, win=None):
    out, bound = reference(w, four_bits, win)
    got = st.out.double().cpu().numpy()
    assert int(st.status[0]) == 0, f"device status {int(st.status[0])}"
    assert np.isfinite(got).all()
    worst = float((np.abs(got - out) / bound).max())
    assert worst <= 1.0, f"error is {worst} of its bound"
    return worst


def blocks_of(st, b):
    """(K, V) block bytes of sequence b, [Hkv, blocks, bytes] uint8 (CPU)."""
    d, hkv = st.desc.head_dim, st.desc.num_kv_heads
    kb, vb = 8 * d + d // 2, 8 * d + 16
    if st.page_table is None:
        nb = st.desc.capacity // 16
        return (st.k4.view(-1, hkv, nb, kb)[b].cpu(), st.v4.view(-1, hkv, nb, vb)[b].cpu())
    ids = st.page_table[b].long()
    ids = ids[ids >= 0]
    return (st.k4.view(-1, hkv, kb)[ids].transpose(0, 1).cpu(), st.v4.view(-1, hkv, vb)[ids].transpose(0, 1).cpu())


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
