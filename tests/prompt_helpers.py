"""Shared pieces of the prompt tests: packed sequences on the GPU, the oracle's
attention of them and how far a correct kernel may be from it."""
import numpy as np
import torch

import speculative_decoding_tree_gb300 as tv
from oracle import prompt as op

PAGE = 16


class Prompts:
    """B sequences of n[b] rows behind p[b] cached positions, on the GPU; what no row may see is NaN."""

    def __init__(self, p, n, hq, hkv, d, dtype, paged=False, pad=0, seed=0, scale=0.0, out_f32=False, amp=1.0,
                 max_rows=None, max_prefix=None):
        g = torch.Generator().manual_seed(seed)
        self.p, self.n, self.hq, self.hkv, self.d = list(p), list(n), hq, hkv, d
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.bf16 = dtype == "bf16"
        B, R = len(p), sum(n)
        self.R = R + pad
        cap = (max(a + b for a, b in zip(p, n)) // PAGE + 2) * PAGE
        rnd = lambda *s: (torch.randn(*s, generator=g) * amp).to(self.dt)
        self.q = rnd(self.R, hq, d)
        self.k_rows, self.v_rows = rnd(hkv, self.R, d), rnd(hkv, self.R, d)
        self.k_rows[:, R:], self.v_rows[:, R:], self.q[R:] = float("nan"), float("nan"), float("nan")
        k, v = rnd(B, hkv, cap, d), rnd(B, hkv, cap, d)
        for b in range(B):
            k[b, :, p[b]:], v[b, :, p[b]:] = float("nan"), float("nan")
        self.past = [(k[b, :, :p[b]], v[b, :, :p[b]]) for b in range(B)]
        self.table = None
        pages = 0
        if paged:
            cols = cap // PAGE
            pages = B * cols + 3
            ids = torch.randperm(pages, generator=g)[:B * cols].reshape(B, cols)
            kp, vp = (torch.full((pages, hkv, PAGE, d), float("nan"), dtype=self.dt) for _ in range(2))
            for x, y in ((kp, k), (vp, v)):
                x[ids.flatten()] = y.reshape(B, hkv, cols, PAGE, d).transpose(1, 2).flatten(0, 1)
            k, v = kp, vp
            self.table = ids.to(torch.int32).cuda()
        self.k_cache, self.v_cache = k.cuda(), v.cuda()
        self.offsets_cpu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.offsets, self.prefix = torch.tensor(self.offsets_cpu).cuda(), torch.tensor(p, dtype=torch.int32).cuda()
        self.max_rows = max(max(n), 1) if max_rows is None else max_rows
        self.desc = tv.make_desc(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                 dtype=tv.BF16 if self.bf16 else tv.F32, max_nodes=1, total_rows=B, capacity=cap,
                                 max_prefix=max(p) if max_prefix is None else max_prefix,
                                 page_size=PAGE if paged else 0, num_pages=pages, out_f32=int(out_f32), scale=scale)
        self.scale = scale or d ** -0.5
        self.out_f32 = out_f32 or not self.bf16
        self.gpu = [x.cuda() for x in (self.q, self.k_rows, self.v_rows)]
        self.out = torch.full((self.R, hq, d), 7.0, dtype=torch.float32 if self.out_f32 else self.dt, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.ws_bytes = tv.tv_prompt_workspace_size(self.desc, self.R, self.max_rows)
        self.ws = torch.full((max(256, self.ws_bytes),), 0xFF, dtype=torch.uint8, device="cuda")

    def plan(self):
        return tv.tv_prompt_attn_plan(self.desc, self.R, self.max_rows)

    def attn(self, stream=None):
        q, k, v = self.gpu
        tv.tv_prompt_attn(self.desc, self.R, self.max_rows, q, self.k_cache, self.v_cache, self.table, self.prefix,
                          self.offsets, k, v, self.out, self.ws, self.ws_bytes, self.status, stream)

    def seq(self, b):
        o, e = self.offsets_cpu[b], self.offsets_cpu[b + 1]
        f = lambda x: x.double().numpy()
        return f(self.q[o:e]), f(self.past[b][0]), f(self.past[b][1]), f(self.k_rows[:, o:e]), f(self.v_rows[:, o:e])

    def check(self, status=0):
        """Every row within its bound, the padding as it was."""
        torch.cuda.synchronize()
        assert int(self.status[0]) == status, f"device status {int(self.status[0])}"
        got = self.out.double().cpu().numpy()
        worst = 0.0
        for b in range(len(self.n)):
            if self.n[b] == 0:
                continue
            o, e = self.offsets_cpu[b], self.offsets_cpu[b + 1]
            ref, lim = reference(*self.seq(b), self.scale, self.bf16, self.out_f32)
            assert np.isfinite(got[o:e]).all(), f"sequence {b}"
            worst = max(worst, float((np.abs(got[o:e] - ref) / lim).max()))
        assert worst <= 1.0, f"error is {worst} of its bound"
        assert (got[self.offsets_cpu[-1]:] == 7.0).all(), "padding rows written"
        return worst


def reference(q, kp, vp, kr, vr, scale, bf16, out_f32):
    """(out, bound): the oracle's rows and how far a correct kernel may be, value by value.

    With A = sum_j p_j |v_j| and S the largest sum_c |q_c k_c| * scale:
    * scores: d products and sums in fp32, u = 2^-24 each (2^-22 on the tensor cores, whose adder may drop bits of the
      smaller operand): |ds| <= (d + 4) u S, so each weight is off by 2 |ds| relative;
    * exponentials: 2^-21 relative (two units, and a rounded base-2 exponent of magnitude up to 2 S: 4 u S);
    * sums over n keys in fp32: 2 (n + 8) u relative;
    * bf16: each weight rounded (2^-8 of p_j |v_j|), the result rounded to its type (2^-8 or 2^-24 of |out|)."""
    out = op.attention(q, kp, vp, kr, vr, scale)
    A = op.attention(q, kp, np.abs(vp), kr, np.abs(vr), scale)
    G = q.shape[1] // kr.shape[0]
    keys = np.abs(np.concatenate([kp, kr], 1))
    S = max(float((np.abs(q[:, g * G:(g + 1) * G]).reshape(-1, q.shape[2]) @ keys[g].T).max())
            for g in range(kr.shape[0])) * scale
    u = 2.0 ** -22 if bf16 else 2.0 ** -24
    rel = 2 * (q.shape[2] + 6) * u * S + 2.0 ** -21 + 2 * (keys.shape[1] + 8) * u + (2.0 ** -8 if bf16 else 0.0)
    return out, rel * A + (2.0 ** -24 if out_f32 else 2.0 ** -8) * np.abs(out) + 1e-30
