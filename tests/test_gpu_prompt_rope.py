"""Prompt RoPE and its writes against the float64 oracle (GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from oracle import prompt as op

pytestmark = pytest.mark.gpu
PAGE = 16


class Rows:
    def __init__(self, p, n, hq, hkv, d, dtype, paged=False, pad=0, cap=None, cache=True, rows=True, seed=0,
                 max_prefix=None):
        g = torch.Generator().manual_seed(seed)
        self.p, self.n, self.hq, self.hkv, self.d, self.paged = p, n, hq, hkv, d, paged
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        B, R = len(p), sum(n)
        self.R = R + pad
        self.cap = cap or (max(a + b for a, b in zip(p, n)) // PAGE + 2) * PAGE
        rnd = lambda *s: torch.randn(*s, generator=g).to(self.dt)
        self.q, self.k, self.v = rnd(self.R, hq, d).cuda(), rnd(self.R, hkv, d).cuda(), rnd(self.R, hkv, d).cuda()
        cols = self.cap // PAGE
        pages = B * cols + 2
        self.table = torch.randperm(pages, generator=g)[:B * cols].reshape(B, cols).to(torch.int32).cuda() if paged else None
        pool = (pages, hkv, PAGE, d) if paged else (B, hkv, self.cap, d)
        self.caches = [rnd(*pool).cuda() for _ in range(2)] if cache else [None, None]
        self.before = [x.clone() if cache else None for x in self.caches]
        self.rows = [torch.full((hkv, self.R, d), 3.0, dtype=self.dt, device="cuda") for _ in range(2)] if rows else [None] * 2
        self.q_out = torch.full_like(self.q, 3.0)
        self.prefix = torch.tensor(p, dtype=torch.int32).cuda()
        self.offs = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.offsets = torch.tensor(self.offs).cuda()
        self.new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.desc = tv.make_desc(batch=B, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                 dtype=tv.BF16 if dtype == "bf16" else tv.F32, max_nodes=1, total_rows=B,
                                 capacity=self.cap, max_prefix=max(p) if max_prefix is None else max_prefix,
                                 page_size=PAGE if paged else 0, num_pages=pages if paged else 0)

    def run(self, theta=1e4, q_out=None, new=True, stream=None):
        tv.tv_prompt_rope_store(self.desc, self.R, max(max(self.n), 1), theta, self.q, self.k, self.v, self.prefix,
                                self.offsets, self.q_out if q_out is None else q_out, *self.rows, *self.caches,
                                self.table, self.new if new else None, self.status, stream)
        torch.cuda.synchronize()

    def check(self, q0, theta=1e4, skipped=()):
        """Turned values within half a step of their type and fp32 rounding; values, lengths and all else equal."""
        pos = op.positions(self.p, self.offs)
        # rotation in fp32 of exact inputs: two products and a sum (2^-24 each of |lo| + |hi|) with sine and cosine
        # each off by at most 2^-22, then the type's half step
        half = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        live = np.concatenate([np.full(m, b not in skipped) for b, m in enumerate(self.n)] + [np.zeros(self.R - len(pos), bool)])
        pos = np.concatenate([pos, np.zeros(self.R - len(pos))])

        def near(got, x):
            x = x.double().cpu().numpy()
            want = op.rotate(x, pos, theta)
            d2 = self.d // 2
            size = np.abs(x[..., :d2]) + np.abs(x[..., d2:])
            lim = np.concatenate([size, size], -1) * (3 * 2.0 ** -24 + 2.0 ** -22) + half * np.abs(want) + 1e-30
            got = got.double().cpu().numpy()
            bad = np.abs(got[live] - want[live]) / lim[live]
            assert not bad.size or bad.max() <= 1, bad.max()

        near(self.q_out, q0)
        assert (self.q_out[torch.tensor(~live).cuda()] == 3.0).all()
        lt = torch.tensor(live).cuda()
        if self.rows[0] is not None:
            near(self.rows[0].transpose(0, 1), self.k)
            assert torch.equal(self.rows[1][:, lt], self.v.transpose(0, 1)[:, lt])
            assert (self.rows[0][:, ~lt] == 3.0).all() and (self.rows[1][:, ~lt] == 3.0).all()
        if self.caches[0] is not None:
            at = [x.clone() for x in self.before]
            r = 0
            for b, m in enumerate(self.n):
                for i in range(m):
                    t = self.p[b] + i
                    if b not in skipped:
                        krow = self.rows[0][:, r] if self.rows[0] is not None else None
                        for kind, src in ((0, krow), (1, self.v[r])):
                            sl = (int(self.table[b, t // PAGE]), slice(None), t % PAGE) if self.paged else (b, slice(None), t)
                            at[kind][sl] = self.caches[0][sl] if src is None else src
                    r += 1
            for x, y in zip(self.caches, at):
                assert torch.equal(x, y)
        assert self.new.tolist() == [p + (0 if b in skipped else m) for b, (p, m) in enumerate(zip(self.p, self.n))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (5, 1, 256), (4, 4, 512), (1, 1, 128), (64, 8, 128)])
def test_rows_and_cache(hq, hkv, d, paged, dtype):
    c = Rows([0, 17, 300, 5, 31], [1, 33, 0, 15, 16], hq, hkv, d, dtype, paged, pad=3, seed=d)
    c.run(1e6)
    assert int(c.status[0]) == 0
    c.check(c.q, 1e6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_far_positions_and_in_place(dtype):
    c = Rows([100000, 3], [700, 900], 4, 2, 128, dtype, paged=True, seed=1)
    q0 = c.q.clone()
    c.run(1e4, q_out=c.q)
    c.q_out = c.q
    assert int(c.status[0]) == 0
    c.check(q0)


def test_positions_near_the_last():
    """Angles at positions near 2^31 (the packed rows alone; no cache)."""
    c = Rows([2 ** 31 - 100], [64], 2, 1, 128, "f32", cache=False, cap=2 ** 31 - 16, seed=2)
    c.run(1e4)
    assert int(c.status[0]) == 0
    # the fraction of a turn a position times is off by at most 2^-52 relative: 2^31 * 0.16 * 2^-52 turns
    pos = op.positions(c.p, c.offs)
    want = op.rotate(c.q.double().cpu().numpy(), pos, 1e4)
    assert np.abs(c.q_out.double().cpu().numpy() - want).max() < 5e-6


@pytest.mark.parametrize("rows,cache", [(True, False), (False, True)])
def test_one_kind_of_output(rows, cache):
    c = Rows([9, 0], [20, 40], 4, 2, 128, "bf16", rows=rows, cache=cache)
    c.run()
    c.check(c.q)


def test_without_new_lengths():
    c = Rows([9], [20], 4, 2, 128, "bf16")
    c.run(new=False)
    assert c.new.tolist() == [-9]


@pytest.mark.parametrize("paged", [False, True])
def test_device_faults(paged):
    # what does not fit is skipped whole
    c = Rows([5, 60, 3], [10, 5, 0], 4, 2, 128, "bf16", paged, cap=64)
    c.run()
    assert int(c.status[0]) == 16
    c.check(c.q, skipped=(1,))
    # a prefix length out of range: skipped with a cache
    c = Rows([5, 6], [10, 5], 4, 2, 128, "bf16", paged)
    c.prefix[1] = -3
    c.run()
    assert int(c.status[0]) == 4 and c.new.tolist() == [15, -3]
    c.new[1] = 6
    c.check(c.q, skipped=(1,))
    # bad offsets
    c = Rows([5, 6], [10, 5], 4, 2, 128, "bf16", paged)
    c.offsets.copy_(torch.tensor([0, 40, 15], dtype=torch.int32))
    c.run()
    assert int(c.status[0]) == 2 and c.new.tolist() == [5, 6] and (c.q_out == 3.0).all()
    if paged:
        c = Rows([0, 6], [32, 5], 4, 2, 128, "bf16", True)
        c.table[0, 1] = 10 ** 6
        c.run()
        assert int(c.status[0]) == 8
        assert torch.equal(c.rows[1], c.v.transpose(0, 1)) and c.new.tolist() == [32, 11]


def test_clamped_without_a_cache():
    c = Rows([50], [4], 2, 1, 128, "f32", cache=False)
    c.prefix.fill_(10 ** 6)
    c.run()
    assert int(c.status[0]) == 4 and c.new.tolist() == [54]
    c.check(c.q)
