"""The control of tree logits and the token counts against the oracle (GPU)."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_gb300 as tv
from oracle import logits as ol

pytestmark = pytest.mark.gpu


class Tree:
    def __init__(self, nodes, V, dtype, counted=True, bias=0, mask=True, paths=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.nodes, self.V, B, R = nodes, V, len(nodes), sum(nodes)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.x = (torch.randn(R, V, generator=g) * 3).to(self.dt)
        width = (V + 7) // 8 * 8
        c = torch.randint(0, 6, (B, width), generator=g) * (torch.rand(B, width, generator=g) < 0.1)
        c = c + 0x8000 * (torch.rand(B, width, generator=g) < 0.1)
        self.counts = c.numpy() if counted else None
        self.pen = torch.stack([torch.rand(B, generator=g) + 0.7, torch.randn(B, generator=g), torch.randn(B, generator=g)], 1)
        self.offs = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        few = max(1, min(V, 12))                              # drafts and biases meet often
        self.draft = torch.randint(0, few, (R,), generator=g).to(torch.int32)
        self.parents = []
        anc = []
        for n in nodes:
            par = [-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, n)]
            self.parents.append(par)
            a = []
            for i in range(n):
                a.append(1 << i | (a[par[i]] if i else 0))
            anc += a
        self.anc = torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64)
        self.paths = paths
        self.nb = [bias if b % 3 != 1 else 0 for b in range(B)]
        self.bo = np.concatenate([[0], np.cumsum(self.nb)]).astype(np.int32)
        T = int(self.bo[-1])
        near = torch.randint(0, few, (T,), generator=g)
        self.bt = torch.where(torch.rand(T, generator=g) < 0.5, near, torch.randint(0, V, (T,), generator=g)).to(torch.int32)
        self.bv = torch.randn(T, generator=g)
        words = (V + 31) // 32
        self.mask = torch.randint(-2 ** 31, 2 ** 31, (R, words), generator=g).to(torch.int32) if mask else None
        if mask:
            self.mask[0] = 0                                  # a row with nothing allowed
            self.mask[-1] = -1
        self.desc = tv.make_logits_desc(batch=B, vocab=V, max_nodes=max(nodes), total_rows=R,
                                        logits_dtype=tv.BF16 if dtype == "bf16" else tv.F32, biases=T)
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def run(self, inplace=False, stream=None, logits=None):
        to = lambda x: None if x is None else (torch.as_tensor(x)).cuda()
        x = self.x.cuda() if logits is None else logits
        out = x if inplace else torch.full_like(x, 5.0)
        counts = None if self.counts is None else torch.tensor(self.counts.astype(np.uint16).view(np.int16)).cuda()
        bias = [to(self.bo), to(self.bt), to(self.bv)] if self.bo[-1] > 0 else [None] * 3
        path = [to(self.draft), to(self.anc)] if self.paths else [None, None]
        keep = [to(self.pen) if counts is not None else None, to(self.mask), to(self.offs)]
        torch.cuda.synchronize()
        tv.tv_tree_logits_process(self.desc, x, counts, keep[0], *bias, keep[1], path[0], keep[2], path[1], out,
                                  self.status, stream)
        torch.cuda.synchronize()
        return out.cpu()

    def expected(self):
        out = np.zeros((len(self.x), self.V))
        for b, n in enumerate(self.nodes):
            for i in range(n):
                r = self.offs[b] + i
                path = ol.path_drafts(self.parents[b], self.draft[self.offs[b]:], i) if self.paths else []
                sl = slice(self.bo[b], self.bo[b + 1])
                out[r] = ol.process_row(self.x[r].double().numpy(), None if self.counts is None else self.counts[b, :self.V],
                                        None if self.counts is None else self.pen[b].tolist(),
                                        (self.bt[sl].tolist(), self.bv[sl].tolist()) if self.nb[b] else None,
                                        None if self.mask is None else self.mask[r].numpy().view(np.uint32), path)
        return out

    def check(self, got):
        """Five fp32 roundings of values no larger than the terms' sum, then the type's half step."""
        want = self.expected()
        got = got.double().numpy()
        assert np.array_equal(np.isneginf(want), np.isneginf(got))
        fin = np.isfinite(want)
        top = float(np.abs(self.x.double().numpy()[np.isfinite(self.x.double().numpy())]).max())
        size = 2 * top + 80 * float(self.pen.abs().max()) + (float(self.bv.abs().max()) if len(self.bv) else 0)
        half = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -24
        lim = 6 * 2.0 ** -24 * size + half * np.abs(want[fin])
        assert (np.abs(got[fin] - want[fin]) <= lim).all()
        untouched = (got == self.x.double().numpy())
        return untouched


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 8, 31, 32, 33, 1000, 2047, 2048, 2049, 4104, 5003])
def test_vocabularies(V, dtype):
    t = Tree([5, 1, 17], V, dtype, bias=9, seed=V)
    t.check(t.run())
    assert int(t.status[0]) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [2056, 2051])
@pytest.mark.parametrize("counted,bias,mask,paths", [(False, 0, False, False), (True, 0, False, False),
                                                     (True, 0, False, True), (False, 5, False, True),
                                                     (False, 0, True, False), (True, 700, True, True)])
def test_parts(V, dtype, counted, bias, mask, paths):
    t = Tree([64, 3], V, dtype, counted, bias, mask, paths, seed=bias)
    t.check(t.run())
    t.check(t.run(inplace=True))


@pytest.mark.parametrize("V", [40000, 40001])
def test_many_rows(V):
    """Several rows a CTA: paths come and go from row to row."""
    t = Tree([64, 1, 2, 33, 64, 64, 64, 7], V, "bf16", bias=40, seed=2)
    t.check(t.run())


def test_specials():
    t = Tree([3], 64, "f32", bias=4, seed=3)
    t.mask[:] = -1
    t.x[1, 5], t.x[1, 6], t.x[2, 7] = float("nan"), float("-inf"), float("inf")
    got = t.run()
    assert torch.isnan(got[1, 5]) and got[1, 6] == float("-inf") and got[2, 7] == float("inf")


def test_rows_of_bad_offsets_keep_their_contents():
    t = Tree([4, 4, 4], 300, "f32", seed=4)
    good = t.run()
    t.offs = np.array([0, 4, 3, 12], np.int32)
    got = t.run()
    assert int(t.status[0]) == 2
    assert torch.equal(got[:4], good[:4]) and (got[4:] == 5.0).all()


def test_bad_tokens_and_biases():
    t = Tree([4, 1], 300, "f32", bias=6, mask=False, seed=5)
    t.bt[1], t.bt[2] = -1, 300
    t.check(t.run())
    assert int(t.status[0]) == 256
    t = Tree([4, 1], 300, "f32", bias=6, mask=False, seed=5)
    t.bo = np.array([0, 7, 6], np.int32)
    t.run()
    assert int(t.status[0]) == 2
    t = Tree([4], 300, "f32", seed=6)
    t.draft[2], t.draft[3] = -7, 300
    t.check(t.run())
    assert int(t.status[0]) == 0


@pytest.mark.parametrize("V", [10, 1001, 40000])
def test_counts(V):
    g = torch.Generator().manual_seed(V)
    B, width = 5, (V + 7) // 8 * 8
    desc = tv.make_logits_desc(batch=B, vocab=V, max_nodes=1, total_rows=B, logits_dtype=tv.F32)
    counts = torch.zeros(B, width, dtype=torch.int16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    want = np.zeros((B, width), np.int64)
    lens = [0, 1, 300, 5000, 64]
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    toks = (torch.rand(int(offs[-1]), generator=g) ** 6 * V).to(torch.int32).clamp(max=V - 1)
    toks[2] = -1
    for prompt in (True, False, False):
        tv.tv_token_counts_add(desc, toks.cuda(), torch.tensor(offs).cuda(), len(toks), prompt, counts, status)
        for b in range(B):
            want[b] = ol.add_counts(want[b], toks[offs[b]:offs[b + 1]].tolist(), prompt)
    rows = torch.randint(-1, V, (B, 33), generator=g).to(torch.int32)
    tv.tv_token_counts_add(desc, rows.cuda(), None, 33, False, counts, status)
    for b in range(B):
        want[b] = ol.add_counts(want[b], rows[b].tolist(), False)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    assert np.array_equal(counts.cpu().numpy().view(np.uint16).astype(np.int64), want)


def test_counts_saturate_and_leave_their_neighbours():
    V = 16
    desc = tv.make_logits_desc(batch=1, vocab=V, max_nodes=1, total_rows=1, logits_dtype=tv.F32)
    counts = torch.zeros(1, V, dtype=torch.int16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    toks = torch.full((40000,), 3, dtype=torch.int32)
    toks[::10] = 2
    for _ in range(2):
        tv.tv_token_counts_add(desc, toks.cuda(), None, 40000, False, counts, status)
    bad = torch.tensor([16, 5, -3, 1 << 30], dtype=torch.int32).cuda()
    tv.tv_token_counts_add(desc, bad, None, 4, True, counts, status)
    tv.tv_token_counts_add(desc, bad, torch.tensor([0, 5], dtype=torch.int32).cuda(), 4, True, counts, status)
    torch.cuda.synchronize()
    assert int(status[0]) == 256 | 2
    want = [0] * V
    want[2], want[3], want[5] = 8000, 32767, -32768
    assert counts[0].tolist() == want
