"""Device-resident buffers for one verify workload and the C-ABI calls of a
verify step, in stream order: tree mask, attention, accept + commit; and the
same for one dynamic draft-tree expansion (DeviceExpand).

Used by the benchmark, the GPU tests and the smoke check.  It only moves a
workload's tensors to the GPU, allocates the outputs and workspace with
torch, and calls the library; it computes nothing itself.
"""
from __future__ import annotations

import contextlib

import torch

from . import (BF16, F32, make_desc, make_expand_desc, tree_accept_commit, tree_accept_commit_sampled,
               tree_verify_attn, tv_attn_merge, tv_attn_partials, tv_build_tree_mask, tv_expand_steps,
               tv_expand_workspace_size, tv_tree_expand_step, tv_workspace_size, make_lmhead_desc,
               tv_lm_head_argmax, tv_lm_head_workspace_size, tree_accept_commit_argmax,
               make_window, tree_verify_attn_window, tv_window_workspace_size, tree_verify_attn_kv4,
               tree_accept_commit_argmax_kv4, tv_kv4_append, tv_kv4_cache_bytes, tv_kv4_read, tv_kv4_workspace_size,
               tv_attn_plan, tv_kv4_attn_plan, tv_window_attn_plan, tv_prompt_attn, tv_prompt_rope_store,
               tv_prompt_workspace_size, make_logits_desc, tv_token_counts_add, tv_tree_logits_process)

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _torch_stream(stream):
    return torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream


def _on(stream):
    """A context in which torch allocates and copies on `stream` (None: the current one)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(_torch_stream(stream))


def _keep(stream, *tensors):
    """The tensors' memory is not given on before `stream` has passed this point
    (None and addresses: nothing of torch's to keep)."""
    if stream is not None:
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(_torch_stream(stream))


class DeviceStep:
    def __init__(self, w, device="cuda", out_f32=False, max_prefix=None, vocab=None, max_nodes=None):
        self.w = w
        dev = torch.device(device)
        self.device = dev
        sp = w.spec
        self.dtype = _DT[w.q.dtype]
        self.logits_dtype = _DT[w.logits.dtype]
        self.vocab = vocab if vocab is not None else w.logits.shape[1]
        mp = int(w.prefix_len.max()) if max_prefix is None else int(max_prefix)
        self.desc = make_desc(
            batch=sp.batch, num_q_heads=sp.hq, num_kv_heads=sp.hkv, head_dim=sp.d, dtype=self.dtype,
            max_nodes=w.max_nodes if max_nodes is None else int(max_nodes), total_rows=w.total_rows, capacity=w.capacity, max_prefix=mp,
            page_size=16 if w.page_table is not None else 0,
            num_pages=w.k_cache.shape[0] if w.page_table is not None else 0,
            out_f32=int(out_f32))
        to = lambda t: None if t is None else t.to(dev).contiguous()
        self.q, self.k_tree, self.v_tree = to(w.q), to(w.k_tree), to(w.v_tree)
        self.page_table = to(w.page_table)
        self.prefix_len = to(w.prefix_len)
        self.node_offsets = to(w.node_offsets)
        self.parents = to(w.parents_flat)
        self.logits = to(w.logits)
        self.draft = to(w.draft_tokens) if w.draft_tokens is not None else None
        R, B, mn = w.total_rows, sp.batch, self.desc.max_nodes
        self.anc = torch.zeros(R, dtype=torch.int64, device=dev)
        self.depth = torch.zeros(R, dtype=torch.int32, device=dev)
        odt = torch.float32 if (self.dtype == F32 or out_f32) else torch.bfloat16
        self.out = torch.zeros(R, sp.hq, sp.d, dtype=odt, device=dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.argmax = torch.zeros(R, dtype=torch.int32, device=dev)
        self.accept_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.path = torch.zeros(B, mn, dtype=torch.int32, device=dev)
        self.tokens = torch.zeros(B, mn, dtype=torch.int32, device=dev)
        self._buffers(to)

    def _buffers(self, to):
        """The cache and the calls' workspace."""
        self.k_cache, self.v_cache = to(self.w.k_cache), to(self.w.v_cache)
        self.ws_bytes, self.workspace = self._workspace(tv_workspace_size(self.desc, self.vocab))

    def _workspace(self, size):
        return size, torch.empty(max(size, 256), dtype=torch.uint8, device=self.device)

    # one call each ------------------------------------------------------
    def mask(self, stream=None):
        tv_build_tree_mask(self.desc, self.parents, self.node_offsets, self.anc, self.depth, self.status, stream)

    def attn(self, stream=None):
        tree_verify_attn(self.desc, self.q, self.k_cache, self.v_cache, self.page_table, self.prefix_len,
                         self.node_offsets, self.k_tree, self.v_tree, self.anc, self.out, self.workspace,
                         self.ws_bytes, self.status, stream)

    def partials(self, stream=None):
        tv_attn_partials(self.desc, self.q, self.k_cache, self.v_cache, self.page_table, self.prefix_len,
                         self.node_offsets, self.k_tree, self.v_tree, self.anc, self.workspace, self.ws_bytes,
                         self.status, stream)

    def merge(self, stream=None):
        tv_attn_merge(self.desc, self.prefix_len, self.node_offsets, self.out, self.workspace, self.ws_bytes,
                      self.status, stream)

    def accept_commit(self, stream=None):
        tree_accept_commit(self.desc, self.vocab, self.logits_dtype, self.logits, self.draft, self.parents,
                           self.node_offsets, self.k_tree, self.v_tree, self.k_cache, self.v_cache,
                           self.page_table, self.prefix_len, self.argmax, self.accept_len, self.path,
                           self.tokens, self.workspace, self.ws_bytes, self.status, stream)

    def accept_commit_sampled(self, temperature, seed, offset, stream=None):
        """Sampled verification: one draw per tree row (written to self.argmax),
        then the same walk and commit."""
        tree_accept_commit_sampled(self.desc, self.vocab, self.logits_dtype, self.logits, temperature, seed, offset,
                                   self.draft, self.parents, self.node_offsets, self.k_tree, self.v_tree,
                                   self.k_cache, self.v_cache, self.page_table, self.prefix_len, self.argmax,
                                   self.accept_len, self.path, self.tokens, self.workspace, self.ws_bytes,
                                   self.status, stream)

    def accept_commit_argmax(self, argmax, stream=None):
        """The walk and commit on a given argmax [rows] int32 (device)."""
        tree_accept_commit_argmax(self.desc, argmax, self.draft, self.parents, self.node_offsets, self.k_tree,
                                  self.v_tree, self.k_cache, self.v_cache, self.page_table, self.prefix_len,
                                  self.accept_len, self.path, self.tokens, self.status, stream)

    def step(self, stream=None):
        """One verify step: mask, attention, accept + commit."""
        self.mask(stream)
        self.attn(stream)
        self.accept_commit(stream)

    def plan(self):
        """The plan of this step's attention."""
        return tv_attn_plan(self.desc)

    def kernels_per_step(self):
        """Our kernel launches in one step: mask, split, merge (skipped when
        the plan has one key chunk), argmax, walk + commit."""
        return 4 + (1 if self.plan()["num_splits"] > 1 else 0)


class DeviceWindowStep(DeviceStep):
    """A verify step whose rows see a sliding window and the first positions
    (sinks) of the prefix; acceptance and commit are DeviceStep's.  The
    windowed attention is one call: it has no halves."""

    def __init__(self, w, window, sinks=0, **kw):
        self.win = make_window(window, sinks)
        super().__init__(w, **kw)

    def _buffers(self, to):
        super()._buffers(to)
        self.attn_ws_bytes, self.attn_workspace = self._workspace(tv_window_workspace_size(self.desc, self.win))

    def attn(self, stream=None):
        tree_verify_attn_window(self.desc, self.win, self.q, self.k_cache, self.v_cache, self.page_table,
                                self.prefix_len, self.node_offsets, self.k_tree, self.v_tree, self.anc, self.depth,
                                self.out, self.attn_workspace, self.attn_ws_bytes, self.status, stream)

    def plan(self):
        return tv_window_attn_plan(self.desc, self.win)

    def partials(self, stream=None):
        raise NotImplementedError("the windowed attention has no call of its own for its partials: use attn")

    def merge(self, stream=None):
        raise NotImplementedError("the windowed attention has no call of its own for its merge: use attn")


class DeviceKv4Step(DeviceStep):
    """A verify step on a cache held in 4 bits (win: (window, sinks) or None).
    The workload's prefix rows are written by tv_kv4_append; acceptance walks
    on a given target argmax and quantises the accepted rows."""

    def __init__(self, w, win=None, **kw):
        self.win = None if win is None else make_window(*win)
        super().__init__(w, **kw)

    def _buffers(self, to):
        kb, vb = tv_kv4_cache_bytes(self.desc)
        self.k4 = torch.zeros(kb, dtype=torch.uint8, device=self.device)
        self.v4 = torch.zeros(vb, dtype=torch.uint8, device=self.device)
        self.attn_ws_bytes, self.attn_workspace = self._workspace(tv_kv4_workspace_size(self.desc, self.win))
        k, v, lens = self._prefix_rows()
        self.append(to(k), to(v), lens, torch.zeros_like(self.prefix_len))

    def _prefix_rows(self):
        """The prefix of every sequence as [Hkv, sum P, d] rows, and their counts."""
        w, lens = self.w, self.w.prefix_len.tolist()
        rows = []
        for x in (w.k_cache, w.v_cache):
            if w.page_table is None:
                rows.append([x[b, :, :n] for b, n in enumerate(lens)])
            else:
                flat = [x[w.page_table[b].long()].transpose(0, 1).flatten(1, 2) for b in range(len(lens))]
                rows.append([f[:, :n] for f, n in zip(flat, lens)])
        return torch.cat(rows[0], 1).contiguous(), torch.cat(rows[1], 1).contiguous(), lens

    def _offsets(self, counts):
        return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=self.device)

    def append(self, k, v, counts, start, stream=None):
        """Write k, v [Hkv, sum counts, d] at positions start[b] + i.  With a
        stream, the inputs are kept from reuse until it has read them; that it
        runs after what made them is the caller's."""
        with _on(stream):                                # the offsets live and die on the call's stream
            tv_kv4_append(self.desc, k.shape[1], max(counts), k, v, self._offsets(counts), start, self.k4, self.v4,
                          self.page_table, self.status, stream)
        _keep(stream, k, v, start)

    def read(self, counts, start, stream=None):
        """The values at positions start[b] + i, [Hkv, sum counts, d] each;
        with a stream, tensors of that stream, as torch's are under
        torch.cuda.stream(stream)."""
        with _on(stream):
            k = torch.empty(self.desc.num_kv_heads, sum(counts), self.desc.head_dim, dtype=self.q.dtype,
                            device=self.device)
            v = torch.empty_like(k)
            tv_kv4_read(self.desc, k.shape[1], max(counts), self.k4, self.v4, self.page_table, self._offsets(counts),
                        start, k, v, self.status, stream)
        _keep(stream, start)
        return k, v

    def attn(self, stream=None):
        tree_verify_attn_kv4(self.desc, self.win, self.q, self.k4, self.v4, self.page_table, self.prefix_len,
                             self.node_offsets, self.k_tree, self.v_tree, self.anc, self.depth, self.out,
                             self.attn_workspace, self.attn_ws_bytes, self.status, stream)

    def accept_commit_argmax(self, argmax, stream=None):
        tree_accept_commit_argmax_kv4(self.desc, argmax, self.draft, self.parents, self.node_offsets, self.k_tree,
                                      self.v_tree, self.k4, self.v4, self.page_table, self.prefix_len,
                                      self.accept_len, self.path, self.tokens, self.status, stream)

    def step(self, argmax, stream=None):
        """One verify step on the target's argmax [rows] int32 (device): mask,
        attention, walk + commit."""
        self.mask(stream)
        self.attn(stream)
        self.accept_commit_argmax(argmax, stream)

    def plan(self):
        return tv_kv4_attn_plan(self.desc, self.win)

    def kernels_per_step(self):
        """Mask, split, merge (skipped when the plan has one key chunk), walk + commit."""
        return 3 + (1 if self.plan()["num_splits"] > 1 else 0)

    def partials(self, stream=None):
        raise NotImplementedError("the 4-bit cache's attention has no call of its own for its partials: use attn")

    def merge(self, stream=None):
        raise NotImplementedError("the 4-bit cache's attention has no call of its own for its merge: use attn")

    def accept_commit(self, stream=None):
        raise NotImplementedError("the 4-bit cache is committed on a given argmax: use accept_commit_argmax")

    def accept_commit_sampled(self, temperature, seed, offset, stream=None):
        raise NotImplementedError("the 4-bit cache is committed on a given argmax: use accept_commit_argmax")


class DeviceExpand:
    """Device buffers of one expansion workload (workloads.ExpandSpec): the
    synthetic drafter's logits of every step (resident), the roots, the tree
    outputs and the workspace; step(s) is one tv_tree_expand_step call."""

    def __init__(self, spec, device="cuda", rows=None, token_map=None, steps=None):
        from . import workloads as wl
        dev = torch.device(device)
        self.spec = spec
        dt = {"f32": F32, "bf16": BF16}[spec.dtype]
        self.desc = make_expand_desc(batch=spec.batch, vocab=spec.vocab, top_k=spec.top_k, width=spec.width,
                                     max_nodes=spec.max_nodes, max_depth=spec.max_depth, logits_dtype=dt)
        self.steps = tv_expand_steps(self.desc) if steps is None else int(steps)
        if rows is None:
            rows = [wl.draft_rows(spec, s) for s in range(self.steps)]
        self.rows = [r.to(dev).contiguous() for r in rows]
        self.roots = wl.root_tokens(spec).to(dev)
        self.token_map = None if token_map is None else token_map.to(dev).to(torch.int32).contiguous()
        B, N = spec.batch, spec.max_nodes
        self.tokens = torch.zeros(B, N, dtype=torch.int32, device=dev)
        self.parents = torch.zeros(B, N, dtype=torch.int32, device=dev)
        self.depths = torch.zeros(B, N, dtype=torch.int32, device=dev)
        self.cum = torch.zeros(B, N, dtype=torch.float64, device=dev)
        self.n_nodes = torch.zeros(B, dtype=torch.int32, device=dev)
        self.expand_count = torch.zeros(B, dtype=torch.int32, device=dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.ws_bytes = tv_expand_workspace_size(self.desc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def step(self, s, stream=None):
        x = self.rows[s]
        tv_tree_expand_step(self.desc, s, x, x.shape[1] * x.shape[2], self.roots, self.token_map, self.tokens,
                            self.parents, self.depths, self.cum, self.n_nodes, self.expand_count, self.workspace,
                            self.ws_bytes, self.status, stream)

    def run(self, stream=None):
        """Every step, in order (two kernel launches each)."""
        for s in range(self.steps):
            self.step(s, stream)


class DevicePrompt:
    """Prompts (or chunks of them) on their way into a step's cache: `lens[b]`
    new rows of sequence b behind what is committed.  run() rotates the rows,
    writes their keys and values into the cache, attends to prefix and rows, and
    moves the step's prefix lengths on.  max_prefix: a bound on what is committed
    before (the step's own if None).  A windowed step's prompts have to fit the
    window, where rows see all that is before them; a 4-bit step's go through
    its append.  With a stream, a call keeps the inputs and this object's buffers
    from reuse until the stream has passed it; that it runs after what made them
    is the caller's."""

    def __init__(self, step, lens, theta=1e4, max_prefix=None):
        if isinstance(step, DeviceKv4Step):
            raise NotImplementedError("prompts into the 4-bit cache have no DevicePrompt: use DeviceKv4Step.append")
        d, dev = step.desc, step.device
        if len(lens) != d.batch or min(lens) < 0:
            raise ValueError(f"lens: {d.batch} sequences want a number of rows each, 0 or more, not {list(lens)}")
        max_prefix = d.max_prefix if max_prefix is None else int(max_prefix)
        self.step, self.theta, self.rows, self.max_rows = step, theta, sum(lens), max(lens)
        if isinstance(step, DeviceWindowStep) and step.win.window < max_prefix + self.max_rows:
            raise NotImplementedError(f"rows at positions up to {max_prefix + self.max_rows - 1} in a window of "
                                      f"{step.win.window}: the prompt attention has no window")
        self.desc = make_desc(batch=d.batch, num_q_heads=d.num_q_heads, num_kv_heads=d.num_kv_heads,
                              head_dim=d.head_dim, dtype=d.dtype, max_nodes=1, total_rows=d.batch,
                              capacity=d.capacity, max_prefix=max_prefix, page_size=d.page_size,
                              num_pages=d.num_pages, out_f32=d.out_f32, scale=d.scale)
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        self.offsets = torch.tensor(offs, dtype=torch.int32, device=dev)
        dt = step.q.dtype
        self.q = torch.empty(self.rows, d.num_q_heads, d.head_dim, dtype=dt, device=dev)
        self.k_rows = torch.empty(d.num_kv_heads, self.rows, d.head_dim, dtype=dt, device=dev)
        self.v_rows = torch.empty_like(self.k_rows)
        self.out = torch.empty(self.rows, d.num_q_heads, d.head_dim, dtype=step.out.dtype, device=dev)
        self.new_prefix = torch.empty(d.batch, dtype=torch.int32, device=dev)
        self.ws_bytes = tv_prompt_workspace_size(self.desc, self.rows, self.max_rows)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def rope_store(self, q, k, v, stream=None):
        st = self.step
        _keep(stream, q, k, v, self.q, self.k_rows, self.v_rows, self.offsets, self.new_prefix)
        if self.rows == 0:                               # the call would enqueue nothing, the lengths neither
            with _on(stream):
                self.new_prefix.copy_(st.prefix_len)
            return
        tv_prompt_rope_store(self.desc, self.rows, self.max_rows, self.theta, q, k, v, st.prefix_len, self.offsets,
                             self.q, self.k_rows, self.v_rows, st.k_cache, st.v_cache, st.page_table, self.new_prefix,
                             st.status, stream)

    def attn(self, stream=None):
        st = self.step
        _keep(stream, self.q, self.k_rows, self.v_rows, self.offsets, self.out, self.workspace)
        tv_prompt_attn(self.desc, self.rows, self.max_rows, self.q, st.k_cache, st.v_cache, st.page_table,
                       st.prefix_len, self.offsets, self.k_rows, self.v_rows, self.out, self.workspace, self.ws_bytes,
                       st.status, stream)

    def run(self, q, k, v, stream=None):
        """q [rows, Hq, d], k and v [rows, Hkv, d] as the projections leave them."""
        self.rope_store(q, k, v, stream)
        self.attn(stream)
        with _on(stream):
            self.step.prefix_len.copy_(self.new_prefix)


class LogitControl:
    """Penalties, biases and grammar masks on a step's logits, with the token
    counts they go by.  penalties [B, 3] float (repetition, frequency,
    presence); biases: (offsets, tokens, values) or None; mask [rows, words]
    int32 or None.  Streams are as DevicePrompt takes them."""

    def __init__(self, step, penalties, biases=None, mask=None):
        B = step.desc.batch
        self.step, self.mask = step, mask
        self.penalties = penalties
        if biases is not None and biases[1].numel() == 0:
            biases = None                                # an empty tensor has no address for the call
        self.biases = (None, None, None) if biases is None else biases
        self.counts = torch.zeros(B, (step.vocab + 7) // 8 * 8, dtype=torch.int16, device=step.device)
        self.desc = make_logits_desc(batch=B, vocab=step.vocab, max_nodes=step.desc.max_nodes,
                                     total_rows=step.desc.total_rows, logits_dtype=step.logits_dtype,
                                     biases=0 if biases is None else biases[1].numel())

    def read(self, tokens, offsets, stream=None):
        """The prompts' tokens (packed, int32)."""
        tv_token_counts_add(self.desc, tokens, offsets, tokens.numel(), True, self.counts, self.step.status, stream)
        _keep(stream, tokens, offsets, self.counts)

    def started(self, stream=None):
        """The roots of the step's trees, as emitted.  Once, before a sequence's
        first step: a later root is the last token that emitted() counted."""
        st = self.step
        with _on(stream):                                # the tokens live and die on the call's stream
            roots = st.draft[st.node_offsets[:-1].long()]
            tv_token_counts_add(self.desc, roots, None, 1, False, self.counts, st.status, stream)
        _keep(stream, self.counts)

    def emitted(self, stream=None):
        """What the step's accept + commit emitted."""
        st = self.step
        tv_token_counts_add(self.desc, st.tokens, None, st.desc.max_nodes, False, self.counts, st.status, stream)
        _keep(stream, self.counts)

    def process(self, stream=None):
        """The step's logits, in place (after its mask call)."""
        st = self.step
        tv_tree_logits_process(self.desc, st.logits, self.counts, self.penalties, *self.biases, self.mask, st.draft,
                               st.node_offsets, st.anc, st.logits, st.status, stream)
        _keep(stream, self.counts, self.penalties, self.mask, *self.biases)


class DeviceLmHead:
    """Device buffers of one lm_head workload (workloads.LmHeadSpec): hidden
    rows and weights resident, the argmax and max-logit outputs, the
    workspace; run() is one tv_lm_head_argmax call."""

    def __init__(self, spec, device="cuda", hidden=None, weight=None):
        from . import workloads as wl
        dev = torch.device(device)
        self.spec = spec
        if hidden is None or weight is None:
            hidden, weight = wl.lm_head_inputs(spec)
        self.hidden = hidden.to(dev).contiguous()
        self.weight = weight.to(dev).contiguous()
        self.desc = make_lmhead_desc(rows=spec.rows, hidden=spec.hidden, vocab=spec.vocab)
        self.argmax = torch.zeros(spec.rows, dtype=torch.int32, device=dev)
        self.max_logit = torch.zeros(spec.rows, dtype=torch.float32, device=dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.ws_bytes = tv_lm_head_workspace_size(self.desc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def run(self, stream=None, weight=None):
        tv_lm_head_argmax(self.desc, self.hidden, self.weight if weight is None else weight, self.argmax,
                          self.max_logit, self.workspace, self.ws_bytes, self.status, stream)


def main(argv=None):
    """Run one seeded input set of a workload through the verify step a few
    times (e.g. under a profiler): python -m speculative_decoding_tree_gb300.runner
    --config 4 --steps 3.  Prints the device status word and exits non-zero
    when it is not 0."""
    import argparse

    from . import _build, workloads as wl

    ap = argparse.ArgumentParser()
    ap.add_argument("--config", type=int, default=4, help="workload 1..5")
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--attn-only", action="store_true", help="mask and attention only")
    ap.add_argument("--sampled", type=float, default=0.0,
                    help="temperature > 0: sampled verification (tree_accept_commit_sampled)")
    ap.add_argument("--window", default="", help="W,S: rows see the last W and the first S positions")
    ap.add_argument("--kv4", action="store_true",
                    help="the prefix in a 4-bit cache (with --window too); acceptance on the logits' argmax")
    ap.add_argument("--prompt", type=int, default=0,
                    help="N: first put N prompt rows a sequence through RoPE, the cache's writes and causal attention")
    ap.add_argument("--steer", action="store_true", help="penalties on the logits before acceptance")
    ap.add_argument("--expand", default="", help="run a dynamic-expansion workload instead (eagle2, batched)")
    ap.add_argument("--lm-head", default="", help="run a fused lm_head + argmax workload instead (qwen, batched)")
    ap.add_argument("--vocab", type=int, default=0, help="with --lm-head: a smaller vocabulary (e.g. for a profiler)")
    a = ap.parse_args(argv)
    if a.kv4 and a.sampled > 0:
        ap.error("--sampled: the 4-bit cache is committed on a given argmax only")
    if a.kv4 and a.prompt:
        ap.error("--prompt: prompts into the 4-bit cache go through its append")
    if a.window and a.prompt:
        ap.error("--prompt: the prompt attention has no window")
    _build.build()
    if a.lm_head:
        spec = wl.LMHEAD_CONFIGS[a.lm_head]
        lm = DeviceLmHead(spec.replace(vocab=a.vocab, name=f"{spec.name}-v{a.vocab}") if a.vocab else spec)
        for _ in range(a.steps):
            lm.run()
        torch.cuda.synchronize()
        status = int(lm.status[0].item())
        print(f"{lm.spec.name}: {a.steps} calls, device status {status}")
        return 0 if status == 0 else 1
    if a.expand:
        dx = DeviceExpand(wl.EXPAND_CONFIGS[a.expand])
        for _ in range(a.steps):
            dx.run()
        torch.cuda.synchronize()
        status = int(dx.status[0].item())
        print(f"{dx.spec.name}: {a.steps} expansions of {dx.steps} steps, {int(dx.n_nodes.sum())} nodes, "
              f"device status {status}")
        return 0 if status == 0 else 1
    w = wl.make_workload(wl.CONFIGS[a.config], canary=0.0,
                         argmax_fn=lambda x: torch.argmax(x.float(), dim=1))   # plants the draft tokens
    win = tuple(int(x) for x in a.window.split(",")) if a.window else None
    st = DeviceKv4Step(w, win) if a.kv4 else (DeviceWindowStep(w, *win) if win else DeviceStep(w))
    argmax = lambda: st.logits.float().argmax(1).to(torch.int32)
    target = argmax() if a.kv4 else None
    p0 = st.prefix_len.clone()
    prompt = control = None
    if a.prompt:                                 # rows of noise, into positions the workload's prefix holds after it
        fill = min(a.prompt, int(p0.min()))
        prompt = DevicePrompt(st, [fill] * st.desc.batch)
        rows = [torch.randn(prompt.rows, h, st.desc.head_dim, device=st.device).to(st.q.dtype)
                for h in (st.desc.num_q_heads, st.desc.num_kv_heads, st.desc.num_kv_heads)]
    if a.steer:
        control = LogitControl(st, torch.tensor([[1.1, 0.1, 0.1]] * st.desc.batch, device=st.device))
        control.started()
        raw = st.logits.clone()                  # the target's logits are the same every step
    for _ in range(a.steps):
        if prompt:
            st.prefix_len.zero_()
            prompt.run(*rows)
        st.prefix_len.copy_(p0)
        if control:
            st.logits.copy_(raw)
            st.mask()
            control.process()
        if a.attn_only:
            st.mask()
            st.attn()
        elif a.sampled > 0:
            st.mask()
            st.attn()
            st.accept_commit_sampled(a.sampled, 1234, _)
        elif a.kv4:
            st.step(argmax() if control else target)
        else:
            st.step()
        if control and not a.attn_only:
            control.emitted()
    torch.cuda.synchronize()
    status = int(st.status[0].item())
    print(f"{w.spec.name}: {a.steps} steps, device status {status}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    raise SystemExit(main())
