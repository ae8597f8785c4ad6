"""Verify attention over a cache held in 4 bits, over a sliding window with sinks, and the 4-bit cache's own writes.

Three operators of the library, each in its plain form (elementary torch operations in 32 bits) and, where `own` is
true, as the library's calls:

  kv4     tree_verify_attn_kv4: each draft-tree row attends to the committed prefix, held in 4 bits, and to its
          ancestors, held in the inputs' type
  store   tv_kv4_append / tree_accept_commit_argmax_kv4 and tv_kv4_read: rows are put into the 4-bit cache (a whole
          prompt, or the accepted path of a verify step) and read back as the values it then stands for
  window  tree_verify_attn_window: the same attention over an fp32 or bf16 cache, where a row sees the first `sinks`
          positions and the last `window` ones

The 4-bit cache holds blocks of 16 positions for each KV head.  A value is (u - 8) * s with u in 0..15 and a scale
s = 2^(e - 15) * (1 + m / 8) in a byte e * 8 + m.  K has a scale for every 32 channels of a position, V one for all
channels of a position.  A K block: for each 32 channels, 16 positions x 16 bytes, then for each 32 channels 16 scale
bytes.  A V block: for each channel 8 bytes (16 positions), then 16 scale bytes.  Eight values are one little-endian
32-bit word, value 2j at bit 4j and value 2j + 1 at bit 16 + 4j.
"""
import math

import torch

own = False

BLOCK = 16
GROUP = 32


def listed():
    return [
        # one token a sequence against a medium context: the smallest call, latency
        _attn("kv4-decode-8k", "kv4", 1, 32, 8, 128, "bf16", (8192, 8192), (1, 1)),
        # a 4-node draft chain at the widest head
        _attn("kv4-chain-d512-20k", "kv4", 1, 16, 2, 512, "bf16", (20011, 20011), (4, 4)),
        # a 60-node draft tree over a long context, one sequence
        _attn("kv4-tree60-32k", "kv4", 1, 16, 4, 256, "bf16", (32768, 32768), (60, 60)),
        # a batch of ragged trees over a paged cache
        _attn("kv4-batch16-paged", "kv4", 16, 32, 8, 128, "bf16", (512, 8192), (16, 64), paged=True),
        # plain decoding of a large ragged batch over a paged cache: the largest read
        _attn("kv4-decode-batch64", "kv4", 64, 32, 8, 128, "bf16", (1000, 16384), (1, 1), paged=True),
        # the commit of a batch's accepted paths after a verify step
        _store("store-commit-batch16", 16, 8, 128, "bf16", (20, 200), (16, 64), paged=True),
        # a prompt of odd length into a contiguous fp32-fed cache
        _store("store-prompt-f32", 1, 4, 256, "f32", (0, 0), (4099, 4099), commit=False),
        # several long prompts into a paged cache
        _store("store-prompts-paged", 4, 8, 128, "bf16", (0, 1000), (8000, 32768), paged=True, commit=False),
        # one token against the last 4096 positions and 4 sinks of a long context
        _attn("window-decode-32k", "window", 1, 32, 8, 128, "bf16", (32768, 32768), (1, 1), window=4096, sinks=4),
        # a draft tree over the same window
        _attn("window-tree60-32k", "window", 1, 16, 4, 256, "bf16", (32768, 32768), (60, 60), window=4096, sinks=4),
        # ragged trees over a paged cache with a short odd window
        _attn("window-batch16-paged", "window", 16, 32, 8, 128, "bf16", (512, 8192), (16, 64), paged=True,
              window=1023, sinks=16),
        # the small fp32 tree with a window that cuts its own context
        _attn("window-tree8-f32", "window", 1, 4, 4, 256, "f32", (2000, 2000), (8, 8), window=500, sinks=3),
    ]


def _attn(name, op, batch, hq, hkv, d, dtype, prefix, nodes, paged=False, window=0, sinks=0):
    return dict(name=name, op=op, batch=batch, hq=hq, hkv=hkv, d=d, dtype=dtype, plo=prefix[0], phi=prefix[1],
                nlo=nodes[0], nhi=nodes[1], paged=paged, window=window, sinks=sinks)


def _store(name, batch, hkv, d, dtype, prefix, rows, paged=False, commit=True):
    return dict(name=name, op="store", batch=batch, hq=hkv, hkv=hkv, d=d, dtype=dtype, plo=prefix[0], phi=prefix[1],
                nlo=rows[0], nhi=rows[1], paged=paged, commit=commit)


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    """One more case: heads, types, lengths, trees, windows and layouts over the listed cases' ranges."""
    op = rng.choice(["kv4", "kv4", "store", "window"])
    d = rng.choice([128, 128, 256, 512])
    hkv = rng.choice([1, 2, 4, 8])
    batch = _log(rng, 1, 64) if rng.random() < 0.5 else 1
    paged = rng.random() < 0.5
    most = 64 * 8 * 128 * 8000 // (batch * hkv * d)          # positions a sequence, as in the largest listed case
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op == "store":
        commit = rng.random() < 0.5
        c = _store("", batch, hkv, d, dtype, (0, 0), (1, 1), paged, commit)
        most = min(32768, most // 4)
        c["phi"] = _log(rng, 16, 400)
        c["plo"] = rng.randint(0, c["phi"])
        c["nhi"] = _log(rng, 1, 64) if commit else _log(rng, 1, max(2, most))
        c["nlo"] = rng.randint(max(1, c["nhi"] // 4), c["nhi"])
    else:
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        nhi = 1 if rng.random() < 0.35 else _log(rng, 2, 64)
        if dtype == "f32":
            most //= 32                                      # the wide type's calls stay below the largest listed one
        if nhi * hq // hkv > 16:
            most //= 4
        phi = _log(rng, 100, max(101, min(32768, most)))
        c = _attn("", op, batch, hq, hkv, d, dtype, (rng.randint(0, phi), phi), (rng.randint(1, nhi), nhi), paged)
        if op == "window" or rng.random() < 0.3:
            c["window"] = _log(rng, 1, 8192)
            c["sinks"] = rng.choice([0, 1, 4, 16, 130])
    del c["name"]
    return c


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, the same for every seed; the last is hi."""
    return [hi if b == n - 1 else lo + int((hi - lo + 1) * ((0.5 + b * step) % 1.0)) for b in range(n)]


def _sizes(case):
    B = case["batch"]
    return _spread(case["plo"], case["phi"], B, 0.6180339887), _spread(case["nlo"], case["nhi"], B, 0.4142135623)


def work(case):
    """Bytes and operations of one pass: every visible cache row read once, the tree's rows, queries and results."""
    P, N = _sizes(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    packed = hkv * (8.5 * d + 8 * d + 16) / 16                # K and V of one position over the KV heads
    plain = 2 * hkv * d * es
    if case["op"] == "store":
        rows = sum(N)
        if case["commit"]:                                    # the rows an accepted path may hold, then the read-back
            return {"bytes": (sum(P) + rows) * (packed + plain), "flops": 4.0 * rows * hkv * d}
        return {"bytes": 2 * rows * (plain + packed), "flops": 8.0 * rows * hkv * d}
    W, S = case["window"], case["sinks"]
    seen = [min(p, min(p, S) + max(0, W - 1)) if W else p for p in P]
    by = sum(k * (packed if case["op"] == "kv4" else plain) for k in seen)
    by += sum(n * (plain + 2 * hq * d * es) for n in N)
    return {"bytes": by, "flops": sum(4.0 * d * hq * n * (k + 1) for n, k in zip(N, seen))}


# ------------------------------------------------------------------ inputs

def _scales(dev):
    c = torch.arange(256, device=dev, dtype=torch.int32)
    return ((c // 8 + 112 << 23) + (c % 8 << 20)).view(torch.float32)    # exact: the bits of the 32-bit number


def _quantise(x, dim_groups):
    """x [..., n] in groups of n / dim_groups: (u, scale code, values); the smallest scale whose 7 steps reach the
    group's largest magnitude."""
    t = _scales(x.device)
    g = x.double().reshape(*x.shape[:-1], dim_groups, -1)
    code = torch.searchsorted(t.double() * 7, g.abs().amax(-1)).clamp(max=255)
    s = t.double()[code]
    q = (g / s[..., None]).round().clamp(-7, 7)
    return (q + 8).to(torch.uint8).reshape(x.shape), code.to(torch.uint8), (q * s[..., None]).float().reshape(x.shape)


def _words(u):
    """[..., 8 n] values of 4 bits -> [..., 4 n] bytes."""
    u = u.reshape(*u.shape[:-1], -1, 8)
    return torch.stack([u[..., 0] | u[..., 2] << 4, u[..., 4] | u[..., 6] << 4, u[..., 1] | u[..., 3] << 4,
                        u[..., 5] | u[..., 7] << 4], -1).flatten(-2)


def _pack(k, v):
    """[..., T, d] rows (T a multiple of 16) -> K blocks [..., T / 16, 8.5 d] and V blocks [..., T / 16, 8 d + 16]."""
    d = k.shape[-1]
    uk, ck, _ = _quantise(k, d // GROUP)
    uv, cv, _ = _quantise(v, 1)
    lead = k.shape[:-2]
    wk = _words(uk).reshape(*lead, -1, BLOCK, d // GROUP, 16).transpose(-2, -3).flatten(-3)
    sk = ck.reshape(*lead, -1, BLOCK, d // GROUP).transpose(-1, -2).flatten(-2)
    wv = _words(uv.reshape(*lead, -1, BLOCK, d).transpose(-1, -2)).flatten(-2)
    return torch.cat([wk, sk], -1), torch.cat([wv, cv.reshape(*lead, -1, BLOCK)], -1)


def _unwords(b):
    b = b.reshape(*b.shape[:-1], -1, 4)
    lo, hi = b & 15, b >> 4
    return torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1],
                        hi[..., 3]], -1).flatten(-2)


def _unpack(k4, v4, d):
    """The float32 rows [..., T, d] that blocks [..., T / 16, bytes] stand for."""
    t = _scales(k4.device)
    lead = k4.shape[:-2]
    uk = _unwords(k4[..., :8 * d].reshape(*k4.shape[:-1], d // GROUP, BLOCK, 16)).transpose(-2, -3)
    sk = t[k4[..., 8 * d:].long()].reshape(*k4.shape[:-1], d // GROUP, BLOCK).transpose(-1, -2)
    k = (uk.float() - 8) * sk[..., None]
    uv = _unwords(v4[..., :8 * d].reshape(*v4.shape[:-1], d, 8)).transpose(-1, -2)
    v = (uv.float() - 8) * t[v4[..., 8 * d:].long()][..., None]
    return k.reshape(*lead, -1, d), v.reshape(*lead, -1, d)


def _rows(gen, shape, dtype, heavy=False):
    x = torch.randn(shape, generator=gen, device="cuda")
    if heavy:                                                 # a few channels of K are larger than the rest
        x = x * (1 + 3 * (torch.arange(shape[-1], device="cuda") % 37 == 5))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator("cpu").manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    P, N = _sizes(case)
    R, mp, mn = sum(N), max(P), max(N)
    attn = case["op"] != "store"
    tree = attn or case["commit"]
    blocks = [-(-(p + n) // BLOCK) + 1 for p, n in zip(P, N)]
    cap = max(blocks)
    i32 = dict(dtype=torch.int32, device="cuda")
    offs = [0]
    for n in N:
        offs.append(offs[-1] + n)
    st = dict(case=case, dt=dt, cap=cap * BLOCK, mp=mp, mn=mn, R=R, prefix=torch.tensor(P, **i32),
              offsets=torch.tensor(offs, **i32))
    # trees: parents, ancestors (a 64-bit word a row) and depths
    if tree:
        par, anc, dep = [], [], []
        for n in N:
            pick = torch.rand(n, generator=cpu).tolist()
            base = len(par)
            for i in range(n):
                q = -1 if i == 0 else max(0, i - 1 - int(pick[i] * min(i, 9)))
                par.append(q)
                anc.append(1 << i | (anc[base + q] if i else 0))
                dep.append(dep[base + q] + 1 if i else 0)
        st["parents"] = torch.tensor(par, **i32)
        st["anc"] = torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64, device="cuda")
        st["depth"] = torch.tensor(dep, **i32)
    # the page table: every sequence's pages in shuffled order
    if case["paged"]:
        perm = torch.randperm(sum(blocks), generator=cpu).tolist()
        table, at = [], 0
        for n in blocks:
            table.append(perm[at:at + n] + [0] * (cap - n))
            at += n
        st["table"] = torch.tensor(table, **i32)
        st["pages"] = sum(blocks)
    else:
        st["table"], st["pages"] = None, 0
    st["k_rows"] = _rows(gen, (hkv, R, d), dt, True)
    st["v_rows"] = _rows(gen, (hkv, R, d), dt)
    pool = (sum(blocks), hkv, BLOCK) if case["paged"] else (B, hkv, cap * BLOCK)
    if case["op"] == "window":
        st["k_cache"], st["v_cache"] = _rows(gen, (*pool, d), dt, True), _rows(gen, (*pool, d), dt)
    else:
        k4, v4 = [], []
        for h in range(0, pool[0], 512 if case["paged"] else 1):
            n = (min(512, pool[0] - h), *pool[1:], d) if case["paged"] else (1, *pool[1:], d)
            a, b = _pack(_rows(gen, n, dt, True), _rows(gen, n, dt))
            k4.append(a.squeeze(2) if case["paged"] else a)
            v4.append(b.squeeze(2) if case["paged"] else b)
        st["k4"], st["v4"] = torch.cat(k4), torch.cat(v4)
        del k4, v4
    if attn:
        st["q"] = _rows(gen, (R, hq, d), dt)
        st["out"] = torch.empty(R, hq, d, dtype=dt, device="cuda")
    else:
        # a commit is read back from the cache's start, an append the rows it wrote
        ends = [p + n for p, n in zip(P, N)] if case["commit"] else N
        ro = [0]
        for n in ends:
            ro.append(ro[-1] + n)
        st["read_offsets"], st["read_rows"], st["read_most"] = torch.tensor(ro, **i32), ro[-1], max(ends)
        st["zeros"] = torch.zeros(B, **i32)
        st["k_out"] = torch.empty(hkv, ro[-1], d, dtype=dt, device="cuda")
        st["v_out"] = torch.empty(hkv, ro[-1], d, dtype=dt, device="cuda")
        if case["commit"]:
            am = torch.randint(0, 32000, (R,), generator=cpu)
            hit = torch.rand(R, generator=cpu) < 0.7
            first = torch.tensor([offs[b] for b in range(B) for _ in range(N[b])])
            up = am[first + torch.tensor(par).clamp(min=0)]
            st["argmax"] = am.to(torch.int32).cuda()
            st["draft"] = torch.where(hit, up, (up + 1) % 32000).to(torch.int32).cuda()
            st["length"] = st["prefix"].clone()
            st["accept_len"] = torch.empty(B, **i32)
            st["path"], st["tokens"] = torch.empty(B, mn, **i32), torch.empty(B, mn, **i32)
    st["status"] = torch.zeros(4, **i32)
    # where the plain form finds each padded node's row and each position's block
    j = torch.arange(mn, device="cuda")
    n_of = torch.tensor(N, device="cuda")
    st["live"] = j < n_of[:, None]
    st["row_of"] = (torch.tensor(offs[:-1], device="cuda")[:, None] + j).clamp(max=R - 1)
    return st


# ------------------------------------------------------------------ the operators

def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] != "store":
        return _plain_attention(state)
    return _plain_commit(state) if c["commit"] else _plain_append(state)


def _cache_rows(st):
    """The cache as float32 rows [B, Hkv, T, d]."""
    c = st["case"]
    if c["op"] == "window":
        k, v = st["k_cache"], st["v_cache"]
        if c["paged"]:
            k, v = (x[st["table"].long()].transpose(1, 2).flatten(2, 3) for x in (k, v))
        return k.float(), v.float()
    k, v = st["k4"], st["v4"]
    if c["paged"]:
        k, v = (x[st["table"].long()].transpose(1, 2) for x in (k, v))
    return _unpack(k, v, c["d"])


def _plain_attention(st):
    c = st["case"]
    B, hq, hkv, d, mn = c["batch"], c["hq"], c["hkv"], c["d"], st["mn"]
    G = hq // hkv
    k, v = _cache_rows(st)
    k, v = k[:, :, :max(st["mp"], 1)], v[:, :, :max(st["mp"], 1)]
    rows, P = st["row_of"], st["prefix"].long()
    q = st["q"].float()[rows].reshape(B, mn, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, mn * G, d)
    kt, vt = (x.float()[:, rows].transpose(0, 1) for x in (st["k_rows"], st["v_rows"]))
    t = torch.arange(k.shape[2], device=q.device)
    dep = st["depth"].long()[rows]
    see = (t < P[:, None])[:, None].expand(B, mn, -1)
    node = torch.arange(mn, device=q.device)
    tree = (st["anc"][rows][..., None] >> node & 1).bool() & st["live"][:, None]
    if c["window"]:
        here = (P[:, None] + dep)
        see = see & ((t < c["sinks"]) | (here[..., None] - t < c["window"]))
        tree = tree & ((here[:, None] < c["sinks"]) | (dep[..., None] - dep[:, None] < c["window"]))
    s = torch.cat([q @ k.transpose(-1, -2), q @ kt.transpose(-1, -2)], -1).reshape(B, hkv, mn, G, -1)
    s = (s * (1 / math.sqrt(d))).masked_fill(~torch.cat([see, tree], -1)[:, None, :, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, hkv, mn * G, -1)
    o = p[..., :t.numel()] @ v + p[..., t.numel():] @ vt
    o = o.reshape(B, hkv, mn, G, d).permute(0, 2, 1, 3, 4).reshape(B, mn, hq, d)
    return o[st["live"]].to(st["dt"])


def _plain_append(st):
    d = st["case"]["d"]
    return {"k": _quantise(st["k_rows"], d // GROUP)[2].to(st["dt"]), "v": _quantise(st["v_rows"], 1)[2].to(st["dt"])}


def _plain_commit(st):
    c, mn, dev = st["case"], st["mn"], st["prefix"].device
    B, rows, live = c["batch"], st["row_of"], st["live"]
    node = torch.arange(mn, device=dev)
    par = st["parents"].long()[rows].clamp(min=0)
    am, draft, dep = st["argmax"].long()[rows], st["draft"].long()[rows], st["depth"].long()[rows]
    match = (node == 0) | (draft == am.gather(1, par))
    anc = (st["anc"][rows][..., None] >> node & 1).bool()
    good = (match[:, None] | ~anc).all(-1) & live
    best = torch.where(good, dep * 256 + 255 - node, -1).amax(1)
    k, end = best // 256, 255 - best % 256
    on = anc[torch.arange(B, device=dev), end]                # the accepted path's nodes
    place = torch.where(on, dep, mn)
    path = torch.full((B, mn + 1), -1, device=dev).scatter(1, place, node.expand(B, -1))[:, :mn]
    step = node <= k[:, None]
    path = torch.where(step, path, -1)
    after = torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0)
    last = am.gather(1, end[:, None])
    tokens = torch.where(node < k[:, None], draft.gather(1, after), torch.where(node == k[:, None], last, -1))
    # the cache's rows, with the accepted ones put behind the prefix
    P = st["prefix"].long()
    kc, vc = _cache_rows(st)
    T = kc.shape[2]
    t = torch.arange(T, device=dev)
    off = t - P[:, None]
    new = (off >= 0) & (off <= k[:, None])
    src = rows.gather(1, path.gather(1, off.clamp(0, mn - 1)).clamp(min=0))
    kq, vq = _quantise(st["k_rows"], c["d"] // GROUP)[2], _quantise(st["v_rows"], 1)[2]
    kc = torch.where(new[:, None, :, None], kq[:, src].transpose(0, 1), kc)
    vc = torch.where(new[:, None, :, None], vq[:, src].transpose(0, 1), vc)
    keep = t < (st["read_offsets"][1:] - st["read_offsets"][:-1])[:, None]
    return {"accept_len": k.int(), "path": path.int(), "tokens": tokens.int(), "prefix_len": (P + k + 1).int(),
            "k": kc.transpose(0, 1)[:, keep].to(st["dt"]), "v": vc.transpose(0, 1)[:, keep].to(st["dt"])}


def _plan(st):
    """The descriptor, window and workspace that a program keeps between its calls."""
    import speculative_decoding_tree_gb300 as tv
    c = st["case"]
    st["desc"] = tv.make_desc(
        batch=c["batch"], num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
        dtype=tv.BF16 if c["dtype"] == "bf16" else tv.F32, max_nodes=min(st["mn"], 64),
        total_rows=min(st["R"], c["batch"] * min(st["mn"], 64)), capacity=st["cap"], max_prefix=st["mp"],
        page_size=BLOCK if c["paged"] else 0, num_pages=st["pages"])
    if c["op"] != "store":
        st["win"] = tv.make_window(c["window"], c["sinks"]) if c["window"] else None
        size = tv.tv_kv4_workspace_size if c["op"] == "kv4" else tv.tv_window_workspace_size
        st["ws_bytes"] = size(st["desc"], st["win"])
        st["ws"] = torch.empty(max(st["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    st["tv"] = tv


def _run_own(st):
    if "tv" not in st:
        _plan(st)
    tv, c = st["tv"], st["case"]
    if c["op"] == "kv4":
        tv.tree_verify_attn_kv4(st["desc"], st["win"], st["q"], st["k4"], st["v4"], st["table"], st["prefix"],
                                st["offsets"], st["k_rows"], st["v_rows"], st["anc"], st["depth"], st["out"],
                                st["ws"], st["ws_bytes"], st["status"])
        return st["out"]
    if c["op"] == "window":
        tv.tree_verify_attn_window(st["desc"], st["win"], st["q"], st["k_cache"], st["v_cache"], st["table"],
                                   st["prefix"], st["offsets"], st["k_rows"], st["v_rows"], st["anc"], st["depth"],
                                   st["out"], st["ws"], st["ws_bytes"], st["status"])
        return st["out"]
    if c["commit"]:
        st["length"].copy_(st["prefix"])
        tv.tree_accept_commit_argmax_kv4(st["desc"], st["argmax"], st["draft"], st["parents"], st["offsets"],
                                         st["k_rows"], st["v_rows"], st["k4"], st["v4"], st["table"], st["length"],
                                         st["accept_len"], st["path"], st["tokens"], st["status"])
    else:
        tv.tv_kv4_append(st["desc"], st["R"], st["mn"], st["k_rows"], st["v_rows"], st["offsets"], st["prefix"],
                         st["k4"], st["v4"], st["table"], st["status"])
    tv.tv_kv4_read(st["desc"], st["read_rows"], st["read_most"], st["k4"], st["v4"], st["table"],
                   st["read_offsets"], st["zeros"] if c["commit"] else st["prefix"], st["k_out"], st["v_out"],
                   st["status"])
    rows = {"k": st["k_out"], "v": st["v_out"]}
    if not c["commit"]:
        return rows
    return {"accept_len": st["accept_len"], "path": st["path"], "tokens": st["tokens"], "prefix_len": st["length"],
            **rows}


# ------------------------------------------------------------------ the definition in 64 bits

def _value(block, kind, t, ch, d):
    """Position t, channel ch (index tensors) of one head's blocks [n, bytes], from the block format, in 64 bits."""
    n, i = t // BLOCK, t % BLOCK
    if kind == "k":
        base, e, code = (ch // 32) * 256 + i * 16, ch % 32, block[n, 8 * d + (ch // 32) * 16 + i]
    else:
        base, e, code = ch * 8, i, block[n, 8 * d + i]
    bit = 4 * (e % 8 // 2) + 16 * (e % 2)
    u = (block[n, base + e // 8 * 4 + bit // 8].long() >> bit % 8) & 15
    code = code.long()
    return (u - 8) * (8 + code % 8) * _two_to(code // 8 - 18)


def _two_to(e):
    """2^e in 64 bits, exact (a power function may be a unit off, which decides ties)."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _step64(x, groups):
    """x [..., n] on its groups' grids of 4 bits, in 64 bits."""
    x = x.double().unflatten(-1, (groups, -1))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.frexp((top / 7).clamp(min=2.0 ** -15))[1] - 1   # 2^e <= top / 7 < 2^(e + 1)
    unit = _two_to(e - 3)
    m = torch.ceil(top / (7 * unit)).clamp(min=8)             # the scale m * unit, m in 8..16
    s = (m * unit).clamp(max=2.0 ** 16 * 1.875)
    return ((x / s).round().clamp(-7, 7) * s).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    P, N = _sizes(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    offs = st["offsets"].tolist()
    if case["op"] == "store" and not case["commit"]:
        return {"k": _step64(st["k_rows"], d // 32), "v": _step64(st["v_rows"], 1)}
    ch = torch.arange(d, device="cuda")

    def cached(b, g, kind, n):
        t = torch.arange(n, device="cuda")
        ids = st["table"][b].long() if case["paged"] else None
        if case["op"] == "window":
            x = st["k_cache" if kind == "k" else "v_cache"]
            return (x[ids[t // BLOCK], g, t % BLOCK] if case["paged"] else x[b, g, :n]).double()
        x = st["k4" if kind == "k" else "v4"]
        return _value(x[ids, g] if case["paged"] else x[b, g], kind, t[:, None], ch, d)

    if case["op"] == "store":
        ints = [st[x].tolist() for x in ("parents", "argmax", "draft")]
        res = {"accept_len": None, "path": None, "tokens": None, "prefix_len": None, "k": [], "v": []}
        for b in range(case["batch"]):
            par, am, draft = (x[offs[b]:offs[b + 1]] for x in ints)
            roots, best = {0: [0]}, [0]
            for i in range(1, N[b]):
                if par[i] in roots and draft[i] == am[par[i]]:
                    roots[i] = roots[par[i]] + [i]
                    best = roots[i] if len(roots[i]) > len(best) else best
            at = offs[b] + torch.tensor(best, device="cuda")
            for kind, src, groups in (("k", "k_rows", d // 32), ("v", "v_rows", 1)):
                x = torch.stack([cached(b, g, kind, P[b] + N[b]) for g in range(hkv)])
                x[:, P[b]:P[b] + len(best)] = _step64(st[src][:, at], groups)
                res[kind].append(x)
        res["k"], res["v"] = torch.cat(res["k"], 1), torch.cat(res["v"], 1)
        return res
    out = torch.empty(st["R"], hq, d, dtype=torch.float64, device="cuda")
    G, W = hq // hkv, case["window"]
    for b in range(case["batch"]):
        n, o = N[b], offs[b]
        dep = st["depth"][o:o + n].long()
        pos = torch.cat([torch.arange(P[b], device="cuda"), P[b] + dep])
        me = (P[b] + dep)[:, None]
        bits = (st["anc"][o:o + n, None] >> torch.arange(n, device="cuda")) & 1
        vis = torch.cat([torch.ones(n, P[b], device="cuda", dtype=torch.bool), bits == 1], 1)
        if W:
            vis &= (pos < case["sinks"]) | (pos > me - W)
        for g in range(hkv):
            k = torch.cat([cached(b, g, "k", P[b]), st["k_rows"][g, o:o + n].double()])
            v = torch.cat([cached(b, g, "v", P[b]), st["v_rows"][g, o:o + n].double()])
            q = st["q"][o:o + n, g * G:(g + 1) * G].double()
            s = torch.einsum("nhd,td->hnt", q, k) / d ** 0.5
            out[o:o + n, g * G:(g + 1) * G] = torch.einsum(
                "hnt,td->nhd", torch.softmax(s.masked_fill(~vis, -math.inf), -1), v)
    return out
