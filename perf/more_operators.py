"""Prompts into the cache, attention over them, and the control of the logits that verification reads.

Three operators of the library, each in its plain form (elementary torch operations in 32 bits) and, where `own` is
true, as the library's calls:

  attn    tv_prompt_attn: every row of a prompt (or of a chunk of one) attends to its sequence's committed prefix in the
          cache and to the prompt's rows up to itself; packed sequences of different lengths, grouped heads
  rope    tv_prompt_rope_store: queries and keys of those rows are rotated at their positions, keys and values go
          head-major into the rows the attention reads and to their positions of the cache
  steer   tv_tree_logits_process: the target's logits at every tree row, with penalties for repeated tokens (those
          counted for the sequence and the drafts on the row's path), a sparse bias and a grammar mask

A count is 16 bits for each sequence and token: bit 15, the token is in the prompt; bits 0 - 14, how often it was
emitted.  Rows of the table are padded to 8 tokens.  A mask is one bit a token, token 32 w + i at bit i of word w.
"""
import math

import torch

own = False

PAGE = 16
THETA = 1e6


def listed():
    return [
        # one short question to an empty cache: the smallest call, latency
        _rows_case("attn-short", "attn", 1, 32, 8, 128, "bf16", (0, 0), (100, 100)),
        # a turn of a long conversation: some rows over a long prefix
        _rows_case("attn-turn-32k", "attn", 1, 16, 4, 256, "bf16", (32768, 32768), (200, 200)),
        # a ragged batch of prompts, parts of them cached already, over a paged cache
        _rows_case("attn-batch16-paged", "attn", 16, 32, 8, 128, "bf16", (0, 1000), (100, 2000), paged=True),
        # one long document: the largest call
        _rows_case("attn-prompt-16k", "attn", 1, 32, 8, 128, "bf16", (0, 0), (16384, 16384)),
        # a chunk of odd length at the widest head
        _rows_case("attn-chunk-d512", "attn", 1, 16, 2, 512, "bf16", (508, 508), (4001, 4001)),
        # a prompt in the wide type
        _rows_case("attn-f32", "attn", 1, 4, 4, 256, "f32", (24, 24), (2000, 2000)),
        # 64 rows behind a long prefix, contiguous cache
        _rows_case("rope-chunk64", "rope", 1, 16, 4, 256, "bf16", (32768, 32768), (64, 64)),
        # a ragged batch of prompts into a paged cache
        _rows_case("rope-batch16-paged", "rope", 16, 32, 8, 128, "bf16", (0, 1000), (100, 2000), paged=True),
        # one token of one sequence: the smallest call
        _steer("steer-decode", 1, 32000, "f32", (1, 1), bias=0, mask=True),
        # a batch of plain decoding over an odd vocabulary
        _steer("steer-decode64", 64, 50257, "f32", (1, 1), bias=20, mask=True),
        # the draft tree of one sequence
        _steer("steer-tree64", 1, 151936, "bf16", (64, 64), bias=300, mask=False),
        # a batch of ragged trees, everything on
        _steer("steer-batch16", 16, 128256, "bf16", (16, 64), bias=300, mask=True),
    ]


def _rows_case(name, op, batch, hq, hkv, d, dtype, prefix, rows, paged=False):
    return dict(name=name, op=op, batch=batch, hq=hq, hkv=hkv, d=d, dtype=dtype, plo=prefix[0], phi=prefix[1],
                nlo=rows[0], nhi=rows[1], paged=paged)


def _steer(name, batch, vocab, dtype, nodes, bias, mask):
    return dict(name=name, op="steer", batch=batch, vocab=vocab, dtype=dtype, nlo=nodes[0], nhi=nodes[1], bias=bias,
                mask=mask)


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    """One more case: heads, types, lengths, vocabularies and layouts over the listed cases' ranges."""
    op = rng.choice(["attn", "attn", "attn", "rope", "steer"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op == "steer":
        batch = _log(rng, 1, 64)
        nhi = 1 if rng.random() < 0.3 else _log(rng, 2, max(2, min(64, 700 // batch)))
        vocab = _log(rng, 1000, 151936)
        if rng.random() < 0.5:
            vocab = vocab // 8 * 8
        c = _steer("", batch, vocab, dtype, (rng.randint(1, nhi), nhi), rng.choice([0, 1, 20, 300, 900]),
                   rng.random() < 0.7)
        del c["name"]
        return c
    d = rng.choice([128, 128, 256, 512])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    batch = _log(rng, 1, 32) if rng.random() < 0.6 else 1
    paged = rng.random() < 0.5
    if op == "rope":
        nhi = _log(rng, 1, max(2, min(16384, 64 * 16384 * 128 // (batch * hq * d))))
        phi = _log(rng, 16, 2000)
    else:
        most = 32 * 16384 * 16384 // (batch * hq * (d // 128))       # rows x keys a head, as in the largest listed case
        if dtype == "f32":
            most //= 32                                              # the wide type's calls stay well below it
        nhi = _log(rng, 1, max(2, min(16384, math.isqrt(most))))
        phi = _log(rng, 1, max(2, min(32768, most // nhi - nhi, 131072 // batch)))
    c = _rows_case("", op, batch, hq, hkv, d, dtype, (0, phi if rng.random() < 0.7 else 0),
                   (rng.randint(max(1, nhi // 8), nhi), nhi), paged)
    if batch == 1:
        c["plo"] = c["phi"]
    del c["name"]
    return c


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, the same for every seed; the last is hi."""
    return [hi if b == n - 1 else lo + int((hi - lo + 1) * ((0.5 + b * step) % 1.0)) for b in range(n)]


def _sizes(case):
    B = case["batch"]
    return (_spread(case.get("plo", 0), case.get("phi", 0), B, 0.6180339887),
            _spread(case["nlo"], case["nhi"], B, 0.4142135623))


def work(case):
    """Bytes and operations of one pass: every input the operator has to see read once, every output written once."""
    P, N = _sizes(case)
    R = sum(N)
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "steer":
        B, V = case["batch"], case["vocab"]
        return {"bytes": 2.0 * R * V * es + 2.0 * B * V + (R * V / 8 if case["mask"] else 0) + 8.0 * B * case["bias"],
                "flops": 6.0 * R * V}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":                                  # K and V go to the rows and to the cache
        return {"bytes": 1.0 * R * d * es * (2 * hq + 6 * hkv), "flops": 3.0 * R * d * (hq + hkv)}
    seen = sum(n * p + n * (n + 1) // 2 for p, n in zip(P, N))
    return {"bytes": 2.0 * R * hq * d * es + 2.0 * (sum(P) + R) * hkv * d * es, "flops": 4.0 * d * hq * seen}


# ------------------------------------------------------------------ inputs

def _values(gen, shape, dtype, heavy=False):
    x = torch.randn(shape, generator=gen, device="cuda")
    if heavy:                                                 # a few channels of K are larger than the rest
        x = x * (1 + 3 * (torch.arange(shape[-1], device="cuda") % 37 == 5))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator("cpu").manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    P, N = _sizes(case)
    R, mp, mn = sum(N), max(P), max(N)
    i32 = dict(dtype=torch.int32, device="cuda")
    offs = [0]
    for n in N:
        offs.append(offs[-1] + n)
    st = dict(case=case, dt=dt, mp=mp, mn=mn, R=R, prefix=torch.tensor(P, **i32), offsets=torch.tensor(offs, **i32),
              status=torch.zeros(4, **i32))
    j = torch.arange(mn, device="cuda")
    st["live"] = j < torch.tensor(N, device="cuda")[:, None]
    st["row_of"] = (torch.tensor(offs[:-1], device="cuda")[:, None] + j).clamp(max=R - 1)
    (_prepare_steer if case["op"] == "steer" else _prepare_rows)(st, gen, cpu, P, N, offs)
    return st


def _prepare_rows(st, gen, cpu, P, N, offs):
    case, dt, R = st["case"], st["dt"], st["R"]
    B, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    blocks = [-(-(p + n) // PAGE) + 1 for p, n in zip(P, N)]
    cols = max(blocks)
    st["cap"] = cols * PAGE
    if case["paged"]:                                         # every sequence's pages in shuffled order
        perm = torch.randperm(sum(blocks), generator=cpu).tolist()
        table, at = [], 0
        for n in blocks:
            table.append(perm[at:at + n] + [0] * (cols - n))
            at += n
        st["table"], st["pages"] = torch.tensor(table, dtype=torch.int32, device="cuda"), sum(blocks)
        pool = (sum(blocks), hkv, PAGE, d)
    else:
        st["table"], st["pages"] = None, 0
        pool = (B, hkv, cols * PAGE, d)
    st["k_cache"], st["v_cache"] = _values(gen, pool, dt, True), _values(gen, pool, dt)
    st["q"] = _values(gen, (R, hq, d), dt)
    st["out"] = torch.empty(R, hq, d, dtype=dt, device="cuda")
    if case["op"] == "attn":
        st["k_rows"], st["v_rows"] = _values(gen, (hkv, R, d), dt, True), _values(gen, (hkv, R, d), dt)
        return
    st["k"], st["v"] = _values(gen, (R, hkv, d), dt, True), _values(gen, (R, hkv, d), dt)
    st["k_rows"] = torch.empty(hkv, R, d, dtype=dt, device="cuda")
    st["v_rows"] = torch.empty_like(st["k_rows"])
    st["new_prefix"] = torch.empty(B, dtype=torch.int32, device="cuda")


def _prepare_steer(st, gen, cpu, P, N, offs):
    case, R = st["case"], st["R"]
    B, V, nb = case["batch"], case["vocab"], case["bias"]
    st["logits"] = (torch.randn(R, V, generator=gen, device="cuda") * 3).to(st["dt"])
    st["out"] = torch.empty_like(st["logits"])
    # what a sequence has read and written: 500 prompt tokens and 200 emitted ones, some of them often
    width = -(-V // 8) * 8
    zipf = lambda n: (V * torch.rand(B, n, generator=gen, device="cuda") ** 4).long().clamp(max=V - 1)  # noqa: E731
    counts = torch.zeros(B, width, dtype=torch.int64, device="cuda")
    emitted = zipf(200)
    counts.scatter_add_(1, emitted, torch.ones_like(emitted))
    read = torch.zeros(B, width, dtype=torch.int64, device="cuda").scatter_(1, zipf(500), 1)
    st["counts"] = (counts - 32768 * read).to(torch.int16)    # bit 15 is the sign of a 16-bit number
    st["penalties"] = torch.stack([1 + 0.3 * torch.rand(B, generator=gen, device="cuda"),
                                   0.5 * torch.rand(B, generator=gen, device="cuda"),
                                   torch.rand(B, generator=gen, device="cuda")], 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    if nb:
        st["bias_offsets"] = torch.arange(B + 1, **i32) * nb
        st["bias_tokens"] = torch.stack([torch.randperm(V, generator=gen, device="cuda")[:nb] for _ in range(B)]).int()
        st["bias_values"] = torch.randn(B, nb, generator=gen, device="cuda") * 4
    if case["mask"]:
        # most states of a grammar allow few tokens, some nearly all
        words = -(-V // 32)
        w = torch.randint(-2 ** 31, 2 ** 31, (R, words), generator=gen, device="cuda")
        few = w & torch.roll(w, 1, 1) & torch.roll(w, 2, 1) & torch.roll(w, 3, 1) & torch.roll(w, 5, 1)
        st["mask"] = torch.where(torch.arange(R, device="cuda")[:, None] % 3 == 0, w | torch.roll(w, 7, 1), few).int()
    draft, anc = [], []
    for n in N:
        pick = torch.rand(n, generator=cpu).tolist()
        base = len(anc)
        for i in range(n):
            up = max(0, i - 1 - int(pick[i] * min(i, 9)))
            anc.append(1 << i | (anc[base + up] if i else 0))
    st["anc"] = torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64, device="cuda")
    st["draft"] = (V * torch.rand(R, generator=gen, device="cuda") ** 4).int().clamp(max=V - 1)


# ------------------------------------------------------------------ the operators

def run(state):
    if own:
        return _run_own(state)
    return {"attn": _plain_attn, "rope": _plain_rope, "steer": _plain_steer}[state["case"]["op"]](state)


def _plain_attn(st):
    c = st["case"]
    B, hq, hkv, d, mn, mp = c["batch"], c["hq"], c["hkv"], c["d"], st["mn"], st["mp"]
    G, rows, P = hq // hkv, st["row_of"], st["prefix"].long()
    kn, vn = (x.float()[:, rows].transpose(0, 1) for x in (st["k_rows"], st["v_rows"]))          # [B, Hkv, mn, d]
    k, v = st["k_cache"], st["v_cache"]
    if c["paged"]:
        k, v = (x[st["table"].long()].transpose(1, 2).flatten(2, 3) for x in (k, v))
    k, v = torch.cat([k[:, :, :mp].float(), kn], 2), torch.cat([v[:, :, :mp].float(), vn], 2)
    q = st["q"].float()[rows].reshape(B, mn, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * mn, d)
    t, i = torch.arange(mp, device=q.device), torch.arange(mn, device=q.device)
    past = (t < P[:, None])[:, None].expand(B, mn, mp)
    here = (i <= i[:, None]) & st["live"][:, None]
    hide = ~torch.cat([past, here], -1)[:, None, None]                                           # [B, 1, 1, mn, keys]
    s = (q @ k.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(B, hkv, G, mn, -1)
    s = s.masked_fill_(hide, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    s = s.div_(s.sum(-1, keepdim=True)).view(B, hkv, G * mn, -1)
    o = (s @ v).view(B, hkv, G, mn, d).permute(0, 3, 1, 2, 4).reshape(B, mn, hq, d)
    return o[st["live"]].to(st["dt"])


def _plain_rope(st):
    c, dt = st["case"], st["dt"]
    d, live, rows = c["d"], st["live"], st["row_of"]
    i = torch.arange(st["mn"], device=live.device)
    pos = (st["prefix"].long()[:, None] + i)[live]                                               # [R]
    freq = THETA ** (-2.0 * torch.arange(d // 2, device=live.device, dtype=torch.float64) / d)
    a = pos[:, None].double() * freq
    co, si = a.cos().float()[:, None], a.sin().float()[:, None]

    def turn(x):
        x = x.float()
        lo, hi = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([lo * co - hi * si, hi * co + lo * si], -1).to(dt)

    q, k, v = turn(st["q"]), turn(st["k"]), st["v"]
    b = torch.arange(c["batch"], device=live.device)[:, None].expand(live.shape)[live]
    if c["paged"]:
        at = (st["table"].long()[b, pos // PAGE], slice(None), pos % PAGE)
    else:
        at = (b, slice(None), pos)
    st["k_cache"][at], st["v_cache"][at] = k, v
    n = (st["offsets"][1:] - st["offsets"][:-1])
    return {"q": q, "k_rows": k.transpose(0, 1).contiguous(), "v_rows": v.transpose(0, 1).contiguous(),
            "k_cache": st["k_cache"], "v_cache": st["v_cache"], "prefix": st["prefix"] + n}


def _plain_steer(st):
    c, mn = st["case"], st["mn"]
    V, R, dev = c["vocab"], st["R"], st["logits"].device
    live, rows = st["live"], st["row_of"]
    seq = torch.arange(c["batch"], device=dev)[:, None].expand(live.shape)[live]                 # [R]
    table = st["counts"][:, :V]
    times = (table & 32767).float()[seq]
    node = torch.arange(mn, device=dev)
    on = (st["anc"][:, None] >> node & 1 == 1) & (node > 0)                                      # drafts on the path
    times.scatter_add_(1, st["draft"].long()[rows][seq], on.float())
    rep, freq, pres = st["penalties"][seq].T[..., None]
    x = st["logits"].float()
    seen = (table < 0)[seq] | (times > 0)
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * times - pres * (times > 0)
    if c["bias"]:
        x = x.scatter_add(1, st["bias_tokens"].long()[seq], st["bias_values"][seq])
    if c["mask"]:
        bit = torch.arange(32, device=dev)
        allow = (st["mask"][..., None] >> bit & 1).bool().flatten(1)[:, :V]
        x = x.masked_fill(~allow, -math.inf)
    return x.to(st["dt"])


def _plan(st):
    """The descriptor and workspace that a program keeps between its calls."""
    import speculative_decoding_tree_gb300 as tv
    c = st["case"]
    if c["op"] == "steer":
        st["desc"] = tv.make_logits_desc(batch=c["batch"], vocab=c["vocab"], max_nodes=st["mn"], total_rows=st["R"],
                                         logits_dtype=tv.BF16 if c["dtype"] == "bf16" else tv.F32,
                                         biases=c["batch"] * c["bias"])
    else:
        st["desc"] = tv.make_desc(
            batch=c["batch"], num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
            dtype=tv.BF16 if c["dtype"] == "bf16" else tv.F32, max_nodes=1, total_rows=c["batch"], capacity=st["cap"],
            max_prefix=st["mp"], page_size=PAGE if c["paged"] else 0, num_pages=st["pages"])
    if c["op"] == "attn":
        st["ws_bytes"] = tv.tv_prompt_workspace_size(st["desc"], st["R"], st["mn"])
        st["ws"] = torch.empty(max(st["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    st["tv"] = tv


def _run_own(st):
    if "tv" not in st:
        _plan(st)
    tv, op = st["tv"], st["case"]["op"]
    if op == "attn":
        tv.tv_prompt_attn(st["desc"], st["R"], st["mn"], st["q"], st["k_cache"], st["v_cache"], st["table"],
                          st["prefix"], st["offsets"], st["k_rows"], st["v_rows"], st["out"], st["ws"],
                          st["ws_bytes"], st["status"])
        return st["out"]
    if op == "rope":
        tv.tv_prompt_rope_store(st["desc"], st["R"], st["mn"], THETA, st["q"], st["k"], st["v"], st["prefix"],
                                st["offsets"], st["out"], st["k_rows"], st["v_rows"], st["k_cache"], st["v_cache"],
                                st["table"], st["new_prefix"], st["status"])
        return {"q": st["out"], "k_rows": st["k_rows"], "v_rows": st["v_rows"], "k_cache": st["k_cache"],
                "v_cache": st["v_cache"], "prefix": st["new_prefix"]}
    tv.tv_tree_logits_process(st["desc"], st["logits"], st["counts"], st["penalties"], st.get("bias_offsets"),
                              st.get("bias_tokens"), st.get("bias_values"), st.get("mask"), st["draft"],
                              st["offsets"], st["anc"], st["out"], st["status"])
    return st["out"]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    P, N = _sizes(case)
    offs = st["offsets"].tolist()
    return {"attn": _exact_attn, "rope": _exact_rope, "steer": _exact_steer}[case["op"]](st, P, N, offs)


def _exact_attn(st, P, N, offs):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G = hq // hkv
    out = torch.empty(st["R"], hq, d, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        p, n, o = P[b], N[b], offs[b]
        t = torch.arange(p, device="cuda")
        for g in range(hkv):
            ids = st["table"][b].long()[t // PAGE] if c["paged"] else None
            past = [x[ids, g, t % PAGE] if c["paged"] else x[b, g, :p] for x in (st["k_cache"], st["v_cache"])]
            k = torch.cat([past[0], st["k_rows"][g, o:o + n]]).double()
            v = torch.cat([past[1], st["v_rows"][g, o:o + n]]).double()
            for i in range(0, n, 2048):                       # rows i .. m - 1 see the keys 0 .. p + m - 1
                m = min(n, i + 2048)
                q = st["q"][o + i:o + m, g * G:(g + 1) * G].double().transpose(0, 1)
                s = q @ k[:p + m].T / d ** 0.5
                at = torch.arange(p + m, device="cuda")
                s.masked_fill_(at > p + torch.arange(i, m, device="cuda")[:, None], -math.inf)
                out[o + i:o + m, g * G:(g + 1) * G] = (torch.softmax(s, -1) @ v[:p + m]).transpose(0, 1)
    return out


def _exact_rope(st, P, N, offs):
    c = st["case"]
    d = c["d"]
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    for b in range(c["batch"]):
        pos = P[b] + torch.arange(N[b], device="cuda")
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.outer(
            pos.double(), torch.exp(-math.log(THETA) * torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)))
        sl = slice(offs[b], offs[b + 1])
        for x in (q, k):
            y = torch.complex(x[sl, :, :d // 2].contiguous(), x[sl, :, d // 2:].contiguous()) * z[:, None]
            x[sl] = torch.cat([y.real, y.imag], -1)
        for x, cache in ((k, kc), (v, vc)):
            if c["paged"]:
                cache[st["table"][b].long()[pos // PAGE], :, pos % PAGE] = x[sl]
            else:
                cache[b, :, pos] = x[sl].transpose(0, 1)
    return {"q": q, "k_rows": k.transpose(0, 1).contiguous(), "v_rows": v.transpose(0, 1).contiguous(), "k_cache": kc,
            "v_cache": vc, "prefix": None}


def _exact_steer(st, P, N, offs):
    c = st["case"]
    V = c["vocab"]
    out = st["logits"].double()
    anc, draft = st["anc"].tolist(), st["draft"].tolist()
    for b in range(c["batch"]):
        rep, freq, pres = st["penalties"][b].double()
        base = st["counts"][b, :V].long()
        told, base = base < 0, base % 32768
        bias = torch.zeros(V, dtype=torch.float64, device="cuda")
        if c["bias"]:
            bias[st["bias_tokens"][b].long()] = st["bias_values"][b].double()
        for r in range(offs[b], offs[b + 1]):
            path = [draft[offs[b] + j] for j in range(1, N[b]) if anc[r] >> j & 1]
            times = base + torch.bincount(torch.tensor(path, dtype=torch.long, device="cuda"), minlength=V)
            x, hit = out[r], times > 0
            x = torch.where(told | hit, torch.where(x > 0, x / rep, x * rep), x) - freq * times - pres * hit + bias
            if c["mask"]:
                token = torch.arange(V, device="cuda")
                x[st["mask"][r].long()[token // 32] >> token % 32 & 1 == 0] = -math.inf
            out[r] = x
    return out
