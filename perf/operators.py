"""Measured cases of the serving operators over a paged KV cache.

  append   kv_rope_append_paged   new tokens' keys and values into their pages, keys and queries rotated on the way
  window   kv_window_attn_paged   causal attention over a few first tokens (sink) and the newest `local` ones
  prefix   kv_prefix_attn_paged   attention of many sequences over one shared prefix and their own tokens

A case says which operator runs and over what: B sequences of up to `q` new
tokens each, `n` cached tokens (the new ones among them), Hq / Hkv heads of
128 values, pages of P tokens.  A ragged case gives every sequence its own
lengths, drawn from the case alone.  Head layouts, sink, local window and
context lengths are those of the library's decode workloads.
"""

import math

import torch

own = False

D = 128
SINK = 4


def listed():
    return [
        # One decode step of four 128K-context sequences: a single new token
        # each; the smallest call, where latency counts.
        dict(name="append_step", op="append", B=4, q=1, n=131072, ragged=False, Hq=32, Hkv=8, P=256, rot=128,
             interleaved=False),
        # A ragged chunk of seven requests, adjacent-pair rotation of half
        # the head, small pages that end inside every chunk.
        dict(name="append_ragged", op="append", B=7, q=509, n=6000, ragged=True, Hq=8, Hkv=2, P=64, rot=64,
             interleaved=True),
        # A whole 32K prompt of the 64-head layout.
        dict(name="append_prompt", op="append", B=1, q=32768, n=32768, ragged=False, Hq=64, Hkv=8, P=256, rot=128,
             interleaved=False),
        # The decode workload's sink and local tokens alone.
        dict(name="window_step", op="window", B=4, q=1, n=131072, ragged=False, Hq=32, Hkv=8, P=256, local=256),
        # A serving batch decoding with a 4K window, lengths of all sizes.
        dict(name="window_batch", op="window", B=64, q=1, n=8192, ragged=True, Hq=32, Hkv=8, P=128, local=4096),
        # One long sequence, nothing hidden: the cache is split over the GPU.
        dict(name="window_long", op="window", B=1, q=1, n=131072, ragged=False, Hq=64, Hkv=8, P=256, local=131072),
        # Chunked prefill mixed with single-token sequences, odd sizes.
        dict(name="window_mixed", op="window", B=16, q=257, n=5003, ragged=True, Hq=8, Hkv=2, P=64, local=1000),
        # Prefill of a 32K prompt with a 4K window.
        dict(name="window_prompt", op="window", B=1, q=32768, n=32768, ragged=False, Hq=32, Hkv=8, P=256, local=4096),
        # Prefill of an 8K prompt, plain causal attention, 64 heads.
        dict(name="window_causal", op="window", B=1, q=8192, n=8192, ragged=False, Hq=64, Hkv=8, P=256, local=8192),
        # Four short continuations of one instruction.
        dict(name="prefix_small", op="prefix", B=4, q=1, n=37, ragged=True, Hq=8, Hkv=2, P=64, prefix=1000),
        # 32 answers to questions about one 32K document.
        dict(name="prefix_batch", op="prefix", B=32, q=1, n=512, ragged=True, Hq=32, Hkv=8, P=256, prefix=32768),
        # 128 sequences over a 128K prefix.
        dict(name="prefix_large", op="prefix", B=128, q=1, n=1024, ragged=True, Hq=32, Hkv=8, P=256, prefix=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "window", "window", "prefix"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 2), (8, 8), (16, 8), (8, 1)])
    P = rng.choice([64, 128, 256, 1024])
    case = dict(op=op, Hq=Hq, Hkv=Hkv, P=P, ragged=rng.random() < 0.6)
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, 32768 // B))
        case.update(B=B, q=q, n=q + _log(rng, 1, 100000), rot=rng.choice([32, 64, 128]),
                    interleaved=rng.random() < 0.4)
    elif op == "window" and rng.random() < 0.5:
        # decode and speculative steps
        B = _log(rng, 1, 64)
        n = _log(rng, 16, 131072 // B)
        q = min(n, rng.choice([1, 1, 1, 2, 5]))
        case.update(B=B, q=q, n=n, local=rng.choice([n, _log(rng, 1, 8192)]))
    elif op == "window":
        # prefill and chunks
        B = _log(rng, 1, 8)
        q = _log(rng, 16, 8192 // B)
        case.update(B=B, q=q, n=q + rng.choice([0, _log(rng, 1, 8192)]), local=_log(rng, 16, 4096))
    else:
        B = _log(rng, 1, 64)
        q = rng.choice([1, 1, 1, 3])
        case.update(B=B, q=q, n=q + _log(rng, 1, 1024), prefix=_log(rng, 16, 65536))
    return case


def _spread(b, lo, hi, salt):
    """A length in [lo, hi] for sequence b, spread evenly over the range."""
    return lo + ((b + 1) * 2654435761 + salt * 40503) % (1 << 32) * (hi - lo + 1) // (1 << 32)


def _lengths(case):
    """Per sequence: new tokens and cached tokens (the new ones among them)."""
    B, q, n = case["B"], case["q"], case["n"]
    if not case["ragged"]:
        return [q] * B, [n] * B
    ql = [1 if b % 4 == 3 else _spread(b, 1, q, 1) for b in range(B)]
    kl = [_spread(b, max(ql[b], n // 4), n, 2) for b in range(B)]
    return ql, kl


def _span(pos, local):
    """Tokens that a query at `pos` attends to: the first SINK and the newest `local`."""
    lo = max(0, pos - local + 1)
    return pos + 1 - lo + min(SINK, lo)


def work(case):
    ql, kl = _lengths(case)
    T, Hq, Hkv = sum(ql), case["Hq"], case["Hkv"]
    if case["op"] == "append":
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D * 2 + 12 * T, "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    rows = 2 * T * Hq * D * 2 + 4 * T * Hq      # queries, outputs, log-sum-exps
    if case["op"] == "window":
        local = case["local"]
        keys = sum(k - max(0, k - m - local + 1) + min(SINK, max(0, k - m - local + 1)) for m, k in zip(ql, kl))
        pairs = sum(_span(k - m + i, local) for m, k in zip(ql, kl) for i in range(m))
    else:
        keys = case["prefix"] + sum(kl)
        pairs = T * case["prefix"] + sum(m * (k - m) + m * (m + 1) // 2 for m, k in zip(ql, kl))
    return {"bytes": keys * Hkv * D * 2 * 2 + rows, "flops": 4 * D * Hq * pairs}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ql, kl = _lengths(case)
    B, T, Hq, Hkv, P = case["B"], sum(ql), case["Hq"], case["Hkv"], case["P"]
    st = dict(op=case["op"], Hq=Hq, Hkv=Hkv, P=P, qmax=max(ql), nmax=max(kl))

    def bf16(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    # Pages in a random order; the pool has a few that belong to nobody.  An
    # append needs only the pages that it writes to: older ones of long
    # contexts are page 0 of the pool, which nothing touches.
    pps = -(-max(kl) // P)
    firsts = [(k - m) // P if case["op"] == "append" else 0 for m, k in zip(ql, kl)]
    used = sum(-(-k // P) - f for k, f in zip(kl, firsts))
    prefix_pages = -(-case["prefix"] // P) if case["op"] == "prefix" else 0
    num_pages = 1 + used + prefix_pages + 3
    order = (1 + torch.randperm(num_pages - 1, generator=gen, device=dev)).to(torch.int32)
    table = torch.zeros((B, pps), dtype=torch.int32, device=dev)
    cu, at = [0], 0
    for b, (m, k, f) in enumerate(zip(ql, kl, firsts)):
        pages = -(-k // P) - f
        table[b, f:f + pages] = order[at:at + pages]
        at += pages
        cu.append(cu[-1] + m)
    st["K_pool"] = bf16(num_pages, Hkv, P, D)
    st["V_pool"] = bf16(num_pages, Hkv, P, D)
    st["table"] = table
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if st["qmax"] > 1 else None
    st["lens"] = torch.tensor(kl, dtype=torch.int32, device=dev)

    if case["op"] == "append":
        # the projection's output: queries, keys and values side by side
        qkv = bf16(T, Hq + 2 * Hkv, D)
        st["q"], st["k"], st["v"] = qkv.split([Hq, Hkv, Hkv], dim=1)
        half = case["rot"] // 2
        st["inv_freq"] = (500000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        st["interleaved"] = case["interleaved"]
        st["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        return st
    st["q"] = bf16(T, Hq, D)
    if case["op"] == "window":
        st["local"] = case["local"]
    else:
        st["prefix"] = case["prefix"]
        st["prefix_table"] = order[at:at + prefix_pages].contiguous()
    st["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    if own:
        import query_aware_sparse_compressed_gb300 as qasc
        size = (qasc.kv_window_attn_workspace_bytes if case["op"] == "window" else
                qasc.kv_prefix_attn_workspace_bytes)
        st["ws"] = qasc.alloc_workspace(size(T, B, Hq, Hkv, pps * P))
    return st


def run(state):
    if own:
        return _call(state)
    return {"append": _append, "window": _window, "prefix": _prefix}[state["op"]](state)


def _call(s):
    import query_aware_sparse_compressed_gb300 as qasc
    if s["op"] == "append":
        qasc.kv_rope_append_paged(s["q"], s["k"], s["v"], s["q_out"], s["K_pool"], s["V_pool"], s["table"], s["lens"],
                                  s["inv_freq"], cu_q=s["cu"], interleaved=s["interleaved"])
        return dict(q=s["q_out"], K_pool=s["K_pool"], V_pool=s["V_pool"])
    if s["op"] == "window":
        qasc.kv_window_attn_paged(s["q"], s["K_pool"], s["V_pool"], s["table"], s["lens"], s["out"], s["ws"],
                                  sink=SINK, local=s["local"], cu_q=s["cu"], lse=s["lse"])
    else:
        qasc.kv_prefix_attn_paged(s["q"], s["K_pool"], s["V_pool"], s["prefix_table"], s["table"], s["lens"],
                                  s["out"], s["ws"], n_prefix=s["prefix"], cu_q=s["cu"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


# ------------------------------------------------------------- plain forms
def _tokens(s):
    """Of every new token: its sequence, its place among that sequence's new
    tokens, its position in the cache; and per sequence: first token, count,
    cached tokens."""
    lens = s["lens"].long()
    T = s["q"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(T + 1, device=lens.device)
    t = torch.arange(T, device=lens.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    ql = cu[1:] - cu[:-1]
    return b, i, lens[b] - ql[b] + i, cu[:-1], ql, lens


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] with its first rot values rotated by the angles of [T, 1, rot / 2]."""
    half = cos.shape[-1]
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return torch.cat([y, rest], dim=-1).to(torch.bfloat16)


def _append(s):
    b, _, pos, _, _, _ = _tokens(s)
    angle = pos.double()[:, None] * s["inv_freq"].double()      # angles of far positions need 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    page, row = s["table"][b, pos // s["P"]].long(), pos % s["P"]
    s["K_pool"][page, :, row] = _rotate(s["k"], cos, sin, s["interleaved"])
    s["V_pool"][page, :, row] = s["v"]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, s["interleaved"]))
    return dict(q=s["q_out"], K_pool=s["K_pool"], V_pool=s["V_pool"])


def _rows(s, pool, table, j):
    """pool's rows of logical tokens j [B, m] as fp32 [B, Hkv, m, D]."""
    page = torch.gather(table.long(), 1, j // s["P"])
    return pool[page, :, j % s["P"]].float().transpose(1, 2)


def _softmax_parts(z):
    """Row maximum, exp(z - maximum), their sum."""
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - m)
    return m, p, p.sum(dim=-1, keepdim=True)


def _window(s):
    first, ql, lens = _tokens(s)[3:]
    T, Hq, Hkv, local = s["q"].shape[0], s["Hq"], s["Hkv"], s["local"]
    G, B, dev = Hq // Hkv, lens.numel(), lens.device
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    sink = torch.arange(SINK, device=dev)
    for i0 in range(0, s["qmax"], 1024):      # queries of a sequence, a block at a time
        m = min(1024, s["qmax"] - i0)
        i = i0 + torch.arange(m, device=dev)
        there = i < ql[:, None]                                            # [B, m]
        pos = lens[:, None] - ql[:, None] + i                              # [B, m]
        lo = (pos[:, :1] - local + 1).clamp(min=SINK)
        last = min(i0 + m, s["qmax"]) - 1
        span = max(1, min(local + m - 1, s["nmax"] - s["qmax"] + 1 + last if B == 1 else s["nmax"]))
        j = torch.cat([sink.expand(B, SINK), lo + torch.arange(span, device=dev)], dim=1)
        seen = (j[:, None] <= pos[..., None]) & ((j[:, None] > pos[..., None] - local) | (j[:, None] < SINK))
        seen |= ~there[..., None]                                          # padding of short sequences
        jc = j.clamp(max=s["nmax"] - 1)
        K, V = _rows(s, s["K_pool"], s["table"], jc), _rows(s, s["V_pool"], s["table"], jc)
        t = (first[:, None] + i).clamp(max=T - 1)
        q = s["q"][t].float().reshape(B, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, D)
        z = (q @ K.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).reshape(B, Hkv, G, m, -1)
        z.masked_fill_(~seen[:, None, None], -math.inf)
        top, p, total = _softmax_parts(z)
        o = (p.reshape(B, Hkv, G * m, -1) @ V).reshape(B, Hkv, G, m, D) / total
        o, e = o.permute(0, 3, 1, 2, 4).reshape(B, m, Hq, D), (top + total.log())[..., 0].permute(0, 3, 1, 2)
        out[t[there]] = o[there].to(torch.bfloat16)
        lse[t[there]] = e.reshape(B, m, Hq)[there]
    return dict(out=out, lse=lse)


def _prefix(s):
    b, i, pos, first, ql, lens = _tokens(s)
    T, Hq, Hkv, n0 = s["q"].shape[0], s["Hq"], s["Hkv"], s["prefix"]
    G, B, m, dev = Hq // Hkv, lens.numel(), s["qmax"], lens.device
    q = s["q"].float()
    jp = torch.arange(n0, device=dev)[None]
    table0 = s["prefix_table"][None]
    K0, V0 = _rows(s, s["K_pool"], table0, jp)[0], _rows(s, s["V_pool"], table0, jp)[0]    # [Hkv, n0, D]
    js = torch.arange(s["nmax"], device=dev).expand(B, -1)
    K1, V1 = _rows(s, s["K_pool"], s["table"], js), _rows(s, s["V_pool"], s["table"], js)  # [B, Hkv, nmax, D]
    z0 = q.reshape(T, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, T * G, D) @ K0.transpose(1, 2)
    z0 = z0.reshape(Hkv, T, G, n0).permute(1, 0, 2, 3)                                     # [T, Hkv, G, n0]
    t = (first[:, None] + torch.arange(m, device=dev)).clamp(max=T - 1)                    # [B, m]
    qs = q[t].reshape(B, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, D)
    z1 = (qs @ K1.transpose(2, 3)).reshape(B, Hkv, G, m, -1).permute(0, 3, 1, 2, 4)[b, i]  # [T, Hkv, G, nmax]
    z1 = z1.masked_fill(js[0] > pos[:, None, None, None], -math.inf)
    top, p, total = _softmax_parts(torch.cat([z0, z1], dim=-1).mul_(1.0 / math.sqrt(D)))
    p0 = p[..., :n0].permute(1, 0, 2, 3).reshape(Hkv, T * G, n0)
    o0 = (p0 @ V0).reshape(Hkv, T, G, D).permute(1, 0, 2, 3)
    p1 = torch.zeros((B, m, Hkv, G, s["nmax"]), device=dev)
    p1[b, i] = p[..., n0:]
    o1 = p1.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, -1) @ V1
    o1 = o1.reshape(B, Hkv, G, m, D).permute(0, 3, 1, 2, 4)[b, i]
    out = ((o0 + o1) / total).reshape(T, Hq, D).to(torch.bfloat16)
    return dict(out=out, lse=(top + total.log())[..., 0].reshape(T, Hq))


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["P"]
    G = Hq // Hkv
    starts = [sum(ql[:b]) for b in range(len(ql))]

    def cached(pool, pages, n, g):
        """Rows 0..n-1 of KV head g through a list of pages."""
        return pool[pages.long(), g].reshape(-1, D)[:n].double()

    if case["op"] == "append":
        q, Kp, Vp = s["q"].double().contiguous(), s["K_pool"].double(), s["V_pool"].double()
        k, v = s["k"].double(), s["v"].double()
        half = case["rot"] // 2
        e = torch.arange(half, device="cuda")
        a0, a1 = (2 * e, 2 * e + 1) if case["interleaved"] else (e, e + half)
        for b, (t0, m, n) in enumerate(zip(starts, ql, kl)):
            j = torch.arange(n - m, n, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               j.double()[:, None] * s["inv_freq"].double()[None])[:, None]
            rows = []
            for x in (q[t0:t0 + m], k[t0:t0 + m].clone()):
                y = torch.complex(x[..., a0], x[..., a1]) * turn
                x[..., a0], x[..., a1] = y.real, y.imag
                rows.append(x)
            q[t0:t0 + m] = rows[0]
            page = s["table"][b].long()[j // P]
            Kp[page, :, j % P] = rows[1]
            Vp[page, :, j % P] = v[t0:t0 + m]
        return dict(q=q, K_pool=Kp, V_pool=Vp)

    T = sum(ql)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    n0 = case.get("prefix", 0)
    local = case.get("local", max(kl))
    shared = [(cached(s["K_pool"], s["prefix_table"], n0, g), cached(s["V_pool"], s["prefix_table"], n0, g))
              for g in range(Hkv)] if n0 else None
    for b, (t0, m, n) in enumerate(zip(starts, ql, kl)):
        for g in range(Hkv):
            K, V = cached(s["K_pool"], s["table"][b], n, g), cached(s["V_pool"], s["table"][b], n, g)
            for i0 in range(0, m, 512):
                i1 = min(m, i0 + 512)
                p0, p1 = n - m + i0, n - m + i1          # positions p0 .. p1 - 1
                lo = max(0, p0 - local + 1)
                head = min(SINK, lo) if case["op"] == "window" else 0
                Kb, Vb = torch.cat([K[:head], K[lo:p1]]), torch.cat([V[:head], V[lo:p1]])
                at = torch.cat([torch.arange(head, device="cuda"), torch.arange(lo, p1, device="cuda")])
                pos = torch.arange(p0, p1, device="cuda")[:, None]
                hidden = (at > pos) | ((at <= pos - local) & (at >= SINK))
                if n0:
                    Kb, Vb = torch.cat([shared[g][0], Kb]), torch.cat([shared[g][1], Vb])
                    hidden = torch.cat([torch.zeros((i1 - i0, n0), dtype=torch.bool, device="cuda"), hidden], dim=1)
                for h in range(g * G, (g + 1) * G):
                    x = (s["q"][t0 + i0:t0 + i1, h].double() @ Kb.T) / math.sqrt(D)
                    x[hidden] = -math.inf
                    e = torch.logsumexp(x, dim=1)
                    lse[t0 + i0:t0 + i1, h] = e
                    out[t0 + i0:t0 + i1, h] = torch.exp(x - e[:, None]) @ Vb
    return dict(out=out, lse=lse)
