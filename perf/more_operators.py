"""Measured cases of the serving operators over a 4-bit paged KV cache.

  append   kv4_rope_append_paged, kv4_read_paged   new tokens quantised into their pages, keys and queries rotated on
                                                   the way, and the new keys and values read back as the cache holds them
  read     kv4_read_paged                          whole contexts read back in bf16
  window   kv4_window_attn_paged                   causal attention over a few first tokens and the newest `local` ones
  sparse   kv4_sparse_attn_paged                   one decode step over first, selected and newest tokens

The cache holds a head's 128 values as 64 bytes of codes and 8 scales: value = scale * code, the code a 4-bit float
(sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), one e4m3 scale for each 16 values.

A case says which operator runs and over what: B sequences of up to `q` new tokens each, `n` cached tokens (the new
ones among them), Hq / Hkv heads, pages of P tokens.  A ragged case gives every sequence its own lengths, drawn from
the case alone.  Head layouts, sink, local window, budgets and context lengths are those of the library's decode
workloads.
"""

import math

import torch

own = False

D = 128
GROUP = 16
SINK = 4
LOCAL = 256


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
        # Sixteen contexts of all sizes, read back for a call that takes bf16.
        dict(name="read_ragged", op="read", B=16, n=5003, ragged=True, Hq=8, Hkv=2, P=64),
        # One 128K context.
        dict(name="read_long", op="read", B=1, n=131072, ragged=False, Hq=64, Hkv=8, P=256),
        # The decode workload's sink and local tokens alone.
        dict(name="window_step", op="window", B=4, q=1, n=131072, ragged=False, Hq=32, Hkv=8, P=256, local=256),
        # A serving batch decoding with a 4K window, lengths of all sizes.
        dict(name="window_batch", op="window", B=64, q=1, n=8192, ragged=True, Hq=32, Hkv=8, P=128, local=4096),
        # One long sequence, nothing hidden: the cache is split over the GPU.
        dict(name="window_long", op="window", B=1, q=1, n=131072, ragged=False, Hq=64, Hkv=8, P=256, local=131072),
        # Chunked prefill mixed with single-token sequences, odd sizes.
        dict(name="window_mixed", op="window", B=16, q=257, n=5003, ragged=True, Hq=8, Hkv=2, P=64, local=1000),
        # The last 2K chunk of a 32K prompt, everything before it in the cache.
        dict(name="window_chunk", op="window", B=1, q=2048, n=32768, ragged=False, Hq=32, Hkv=8, P=256, local=32768),
        # A 4K context at a 10 % budget, one list for all heads.
        dict(name="sparse_small", op="sparse", B=1, n=4096, ragged=False, Hq=8, Hkv=2, P=64, permille=100,
             per_head=False),
        # Four 128K contexts at a 20 % budget, a list and a length for every KV head.
        dict(name="sparse_long", op="sparse", B=4, n=131072, ragged=True, Hq=32, Hkv=8, P=256, permille=200,
             per_head=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "window", "window", "sparse"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 2), (8, 8), (16, 8), (8, 1)])
    case = dict(op=op, Hq=Hq, Hkv=Hkv, P=rng.choice([64, 128, 256, 1024]), ragged=rng.random() < 0.6)
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, 32768 // B))
        case.update(B=B, q=q, n=q + _log(rng, 1, 100000), rot=rng.choice([32, 64, 128]),
                    interleaved=rng.random() < 0.4)
    elif op == "read":
        B = _log(rng, 1, 64)
        case.update(B=B, n=_log(rng, 1, 131072 // B))
    elif op == "window" and rng.random() < 0.6:
        # decode and speculative steps
        B = _log(rng, 1, 64)
        n = _log(rng, 16, 131072 // B)
        q = min(n, rng.choice([1, 1, 1, 2, 5, 9]))
        case.update(B=B, q=q, n=n, local=rng.choice([n, _log(rng, 1, 8192)]))
    elif op == "window":
        # prefill and chunks
        B = _log(rng, 1, 8)
        q = _log(rng, 16, 3500 // B)
        case.update(B=B, q=q, n=q + rng.choice([0, _log(rng, 1, 8192)]), local=_log(rng, 16, 8192))
    else:
        B = _log(rng, 1, 8)
        case.update(B=B, n=_log(rng, 300, 262144 // B), permille=rng.choice([50, 100, 150, 200, 300]),
                    per_head=rng.random() < 0.5)
    return case


def _spread(b, lo, hi, salt):
    """A length in [lo, hi] for sequence b, spread evenly over the range."""
    return lo + ((b + 1) * 2654435761 + salt * 40503) % (1 << 32) * (hi - lo + 1) // (1 << 32)


def _lengths(case):
    """Per sequence: new tokens (of a read: all) and cached tokens (the new ones among them)."""
    B, n = case["B"], case["n"]
    if case["op"] == "sparse":
        return [1] * B, [n] * B
    if case["op"] == "read":
        kl = [_spread(b, 1, n, 2) for b in range(B)] if case["ragged"] else [n] * B
        return kl, kl
    q = case["q"]
    if not case["ragged"]:
        return [q] * B, [n] * B
    ql = [1 if b % 4 == 3 else _spread(b, 1, q, 1) for b in range(B)]
    kl = [_spread(b, max(ql[b], n // 4), n, 2) for b in range(B)]
    return ql, kl


def _budget(case):
    """Selected tokens of a list, and the candidates [SINK, c1)."""
    c1 = max(SINK, case["n"] - LOCAL)
    return min(case["n"] * case["permille"] // 1000, c1 - SINK), c1


def _uses(case):
    """Entries in use of every list, [B][lists]."""
    K, _ = _budget(case)
    lists = case["Hkv"] if case["per_head"] else 1
    return [[_spread(b * lists + i, K // 2, K, 3) if case["ragged"] else K for i in range(lists)]
            for b in range(case["B"])]


def _span(pos, local):
    """Tokens that a query at `pos` attends to: the first SINK and the newest `local`."""
    lo = max(0, pos - local + 1)
    return pos + 1 - lo + min(SINK, lo)


def work(case):
    ql, kl = _lengths(case)
    T, Hq, Hkv = sum(ql), case["Hq"], case["Hkv"]
    held = 2 * Hkv * (D // 2 + D // GROUP)      # bytes of a cached token, keys and values
    if case["op"] == "append":
        return {"bytes": T * (2 * Hq * 2 * D + 2 * Hkv * 2 * D + held + 2 * Hkv * 2 * D) + 12 * T,
                "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * D}
    if case["op"] == "read":
        return {"bytes": T * (held + 2 * Hkv * 2 * D), "flops": 2 * T * Hkv * D}
    rows = 2 * T * Hq * D * 2 + 4 * T * Hq      # queries, outputs, log-sum-exps
    if case["op"] == "window":
        local = case["local"]
        keys = sum(k - max(0, k - m - local + 1) + min(SINK, max(0, k - m - local + 1)) for m, k in zip(ql, kl))
        pairs = sum(_span(k - m + i, local) for m, k in zip(ql, kl) for i in range(m))
        return {"bytes": keys * held + rows, "flops": 4 * D * Hq * pairs}
    always = min(SINK, case["n"]) + min(LOCAL, max(0, case["n"] - SINK))
    lists = [always + u for us in _uses(case) for u in us]
    share = Hkv // (Hkv if case["per_head"] else 1)      # KV heads that use a list
    return {"bytes": sum(lists) * share * held // Hkv + 4 * sum(lists) + rows,
            "flops": 4 * D * (Hq // Hkv) * share * sum(lists)}


# --------------------------------------------------------- the 4-bit format
_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """x [..., D] of bf16 values: codes [..., D / 2] (uint8, the even value of a pair in the low half) and scales
    [..., D / GROUP] (e4m3), both rounded to nearest, ties to even."""
    g = x.float().unflatten(-1, (D // GROUP, GROUP))
    six = torch.full((), 6.0, dtype=torch.float64, device=x.device)
    scale = (g.abs().amax(-1).double() / six).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    r = torch.where(s > 0, g.abs() / torch.where(s > 0, s, 1.0), 0.0)
    code = (r > 0.25).to(torch.uint8)
    code += r >= 0.75
    code += r > 1.25
    code += r >= 1.75
    code += r > 2.5
    code += r >= 3.5
    code += r > 5.0
    code = (code | (g < 0).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _values(codes, scales, at=()):
    """The values of the rows `at` of codes [..., D / 2] and scales [..., D / GROUP], fp32."""
    codes, scale = codes[at], scales.view(torch.uint8)[at].view(torch.float8_e4m3fn)
    table = torch.tensor(_CODES + tuple(-c for c in _CODES), device=codes.device)
    c = table[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()]
    return (c.unflatten(-1, (D // GROUP, GROUP)) * scale.float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ql, kl = _lengths(case)
    B, T, Hq, Hkv, P = case["B"], sum(ql), case["Hq"], case["Hkv"], case["P"]
    st = dict(op=case["op"], Hq=Hq, Hkv=Hkv, P=P, qmax=max(ql), nmax=max(kl))

    def bf16(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    # Keys have a few channels of larger values, as those of language models do.
    channels = torch.ones(D, device=dev, dtype=torch.bfloat16)
    channels[torch.randperm(D, generator=gen, device=dev)[:4]] = 4.0

    # Pages in a random order; the pool has a few that belong to nobody.  An
    # append needs only the pages that it writes to: older ones of long
    # contexts are page 0 of the pool, which nothing touches.
    pps = -(-max(kl) // P)
    firsts = [(k - m) // P if case["op"] == "append" else 0 for m, k in zip(ql, kl)]
    num_pages = 1 + sum(-(-k // P) - f for k, f in zip(kl, firsts)) + 3
    order = (1 + torch.randperm(num_pages - 1, generator=gen, device=dev)).to(torch.int32)
    table = torch.zeros((B, pps), dtype=torch.int32, device=dev)
    cu, at = [0], 0
    for b, (m, k, f) in enumerate(zip(ql, kl, firsts)):
        pages = -(-k // P) - f
        table[b, f:f + pages] = order[at:at + pages]
        at += pages
        cu.append(cu[-1] + m)
    pools = []
    for width in (channels, torch.ones_like(channels)):
        codes = torch.empty((num_pages, Hkv, P, D // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((num_pages, Hkv, P, D // GROUP), dtype=torch.float8_e4m3fn, device=dev)
        step = max(1, (1 << 18) // (Hkv * P))
        for i in range(0, num_pages, step):
            codes[i:i + step], scales[i:i + step] = _quantise(bf16(min(step, num_pages - i), Hkv, P, D) * width)
        pools += [codes, scales]
    st["cache"] = tuple(pools)      # codes and scales of the keys, of the values
    st["table"] = table
    st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if st["qmax"] > 1 else None
    st["lens"] = torch.tensor(kl, dtype=torch.int32, device=dev)

    if own:
        import query_aware_sparse_compressed_gb300 as qasc
        st["kv4"] = qasc.KV4(*pools)
    if case["op"] in ("append", "read"):
        st["k_back"] = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev)
        st["v_back"] = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=dev)
    if case["op"] == "read":
        return st
    if case["op"] == "append":
        # the projection's output: queries, keys and values side by side
        qkv = bf16(T, Hq + 2 * Hkv, D)
        qkv[:, Hq:Hq + Hkv] *= channels
        st["q"], st["k"], st["v"] = qkv.split([Hq, Hkv, Hkv], dim=1)
        half = case["rot"] // 2
        st["inv_freq"] = (500000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        st["interleaved"] = case["interleaved"]
        st["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
        return st
    st["q"] = bf16(T, Hq, D)
    st["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    if case["op"] == "window":
        st["local"] = case["local"]
    else:
        K, c1 = _budget(case)
        uses = torch.tensor(_uses(case), dtype=torch.int32, device=dev)
        rows = []
        for b in range(B):
            for i in range(uses.shape[1]):
                picked = SINK + torch.randperm(c1 - SINK, generator=gen, device=dev)[:K]
                u = int(uses[b, i])
                rows.append(torch.cat([picked[:u].sort().values, picked[u:]]))   # those behind u are not in use
        st["sel"] = torch.stack(rows).reshape((B, Hkv, K) if case["per_head"] else (B, K)).to(torch.int32)
        st["lengths"] = (uses if case["per_head"] else uses[:, 0].contiguous()) if case["ragged"] else None
        st["n"], st["per_head"] = case["n"], case["per_head"]
    if own:
        if case["op"] == "window":
            size = qasc.kv4_window_attn_workspace_bytes(T, B, Hq, Hkv, pps * P, max_q=st["qmax"], sink=SINK,
                                                        local=st["local"])
        else:
            size = qasc.kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, case["n"], pps * P, st["sel"].shape[-1], SINK,
                                                        LOCAL)
        st["ws"] = qasc.alloc_workspace(size)
    return st


def run(state):
    if own:
        return _call(state)
    return {"append": _append, "read": _read, "window": _window, "sparse": _sparse}[state["op"]](state)


def _call(s):
    import query_aware_sparse_compressed_gb300 as qasc
    if s["op"] == "append":
        qasc.kv4_rope_append_paged(s["q"], s["k"], s["v"], s["q_out"], s["kv4"], s["table"], s["lens"],
                                   s["inv_freq"], cu_q=s["cu"], interleaved=s["interleaved"])
        qasc.kv4_read_paged(s["kv4"], s["table"], s["lens"], s["k_back"], s["v_back"], cu_q=s["cu"])
        return dict(q=s["q_out"], k=s["k_back"], v=s["v_back"])
    if s["op"] == "read":
        qasc.kv4_read_paged(s["kv4"], s["table"], s["lens"], s["k_back"], s["v_back"], cu_q=s["cu"])
        return dict(k=s["k_back"], v=s["v_back"])
    if s["op"] == "window":
        qasc.kv4_window_attn_paged(s["q"], s["kv4"], s["table"], s["lens"], s["out"], s["ws"], sink=SINK,
                                   local=s["local"], cu_q=s["cu"], max_q=s["qmax"], lse=s["lse"])
    else:
        qasc.kv4_sparse_attn_paged(s["q"], s["kv4"], s["table"], s["sel"], s["out"], s["ws"], n=s["n"], sink=SINK,
                                   local=LOCAL, lengths=s["lengths"], per_kv_head=s["per_head"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


# ------------------------------------------------------------- plain forms
def _tokens(s, T):
    """Of every new token: its sequence, its place among that sequence's new
    tokens, its position in the cache; and per sequence: first token, count,
    cached tokens."""
    lens = s["lens"].long()
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(T + 1, device=lens.device)
    t = torch.arange(T, device=lens.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    ql = cu[1:] - cu[:-1]
    return b, i, lens[b] - ql[b] + i, cu[:-1], ql, lens


def _to_bf16(y):
    """fp64 values rounded once to bf16 (a cast goes by way of fp32)."""
    m, e = torch.frexp(y)
    return torch.ldexp((m * 256.0).round(), e - 8).to(torch.bfloat16)


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] with its first rot values rotated by the angles of [T, 1, rot / 2], in fp64: rounded keys
    may stand next to a border of their codes."""
    half = cos.shape[-1]
    x = x.double()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return _to_bf16(torch.cat([y, rest], dim=-1))


def _read(s):
    T = s["k_back"].shape[0]
    b, _, pos, _, _, _ = _tokens(s, T)
    page, row = s["table"][b, pos // s["P"]].long(), pos % s["P"]
    K, K_sf, V, V_sf = s["cache"]
    s["k_back"].copy_(_values(K, K_sf, (page, slice(None), row)))
    s["v_back"].copy_(_values(V, V_sf, (page, slice(None), row)))
    return dict(k=s["k_back"], v=s["v_back"])


def _append(s):
    b, _, pos, _, _, _ = _tokens(s, s["q"].shape[0])
    angle = pos.double()[:, None] * s["inv_freq"].double()      # angles of far positions need 64 bits
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    page, row = s["table"][b, pos // s["P"]].long(), pos % s["P"]
    K, K_sf, V, V_sf = s["cache"]
    k, k_sf = _quantise(_rotate(s["k"], cos, sin, s["interleaved"]))
    v, v_sf = _quantise(s["v"])
    K[page, :, row], V[page, :, row] = k, v
    K_sf.view(torch.uint8)[page, :, row], V_sf.view(torch.uint8)[page, :, row] = (
        k_sf.view(torch.uint8), v_sf.view(torch.uint8))
    s["q_out"].copy_(_rotate(s["q"], cos, sin, s["interleaved"]))
    return dict(q=s["q_out"], **_read(s))


def _rows(s, j):
    """Key and value rows of logical tokens j [B, m], as fp32 [B, Hkv, m, D]."""
    page, row = torch.gather(s["table"].long(), 1, j // s["P"]), j % s["P"]
    K, K_sf, V, V_sf = s["cache"]
    return [_values(c, f, (page, slice(None), row)).transpose(1, 2) for c, f in ((K, K_sf), (V, V_sf))]


def _softmax_parts(z):
    """Row maximum, exp(z - maximum), their sum."""
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - m)
    return m, p, p.sum(dim=-1, keepdim=True)


def _window(s):
    T, Hq, Hkv, local = s["q"].shape[0], s["Hq"], s["Hkv"], s["local"]
    first, ql, lens = _tokens(s, T)[3:]
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
        K, V = _rows(s, j.clamp(max=s["nmax"] - 1))
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


def _sparse(s):
    B, Hq, Hkv, n, dev = s["q"].shape[0], s["Hq"], s["Hkv"], s["n"], s["q"].device
    G = Hq // Hkv
    sink_end = min(SINK, n)
    always = torch.cat([torch.arange(sink_end, device=dev), torch.arange(max(sink_end, n - LOCAL), n, device=dev)])
    sel = s["sel"].long().reshape(B, -1, s["sel"].shape[-1])
    L, K = sel.shape[1:]
    used = torch.ones((B, L, K), dtype=torch.bool, device=dev)
    if s["lengths"] is not None:
        used = torch.arange(K, device=dev) < s["lengths"].reshape(B, L, 1)
    j = torch.cat([always.expand(B, L, -1), sel], dim=-1).expand(B, Hkv, -1)
    used = torch.cat([torch.ones_like(used[..., :1]).expand(B, L, always.numel()), used], dim=-1).expand(B, Hkv, -1)
    page = torch.gather(s["table"].long(), 1, j.reshape(B, -1) // s["P"]).reshape(j.shape)
    at = (page, torch.arange(Hkv, device=dev)[:, None], j % s["P"])
    K4, K_sf, V4, V_sf = s["cache"]
    Kv, Vv = _values(K4, K_sf, at), _values(V4, V_sf, at)
    z = (s["q"].float().reshape(B, Hkv, G, D) @ Kv.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    z.masked_fill_(~used[:, :, None], -math.inf)
    top, p, total = _softmax_parts(z)
    out = ((p @ Vv) / total).reshape(B, Hq, D).to(torch.bfloat16)
    return dict(out=out, lse=(top + total.log()).reshape(B, Hq))


# ------------------------------------------------- the definition in 64 bits
def _nearest(x, grid):
    """Index of the value of the ascending `grid` nearest to x >= 0 (the last one for all above), ties to the
    even index."""
    mids = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.bucketize(x, mids), torch.bucketize(x, mids, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _held(x):
    """What the cache holds for x [..., D] (fp64): the scales' and codes' nearest values, in fp64."""
    e4m3 = [i / 512 if i < 8 else (8 + i % 8) * 2.0 ** (i // 8 - 10) for i in range(127)]
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device=x.device)
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=x.device) / 2
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    scale = e4m3[_nearest(g.abs().max(-1, keepdim=True).values / torch.full_like(g[..., :1], 6), e4m3)]
    code = grid[_nearest(torch.where(scale > 0, g.abs() / scale, torch.zeros_like(g)), grid)]
    return (torch.copysign(code, g) * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    Hq, Hkv, P = case["Hq"], case["Hkv"], case["P"]
    G = Hq // Hkv
    starts = [sum(ql[:b]) for b in range(len(ql))]
    nibble = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    nibble = torch.cat([nibble, -nibble])

    def rows(kv, b, j, g):
        """Rows j of sequence b's KV head g, keys (kv 0) or values (2)."""
        page = s["table"][b].long()[j // P]
        codes = s["cache"][kv][page, g, j % P].long()
        sf = s["cache"][kv + 1].view(torch.uint8)[page, g, j % P].view(torch.float8_e4m3fn).double()
        x = torch.empty((j.numel(), D), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = nibble[codes % 16], nibble[codes // 16]
        return x * sf.repeat_interleave(GROUP, dim=1)

    if case["op"] == "append":
        q, k, v = (s[x].double().contiguous() for x in "qkv")
        half = case["rot"] // 2
        e = torch.arange(half, device="cuda")
        a0, a1 = (2 * e, 2 * e + 1) if case["interleaved"] else (e, e + half)
        for t0, m, n in zip(starts, ql, kl):
            j = torch.arange(n - m, n, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               j.double()[:, None] * s["inv_freq"].double()[None])[:, None]
            for x in (q[t0:t0 + m], k[t0:t0 + m]):
                y = torch.complex(x[..., a0], x[..., a1]) * turn
                x[..., a0], x[..., a1] = y.real, y.imag
        # keys are quantised as bf16 holds them: 45 of a double's 52 bits rounded away
        i = k.view(torch.int64)
        k = (((i + (1 << 44) - 1 + ((i >> 45) & 1)) >> 45) << 45).view(torch.float64)
        return dict(q=q, k=_held(k), v=_held(v))
    if case["op"] == "read":
        back = []
        for kv in (0, 2):
            x = torch.empty((sum(ql), Hkv, D), dtype=torch.float64, device="cuda")
            for b, (t0, n) in enumerate(zip(starts, kl)):
                for g in range(Hkv):
                    x[t0:t0 + n, g] = rows(kv, b, torch.arange(n, device="cuda"), g)
            back.append(x)
        return dict(k=back[0], v=back[1])

    T = sum(ql)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    local = case.get("local", max(kl))

    def attend(x, V, t, h):
        e = torch.logsumexp(x, dim=1)
        lse[t, h] = e
        out[t, h] = torch.exp(x - e[:, None]) @ V

    for b, (t0, m, n) in enumerate(zip(starts, ql, kl)):
        for g in range(Hkv):
            if case["op"] == "sparse":
                sel = s["sel"][b, g] if case["per_head"] else s["sel"][b]
                if s["lengths"] is not None:
                    sel = sel[:int(s["lengths"][b, g] if case["per_head"] else s["lengths"][b])]
                head = min(SINK, n)
                j = torch.cat([torch.arange(head, device="cuda"), sel.long(),
                               torch.arange(max(head, n - LOCAL), n, device="cuda")])
                K, V = rows(0, b, j, g), rows(2, b, j, g)
                for h in range(g * G, (g + 1) * G):
                    attend((s["q"][b:b + 1, h].double() @ K.T) / math.sqrt(D), V, slice(b, b + 1), h)
                continue
            j = torch.arange(n, device="cuda")
            K, V = rows(0, b, j, g), rows(2, b, j, g)
            for i0 in range(0, m, 512):
                i1 = min(m, i0 + 512)
                p0, p1 = n - m + i0, n - m + i1          # positions p0 .. p1 - 1
                lo = max(0, p0 - local + 1)
                head = min(SINK, lo)
                Kb, Vb = torch.cat([K[:head], K[lo:p1]]), torch.cat([V[:head], V[lo:p1]])
                at = torch.cat([torch.arange(head, device="cuda"), torch.arange(lo, p1, device="cuda")])
                pos = torch.arange(p0, p1, device="cuda")[:, None]
                hidden = (at > pos) | ((at <= pos - local) & (at >= SINK))
                t = slice(t0 + i0, t0 + i1)
                for h in range(g * G, (g + 1) * G):
                    x = (s["q"][t, h].double() @ Kb.T) / math.sqrt(D)
                    x[hidden] = -math.inf
                    attend(x, Vb, t, h)
    return dict(out=out, lse=lse)
