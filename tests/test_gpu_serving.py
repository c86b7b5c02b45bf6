"""GPU parity of the packed-batch calls (kv_rope_append*, kv_window_attn*,
kv_prefix_attn_paged) against the fp64 oracle.

Tolerances, fixed before the first run (A = sum_j p_j |V_j|, from the oracle):
  rotated value   2^-8 |y| (one rounding to bf16: half a step) + 2^-20 (|x_a| + |x_b|)
                  (fp32 sine and cosine, products and one sum)
  copied value    equal
  logit           e = 2^-17 max_j sum_e |q_e K_e| / sqrt(d) (128 fp32 additions of
                  exact products, 128 2^-24 each relative to the sum of magnitudes)
  output          2^-8 |out| (one rounding) + 2^-8 A (each bf16 probability)
                  + 2 (e + 2^-18) A (a logit's error moves a weight and the sum)
                  + (n 2^-24 + 2^-20) A (fp32 sums over n keys)
  lse             e + n 2^-24 + 2^-20 + 2^-22 |lse|
Rows of the cache that nothing attends to are NaN, block-table entries that
must not be read lie outside the pool, and outputs are canaries beforehand.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import serving as osv

pytestmark = pytest.mark.gpu

qasc = pytest.importorskip("query_aware_sparse_compressed_gb300")
POISON = -7
CANARY = 77.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qasc._lib.load()


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def f64(x):
    return synth.to_f64(x)


def cdiv(a, b):
    return -(-a // b)


class Pages:
    """A pool with the caches of several sequences: NaN everywhere else, and a
    table whose unused entries lie outside the pool."""

    def __init__(self, lens, Hkv, P, pps, seed, extra=3):
        self.lens, self.Hkv, self.P, self.pps = list(lens), Hkv, P, pps
        used = sum(cdiv(n, P) for n in lens)
        self.num_pages = used + extra
        self.order = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((len(lens), pps), POISON, dtype=torch.int32)
        self.K = torch.full((self.num_pages, Hkv, P, 128), float("nan"), dtype=torch.bfloat16)
        self.V = self.K.clone()
        self.logical = []
        for b, n in enumerate(lens):
            k, v = rand((Hkv, n, 128), seed + 10 * b + 1), rand((Hkv, n, 128), seed + 10 * b + 2)
            self.logical.append((k, v))
            for i in range(cdiv(n, P)):
                page = self.order.pop()
                self.table[b, i] = page
                m = min(P, n - i * P)
                self.K[page, :, :m] = k[:, i * P:i * P + m]
                self.V[page, :, :m] = v[:, i * P:i * P + m]

    def hide(self, b, lo, hi):
        """Rows [lo, hi) of sequence b become NaN; pages wholly inside them
        leave the table."""
        for t in range(lo, hi):
            page = int(self.table[b, t // self.P])
            if page >= 0:
                self.K[page, :, t % self.P] = float("nan")
                self.V[page, :, t % self.P] = float("inf")
        for i in range(cdiv(lo, self.P), hi // self.P):
            self.table[b, i] = POISON

    def cuda(self):
        return self.K.cuda(), self.V.cuda(), self.table.cuda()

    def caches(self):
        return [f64(k) for k, _ in self.logical], [f64(v) for _, v in self.logical]


def batch_tensors(cu, lens):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return c, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_rows(out, lse, ref, n_keys, rows=None):
    want, want_lse, A, zabs = ref
    got, got_lse = f64(out), lse.cpu().numpy().astype(np.float64)
    if rows is not None:
        got, got_lse, want, want_lse, A, zabs = (x[rows] for x in (got, got_lse, want, want_lse, A, zabs))
    e = 2.0 ** -17 * zabs
    sums = n_keys * 2.0 ** -24 + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * (e[..., None] + 2.0 ** -18) + sums) * A + 1e-30
    bad = np.abs(got - want) / tol
    assert np.all(np.isfinite(got)), "output not finite"
    assert bad.max() <= 1.0, "output off by %.2f tolerances at %s" % (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    ltol = e + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, want_lse))
    ldiff = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want_lse))
    assert np.all(ldiff <= ltol), "lse off by %.2f tolerances" % (ldiff / ltol).max()


def window(q, pages, cu, lens, sink, local, Hkv, stream=None, extra_rows=0):
    """kv_window_attn_paged into canary outputs."""
    K, V, table = pages.cuda()
    T, Hq, _ = q.shape
    out = torch.full((T, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), CANARY, dtype=torch.float32, device="cuda")
    B = len(lens)
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(T, B, Hq, Hkv, pages.pps * pages.P))
    ws.fill_(255)
    c, ln = batch_tensors(cu, lens)
    qasc.kv_window_attn_paged(q.cuda(), K, V, table, ln, out, ws, sink=sink, local=local, cu_q=c, lse=lse)
    qasc.qasc_device_error()
    return out, lse


# --------------------------------------------------------------------- append
def cos_error(x, y, pos, inv_freq, interleaved):
    half = len(inv_freq)
    mag = np.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * mag


def freqs(rot):
    return (500000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float()


APPEND = [
    # Hq, Hkv, P, q_lens, lens, rot, interleaved, fused, positions
    (8, 2, 64, [1, 1, 1], [1, 64, 65], 128, False, True, False),
    (8, 2, 64, [70, 0, 1, 129], [70, 5, 100, 200], 64, True, True, False),
    (4, 4, 128, [33], [500], 32, False, False, True),
    (8, 1, 256, [5, 7], [5, 300], 128, True, False, True),
    (16, 8, 64, [3, 2], [3, 77], 0, False, True, False),
    (64, 8, 256, [700], [700], 128, False, True, False),
    (32, 8, 64, [1] * 5, [9, 8, 7, 6, 500], 16, False, False, False),
]


@pytest.mark.parametrize("Hq,Hkv,P,ql,lens,rot,inter,fused,override", APPEND)
@pytest.mark.parametrize("paged", [True, False])
def test_append(Hq, Hkv, P, ql, lens, rot, inter, fused, override, paged):
    B, T = len(ql), sum(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pps = cdiv(max(lens), P) + 1
    pages = Pages(lens, Hkv, P, pps, seed=7)
    for b, n in enumerate(lens):               # pages in front of the new tokens are not read
        pages.table[b, :(n - ql[b]) // P] = POISON
    if fused:
        q, k, v = rand((T, Hq + 2 * Hkv, 128), 5).cuda().split([Hq, Hkv, Hkv], dim=1)
    else:
        q, k, v = (rand((T, H, 128), s).cuda() for H, s in ((Hq, 5), (Hkv, 6), (Hkv, 8)))
    inv = freqs(rot)
    seq, pos = osv.positions(cu, lens, T)
    override_pos = None
    if override:
        override_pos = torch.tensor([(-1) ** t * (2 ** 24 - 3 - 1000 * t) for t in range(T)], dtype=torch.int32)
    rpos = override_pos.numpy() if override else pos
    c, ln = batch_tensors(None if ql == [1] * B else cu, lens)
    q_out = torch.full((T, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
    kw = dict(cu_q=c, interleaved=inter, positions=override_pos.cuda() if override else None)
    inv_dev = inv.cuda() if rot else None
    if paged:
        K, V, table = pages.cuda()
        K0, V0 = K.clone(), V.clone()
        qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, inv_dev, **kw)
    else:
        K = torch.full((B, Hkv, pps * P - 3, 128), CANARY, dtype=torch.bfloat16, device="cuda")
        V = K.clone()
        K0, V0 = K.clone(), V.clone()
        qasc.kv_rope_append(q, k, v, q_out, K, V, ln, inv_dev, **kw)
    qasc.qasc_device_error()

    def row(X, b, p):
        return X[int(pages.table[b, p // P]), :, p % P] if paged else X[b, :, p]

    for x, got in ((q, q_out), (k, None)):
        x = f64(x)
        want = osv.rotate(x, rpos, inv.numpy().astype(np.float64), inter)
        if got is None:
            got = torch.stack([row(K, seq[t], pos[t]) for t in range(T)])
        got = f64(got)
        assert np.all(np.abs(got - want) <= cos_error(x, want, rpos, inv, inter))
        assert np.array_equal(got[..., rot:], x[..., rot:])
    for t in range(T):
        assert torch.equal(row(V, seq[t], pos[t]), v[t])
        row(K0, seq[t], pos[t]).copy_(row(K, seq[t], pos[t]))
        row(V0, seq[t], pos[t]).copy_(row(V, seq[t], pos[t]))
    assert torch.equal(K.view(torch.int16), K0.view(torch.int16)), "a row of no new token was written"
    assert torch.equal(V.view(torch.int16), V0.view(torch.int16))


def test_append_many_tokens_equals_few():
    # enough tokens for the four-token tiles, against the same tokens one
    # sequence at a time
    Hq, Hkv, P = 8, 2, 64
    ql = [611, 1, 0, 300]
    lens = [611, 40, 9, 333]
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    T = cu[-1]
    pages = Pages(lens, Hkv, P, 12, seed=3)
    q, k, v = rand((T, 12, 128), 5).cuda().split([Hq, Hkv, Hkv], dim=1)
    inv = freqs(128).cuda()
    K, V, table = pages.cuda()
    q_out = torch.empty((T, Hq, 128), dtype=torch.bfloat16, device="cuda")
    c, ln = batch_tensors(cu, lens)
    qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, inv, cu_q=c)
    K2, V2, _ = pages.cuda()
    q2 = torch.empty_like(q_out)
    for b in range(4):
        s = slice(cu[b], cu[b + 1])
        c, ln = batch_tensors([0, ql[b]], [lens[b]])
        qasc.kv_rope_append_paged(q[s], k[s], v[s], q2[s], K2, V2, table[b:b + 1], ln, inv, cu_q=c)
    qasc.qasc_device_error()
    assert torch.equal(q_out, q2)
    assert torch.equal(K.view(torch.int16), K2.view(torch.int16))
    assert torch.equal(V.view(torch.int16), V2.view(torch.int16))


def test_append_in_place_and_without_queries():
    Hq, Hkv, P = 8, 2, 64
    pages = Pages([30], Hkv, P, 2, seed=4)
    q, k, v = rand((30, Hq, 128), 1).cuda(), rand((30, Hkv, 128), 2).cuda(), rand((30, Hkv, 128), 3).cuda()
    inv = freqs(128).cuda()
    c, ln = batch_tensors([0, 30], [30])
    K, V, table = pages.cuda()
    q_out = torch.empty_like(q)
    qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, inv, cu_q=c)
    K2, V2, _ = pages.cuda()
    qasc.kv_rope_append_paged(None, k, v, None, K2, V2, table, ln, inv, cu_q=c)
    assert torch.equal(K[:, :, :1].view(torch.int16), K2[:, :, :1].view(torch.int16))
    K3, V3, _ = pages.cuda()
    qasc.kv_rope_append_paged(q, k, v, q, K3, V3, table, ln, inv, cu_q=c)
    qasc.qasc_device_error()
    assert torch.equal(q, q_out)
    assert torch.equal(K2.view(torch.int16), K3.view(torch.int16))


def test_append_skips_what_lies_outside():
    # sequence 0: page outside the pool; sequence 1: positions 62 .. 65 of a
    # 64-token cache; the last two tokens belong to no sequence
    Hkv, P = 2, 64
    pages = Pages([10, 62], Hkv, P, 1, seed=5)
    pages.table[0, 0] = pages.num_pages
    k, v = rand((9, Hkv, 128), 2).cuda(), rand((9, Hkv, 128), 3).cuda()
    q = rand((9, 8, 128), 4).cuda()
    K, V, table = pages.cuda()
    K0 = K.clone()
    q_out = torch.full_like(q, CANARY)
    c, ln = batch_tensors([0, 3, 7], [10, 66])
    qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, freqs(128).cuda(), cu_q=c)
    with pytest.raises(qasc.QascError) as e:
        qasc.qasc_device_error()
    assert e.value.status == 6
    p = int(pages.table[1, 0])
    assert torch.equal(V[p, :, 62:64], v[3:5].transpose(0, 1))
    K0[p, :, 62:64] = K[p, :, 62:64]
    assert torch.equal(K.view(torch.int16), K0.view(torch.int16))
    assert bool((q_out[7:] == CANARY).all()) and not bool((q_out[:7] == CANARY).all())


@pytest.mark.parametrize("ql", [[1, 1, 1], [300, 2, 400]])
def test_append_replays_in_a_graph(ql):
    # the replay follows cu_q, the lengths and the positions on the device
    Hq, Hkv, P, B, T = 8, 2, 64, len(ql), sum(ql)
    lens = [m + 70 * (b + 1) for b, m in enumerate(ql)]
    table = torch.randperm(3 * B * 4, generator=torch.Generator().manual_seed(8)).view(B, -1).to(torch.int32).cuda()
    q, k, v = rand((T, Hq + 2 * Hkv, 128), 9).cuda().split([Hq, Hkv, Hkv], dim=1)
    inv, pos = freqs(128).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    c, ln = batch_tensors(None if T == B else cu, lens)

    def fresh():
        K = torch.zeros((table.numel(), Hkv, P, 128), dtype=torch.bfloat16, device="cuda")
        return K, K.clone(), torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device="cuda")

    def call(K, V, q_out):
        qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, inv, cu_q=c, positions=pos)

    def same(a, b):
        return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))
    a, b, g_out = fresh(), fresh(), fresh()
    call(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(*g_out)
    graph.replay()
    torch.cuda.synchronize()
    assert same(a, g_out)
    ln.copy_(torch.tensor([x - 33 for x in lens], dtype=torch.int32))
    pos.add_(1000)
    if c is not None:
        c.copy_(torch.tensor([0, 5, 290, T - 3], dtype=torch.int32))
        ln[1] = 300
    for x in g_out:
        x.zero_()
    graph.replay()
    call(*b)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    assert same(b, g_out) and not same(a, b)


def test_two_appends_on_two_streams():
    Hq, Hkv, P, T = 8, 2, 64, 600
    q, k, v = rand((T, Hq + 2 * Hkv, 128), 9).cuda().split([Hq, Hkv, Hkv], dim=1)
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None].contiguous()
    inv = freqs(128).cuda()
    c, ln = batch_tensors([0, T], [T + 9])
    pools = [[torch.zeros((10, Hkv, P, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)] +
             [torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device="cuda")] for _ in range(3)]

    def call(K, V, q_out, stream=None):
        qasc.kv_rope_append_paged(q, k, v, q_out, K, V, table, ln, inv, cu_q=c, stream=stream)
    call(*pools[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for pool, s in zip(pools, streams):
            call(*pool, stream=s)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    for pool in pools[:2]:
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(pool, pools[2]))


def test_append_and_attention_read_one_batch_alike():
    # cu_q reaches behind the T = 7 tokens: sequence 1 has the four that are there
    Hq, Hkv, P, T = 8, 2, 64, 7
    lens = [10, 20]
    pages = Pages(lens, Hkv, P, 2, seed=6)
    q, k, v = (rand((T, H, 128), s).cuda() for H, s in ((Hq, 5), (Hkv, 6), (Hkv, 8)))
    inv = freqs(128).cuda()
    got = []
    for cu in ([0, 3, 7], [0, 3, 12]):
        K, V, table = pages.cuda()
        q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
        c, ln = batch_tensors(cu, lens)
        qasc.kv_rope_append_paged(q, k, v, q_rot, K, V, table, ln, inv, cu_q=c)
        ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(T, 2, Hq, Hkv, 2 * P))
        qasc.kv_window_attn_paged(q_rot, K, V, table, ln, out, ws, local=100, cu_q=c)
        qasc.qasc_device_error()
        got.append([x.view(torch.int16) for x in (K, V, q_rot, out)])
    assert torch.equal(V[int(pages.table[1, 0]), :, 16:20], v[3:].transpose(0, 1))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("B,bad", [(3, 2), (600, 599), (600, 0)])
@pytest.mark.parametrize("length", [-1, 129])
def test_append_reports_lengths_of_sequences_without_tokens(B, bad, length):
    # as the attention calls do; the others are written all the same
    Hkv, P = 2, 64
    K = torch.zeros((2, Hkv, P, 128), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    k, v = rand((1, Hkv, 128), 2).cuda(), rand((1, Hkv, 128), 3).cuda()
    table = torch.tensor([[0, 1]] * B, dtype=torch.int32, device="cuda")
    c, ln = batch_tensors([0, 0, 1] + [1] * (B - 2), [5] * B)
    qasc.kv_rope_append_paged(None, k, v, None, K, V, table, ln, None, cu_q=c)
    qasc.qasc_device_error()
    ln[bad] = length
    V.zero_()
    qasc.kv_rope_append_paged(None, k, v, None, K, V, table, ln, None, cu_q=c)
    with pytest.raises(qasc.QascError) as e:
        qasc.qasc_device_error()
    assert e.value.status == 6
    assert torch.equal(V[0, :, 4], v[0]) and not bool(V[0, :, 5:].any())


# --------------------------------------------------------------------- window
WINDOW = [
    # Hq, Hkv, P, q_lens, lens, sink, local
    (8, 2, 64, [1], [1], 4, 256),
    (8, 2, 64, [1, 1, 1, 1], [1, 64, 65, 700], 4, 256),
    (4, 4, 64, [1, 1], [300, 129], 0, 1),
    (8, 1, 256, [1, 1, 1], [1000, 4, 513], 7, 130),
    (16, 8, 128, [1], [2500], 200, 300),
    (8, 2, 64, [200], [200], 4, 64),
    (8, 2, 64, [131, 1, 0, 40], [131, 90, 77, 400], 4, 100),
    (8, 8, 64, [129], [300], 3, 5000),
    (8, 1, 128, [33, 2], [33, 257], 130, 17),
    (8, 4, 64, [64, 65], [64, 321], 0, 128),
    (64, 8, 64, [9], [140], 1, 139),
    (8, 2, 64, [5, 3], [2, 3], 4, 9),          # three tokens stand in front of their cache
    (8, 2, 64, [300], [300], 0, 300),
]


@pytest.mark.parametrize("Hq,Hkv,P,ql,lens,sink,local", WINDOW)
@pytest.mark.parametrize("paged", [True, False])
def test_window(Hq, Hkv, P, ql, lens, sink, local, paged):
    T, B = sum(ql), len(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages(lens, Hkv, P, cdiv(max(lens), P) + 1, seed=11)
    q = rand((T + 2, Hq, 128), 12)             # two tokens of no sequence
    single = ql == [1] * B
    if single:
        q = q[:T]
    ref = osv.window_attention(f64(q[:T]), *pages.caches(), cu, lens, sink, local)
    for b, n in enumerate(lens):               # what no query attends to
        first = max(0, n - ql[b])
        if ql[b] == 0:
            pages.hide(b, 0, n)
        elif first - local + 1 > sink:
            pages.hide(b, sink, first - local + 1)
    cu_arg = None if single else cu
    if paged:
        out, lse = window(q, pages, cu_arg, lens, sink, local, Hkv)
    else:
        n_cap = max(lens) + 5
        K = torch.full((B, Hkv, n_cap, 128), float("nan"), dtype=torch.bfloat16)
        V = K.clone()
        for b, n in enumerate(lens):
            for t in range(n):
                page = int(pages.table[b, t // P])
                if page >= 0:
                    K[b, :, t], V[b, :, t] = pages.K[page, :, t % P], pages.V[page, :, t % P]
        out = torch.full((q.shape[0], Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0], Hq), CANARY, dtype=torch.float32, device="cuda")
        ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(q.shape[0], B, Hq, Hkv, n_cap))
        c, ln = batch_tensors(cu_arg, lens)
        qasc.kv_window_attn(q.cuda(), K.cuda(), V.cuda(), ln, out, ws, sink=sink, local=local, cu_q=c, lse=lse)
        qasc.qasc_device_error()
    check_rows(out[:T], lse[:T], ref, max(lens))
    assert bool((out[T:] == CANARY).all()) and bool((lse[T:] == CANARY).all())


@pytest.mark.parametrize("scale", [0.0, 8.0])
def test_window_flat_and_peaked_logits(scale):
    Hq, Hkv, P, n, m = 8, 2, 64, 700, 70
    pages = Pages([n], Hkv, P, 11, seed=13)
    q = rand((m, Hq, 128), 14, scale)
    ref = osv.window_attention(f64(q), *pages.caches(), [0, m], [n], 4, 400)
    out, lse = window(q, pages, [0, m], [n], 4, 400, Hkv)
    check_rows(out, lse, ref, n)


LARGE = [2048, 1, 0, 33, 500, 1, 64]       # enough rows that items are taken whole


@pytest.mark.parametrize("Hq,Hkv,sink,local", [(64, 8, 4, 300), (64, 8, 0, 1 << 30), (64, 32, 150, 70)])
def test_window_of_many_rows(Hq, Hkv, sink, local):
    ql = LARGE
    lens = [2048, 700, 90, 40, 777, 5, 900]
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    T = cu[-1]
    pages = Pages(lens, Hkv, 64, cdiv(max(lens), 64) + 1, seed=61)
    q = rand((T, Hq, 128), 62)
    rng = np.random.default_rng(63)
    some = sorted({0, 1, 2, 62, 63, 64, 127, 128, 2047, *cu[1:3], cu[3], *range(cu[3], cu[4], 8), cu[4], T - 65, T - 64, T - 1,
                   *rng.integers(0, T, 24).tolist()})
    ref = osv.window_attention(f64(q), *pages.caches(), cu, lens, sink, local, tokens=some)
    pages.hide(2, 0, 90)
    out, lse = window(q, pages, cu, lens, sink, local, Hkv)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, max(lens), rows=some)


def test_prefix_of_many_rows():
    # long own parts: the prefix is walked by each sequence's items
    Hq, Hkv, P, n0, ql = 64, 8, 64, 333, LARGE
    lens = [2048, 700, 90, 40, 777, 0, 60]
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    T = cu[-1]
    both = Pages([n0] + lens, Hkv, P, 34, seed=64)
    q = rand((T, Hq, 128), 65)
    some = sorted({0, 63, 64, 1000, 2047, cu[1], cu[3], cu[4] - 1, cu[5], T - 64, T - 60, T - 1})
    Kc, Vc = both.caches()
    ref = osv.prefix_attention(f64(q), Kc[0], Vc[0], Kc[1:], Vc[1:], cu, lens, tokens=some)
    K, V, table = both.cuda()
    out = torch.full((T, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(T, len(ql), Hq, Hkv, both.pps * P))
    c, ln = batch_tensors(cu, lens)
    qasc.kv_prefix_attn_paged(q.cuda(), K, V, table[0, :cdiv(n0, P)].contiguous(), table[1:].contiguous(), ln, out, ws,
                              n_prefix=n0, cu_q=c, lse=lse)
    qasc.qasc_device_error()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, n0 + max(lens), rows=some)


@pytest.mark.parametrize("B,Hq,Hkv,sink,local", [(400, 8, 2, 4, 2000), (2048, 4, 2, 4, 100), (700, 8, 8, 0, 64)])
def test_window_of_many_sequences(B, Hq, Hkv, sink, local):
    # plans too large for a block's shared memory
    lens = [1 + (37 * b) % 300 for b in range(B)]
    lens[3] = 1500
    pages = Pages(lens, Hkv, 64, cdiv(1500, 64), seed=71)
    q = rand((B, Hq, 128), 72)
    some = sorted({0, 1, 2, 3, 4, B - 1, *range(5, B, 41)})
    ref = osv.window_attention(f64(q), *pages.caches(), list(range(B + 1)), lens, sink, local, tokens=some)
    out, lse = window(q, pages, None, lens, sink, local, Hkv)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, 1500, rows=some)


def test_window_of_many_ragged_sequences():
    B, Hq, Hkv = 500, 8, 2
    ql = [(7 * b) % 5 for b in range(B)]
    lens = [max(1, m) + (53 * b) % 400 for b, m in enumerate(ql)]
    cu = (3 + np.concatenate([[0], np.cumsum(ql)])).tolist()      # three tokens in front of the first sequence
    T = cu[-1] + 2
    pages = Pages(lens, Hkv, 64, 8, seed=73)
    q = rand((T, Hq, 128), 74)
    some = sorted({3, 4, 5, T - 3, *range(6, T - 3, 37)})
    ref = osv.window_attention(f64(q), *pages.caches(), cu, lens, 4, 5000, tokens=some)
    out, lse = window(q, pages, cu, lens, 4, 5000, Hkv)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, 404, rows=some)
    outside = [0, 1, 2, T - 2, T - 1]
    assert bool((out[outside] == CANARY).all()) and bool((lse[outside] == CANARY).all())


def test_prefix_of_many_sequences():
    B, Hq, Hkv, P, n0 = 300, 8, 2, 64, 700
    lens = [(11 * b) % 90 for b in range(B)]
    both = Pages([n0] + lens, Hkv, P, 11, seed=75)
    q = rand((B, Hq, 128), 76)
    some = sorted({0, 1, 2, B - 1, *range(3, B, 23)})
    Kc, Vc = both.caches()
    ref = osv.prefix_attention(f64(q), Kc[0], Vc[0], Kc[1:], Vc[1:], list(range(B + 1)), lens, tokens=some)
    K, V, table = both.cuda()
    out = torch.full((B, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), float("nan"), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(B, B, Hq, Hkv, both.pps * P))
    ws.fill_(255)
    qasc.kv_prefix_attn_paged(q.cuda(), K, V, table[0, :cdiv(n0, P)].contiguous(), table[1:].contiguous(),
                              batch_tensors(None, lens)[1], out, ws, n_prefix=n0, lse=lse)
    qasc.qasc_device_error()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, n0 + 90, rows=some)


@pytest.mark.parametrize("T", [5, 3000])
def test_window_without_any_sequence(T):
    pages = Pages([10, 20], 8, 64, 1, seed=77)
    out, lse = window(rand((T, 64, 128), 78), pages, [0, 0, 0], [10, 20], 4, 100, 8)
    assert bool((out == CANARY).all()) and bool((lse == CANARY).all())


@pytest.mark.parametrize("n,m", [(1900, 1), (900, 200)])
def test_window_not_a_number_stays_visible(n, m):
    # a NaN key makes the queries that attend to it NaN, and no others
    Hq, Hkv, P, local = 8, 2, 64, 300
    pages = Pages([n], Hkv, P, cdiv(n, P), seed=79)
    j = n - 50
    pages.K[int(pages.table[0, j // P]), 1, j % P, 5] = float("nan")
    q = rand((m, Hq, 128), 80)
    out, lse = window(q, pages, [0, m], [n], 4, local, Hkv)
    pos = torch.arange(n - m, n)
    hit = ((pos >= j) & (pos - local < j)).cuda()
    bad = torch.isnan(out).any(-1)
    assert bool((torch.isnan(out).all(-1) == bad).all()) and bool((torch.isnan(lse) == bad).all())
    assert bool((bad[:, 4:] == hit[:, None]).all()) and not bool(bad[:, :4].any())


@pytest.mark.parametrize("n,m", [(1900, 1), (900, 200), (9000, 1)])
def test_window_not_a_number_in_a_value(n, m):
    # it reaches its column of the queries that attend to it; no other column, KV head or lse
    Hq, Hkv, P, local = 8, 2, 64, 300 if n < 9000 else 9000
    pages = Pages([n], Hkv, P, cdiv(n, P), seed=95)
    j = n - 50
    pages.V[int(pages.table[0, j // P]), 1, j % P, 5] = float("nan")
    q = rand((m, Hq, 128), 96)
    out, lse = window(q, pages, [0, m], [n], 4, local, Hkv)
    pos = torch.arange(n - m, n)
    hit = ((pos >= j) & (pos - local < j)).cuda()
    bad = torch.isnan(out)
    assert bool(bad[hit][:, 4:, 5].all())
    bad[:, 4:, 5] = False
    assert not bool(bad.any()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("n,m", [(1, 1), (1900, 1), (900, 200), (9000, 1)])
def test_window_logits_of_minus_infinity(n, m):
    # a row that has no others counts as one that attends to nothing; one that has any is untouched
    Hq, Hkv, P, local = 8, 2, 64, 300 if n < 9000 else 9000
    pages = Pages([n], Hkv, P, cdiv(n, P), seed=97)
    for i in range(cdiv(n, P)):
        page = int(pages.table[0, i])
        pages.K[page, 1, :, 5] = float("-inf")                                 # every key of KV head 1
        pages.K[page, 0, ::3, 5] = float("-inf")                               # every third of KV head 0, by page
        for t in range(i * P, min(n, i * P + P)):
            pages.logical[0][0][:, t] = pages.K[page, :, t % P]
    q = rand((m, Hq, 128), 98)
    q[..., 5] = 1.0
    out, lse = window(q, pages, [0, m], [n], 4, local, Hkv)
    assert bool((out[:, 4:] == 0).all()) and bool(torch.isneginf(lse[:, 4:]).all())
    if n == 1:
        return
    # KV head 0: the keys at -inf leave the sums
    k, v = pages.caches()
    finite = np.isfinite(k[0][0, :, 5])
    for t in sorted({0, m // 2, m - 1}):
        p = n - m + t
        seen = [j for j in range(p + 1) if finite[j] and (j < 4 or j > p - local)]
        one = osv.window_attention(f64(q[t:t + 1, :4]), [k[0][:1, seen]], [v[0][:1, seen]], [0, 1], [len(seen)], 0, n)
        check_rows(out[t:t + 1, :4], lse[t:t + 1, :4], one, n)


# Caches long enough that an item's keys are shared between blocks (the shares'
# borders fall inside items, key tiles of either parity and of the sink).
LONG = [
    # Hq, Hkv, q_lens, lens, sink, local
    (8, 2, [1], [9000], 4, 1 << 30),
    (8, 2, [1, 1, 1], [9000, 10, 3001], 300, 6000),
    (4, 1, [70, 1, 3], [9000, 6000, 10], 4, 1 << 30),
    (16, 2, [100, 40, 0, 1], [8001, 3000, 7, 1], 0, 5000),
    (8, 4, [130, 64, 65], [4000, 6100, 65], 130, 1 << 30),
]


@pytest.mark.parametrize("Hq,Hkv,ql,lens,sink,local", LONG)
def test_window_shared_between_blocks(Hq, Hkv, ql, lens, sink, local):
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages(lens, Hkv, 128, cdiv(max(lens), 128), seed=81)
    q = rand((cu[-1], Hq, 128), 82)
    some = sorted({0, cu[-1] - 1, *(c for c in cu if c < cu[-1]), *(c - 1 for c in cu if c), *range(0, cu[-1], 17)})
    ref = osv.window_attention(f64(q), *pages.caches(), cu, lens, sink, local, tokens=some)
    out, lse = window(q, pages, None if ql == [1] * len(ql) else cu, lens, sink, local, Hkv)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, max(lens), rows=some)


def contiguous(pages, n_cap):
    """The same caches as [B, Hkv, n_cap, 128], NaN behind each sequence."""
    K = torch.full((len(pages.lens), pages.Hkv, n_cap, 128), float("nan"), dtype=torch.bfloat16)
    V = K.clone()
    for b, (k, v) in enumerate(pages.logical):
        K[b, :, :k.shape[1]], V[b, :, :k.shape[1]] = k, v
    return K.cuda(), V.cuda()


# A contiguous cache whose sequences and heads begin anywhere: shared between
# blocks, and with plans too large for a block's shared memory.
@pytest.mark.parametrize("Hq,Hkv,ql,lens,sink,local", LONG + [
    (8, 2, [1] * 400, [1 + (37 * b) % 300 for b in range(400)], 4, 2000),
    (8, 2, [(7 * b) % 5 for b in range(500)], [5 + (53 * b) % 400 for b in range(500)], 4, 5000),
])
def test_window_contiguous_long_and_many(Hq, Hkv, ql, lens, sink, local):
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    T, B, n_cap = cu[-1], len(ql), max(lens) + 5
    pages = Pages(lens, Hkv, 64, cdiv(max(lens), 64), seed=89)
    K, V = contiguous(pages, n_cap)
    q = rand((T, Hq, 128), 90)
    some = sorted({0, T - 1, *range(0, T, 17 if T < 400 else 41)})
    ref = osv.window_attention(f64(q), *pages.caches(), cu, lens, sink, local, tokens=some)
    out = torch.full((T, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(T, B, Hq, Hkv, n_cap))
    ws.fill_(255)
    c, ln = batch_tensors(None if ql == [1] * B else cu, lens)
    qasc.kv_window_attn(q.cuda(), K, V, ln, out, ws, sink=sink, local=local, cu_q=c, lse=lse)
    qasc.qasc_device_error()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, max(lens), rows=some)


@pytest.mark.parametrize("Hq,Hkv,ql,local", [(16, 2, [300] * 6, 90), (8, 8, [1] * 60, 700), (32, 8, [64] * 8, 500)])
def test_window_items_of_half_the_rows(Hq, Hkv, ql, local):
    # several items of 128 rows or less to a block, whose two groups join their sums
    lens = [m + (211 * b) % 1500 for b, m in enumerate(ql)]
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages(lens, Hkv, 64, cdiv(max(lens), 64), seed=83)
    q = rand((cu[-1], Hq, 128), 84)
    some = sorted({0, cu[-1] - 1, *cu[:-1], *range(0, cu[-1], 29)})
    ref = osv.window_attention(f64(q), *pages.caches(), cu, lens, 4, local, tokens=some)
    out, lse = window(q, pages, None if ql == [1] * len(ql) else cu, lens, 4, local, Hkv)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, max(lens), rows=some)


def test_window_long_positions():
    # 2^23 tokens through a table that repeats a few pages: positions, sink and
    # window far apart
    Hq, Hkv, P = 8, 2, 65536
    n = (1 << 23) - 77
    pool_k, pool_v = rand((2, Hkv, P, 128), 81), rand((2, Hkv, P, 128), 82)
    table = (torch.arange(128, dtype=torch.int32) % 2)[None].cuda()
    q = rand((3, Hq, 128), 83)
    j = [*range(0, 150), *range(n - 3 - 399, n)]
    Kj, Vj = (np.stack([f64(x[(t // P) % 2, :, t % P]) for t in j], axis=1) for x in (pool_k, pool_v))
    out = torch.empty((3, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, Hq), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(3, 1, Hq, Hkv, 128 * P))
    c, ln = batch_tensors([0, 3], [n])
    qasc.kv_window_attn_paged(q.cuda(), pool_k.cuda(), pool_v.cuda(), table, ln, out, ws, sink=150, local=400, cu_q=c,
                              lse=lse)
    qasc.qasc_device_error()
    # the same rows as a short cache: the sink, then the window
    ref = osv.window_attention(f64(q), [Kj], [Vj], [0, 3], [len(j)], 150, 400)
    check_rows(out, lse, ref, 552)


def test_window_growing_maximum():
    # every later key scores higher: the running maximum moves in every tile
    Hq, Hkv, P, n = 8, 2, 64, 1500
    pages = Pages([n], Hkv, P, 24, seed=15)
    q = rand((40, Hq, 128), 16)
    for g in range(Hkv):
        base = q[0, g * 4].float()
        ramp = torch.linspace(-1.5, 1.5, n)[:, None] * base
        pages.logical[0][0][g] = ramp.to(torch.bfloat16)
    for i in range(cdiv(n, P)):
        m = min(P, n - i * P)
        pages.K[int(pages.table[0, i]), :, :m] = pages.logical[0][0][:, i * P:i * P + m]
    ref = osv.window_attention(f64(q), *pages.caches(), [0, 40], [n], 4, 1400)
    out, lse = window(q, pages, [0, 40], [n], 4, 1400, Hkv)
    check_rows(out, lse, ref, n)


def test_window_step_equals_sink_and_local_of_the_sparse_step():
    # T = sink + local without selected tokens: the fp32 decode call on the
    # same pool, so the two differ by the bf16 roundings alone
    Hq, Hkv, P, B, n, sink, local = 32, 8, 256, 3, 3000, 4, 1000
    pages = Pages([n] * B, Hkv, P, cdiv(n, P), seed=17)
    q = rand((B, Hq, 128), 18)
    out, lse = window(q, pages, None, [n] * B, sink, local, Hkv)
    K, V, table = pages.cuda()
    ref = torch.empty((B, Hq, 128), dtype=torch.float32, device="cuda")
    ref_lse = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.ts_attn_workspace_bytes(B, Hq, Hkv, n, pages.pps * P, 0, sink, local))
    qasc.ts_sparse_attn_paged(q.cuda(), K, V, table, torch.empty((B, 0), dtype=torch.int32, device="cuda"), ref, ws,
                              n=n, sink=sink, local=local, lse=ref_lse)
    qasc.qasc_device_error()
    # |out - ref| <= 2^-8 |ref| + 2^-8 A with A <= max |V| <= 6, and both fp32 paths' noise
    assert float((out.float() - ref).abs().max()) <= 2.0 ** -8 * (float(ref.abs().max()) + 6) + 1e-3
    assert float((lse - ref_lse).abs().max()) <= 1e-4


# Lengths outside [0, n_cap] are clamped and recorded, on every path: single
# tokens whole and shared between blocks, several tokens, behind a prefix.
@pytest.mark.parametrize("ql,n_cap,n0", [([1, 1, 1], 256, 0), ([1, 1, 1], 8192, 0), ([9, 2, 40], 256, 0),
                                         ([1, 1, 1], 256, 70), ([1, 1, 1], 256, 6000)])
def test_lengths_outside_are_clamped_and_reported(ql, n_cap, n0):
    Hq, Hkv, P, B = 8, 2, 64, 3
    pages = Pages([n_cap] * B + [n0], Hkv, P, cdiv(max(n_cap, n0), P), seed=91)
    K, V, table = pages.cuda()
    own, pt = table[:B, :n_cap // P].contiguous(), table[B, :cdiv(n0, P)].contiguous()
    q = rand((sum(ql), Hq, 128), 92).cuda()
    cu = None if ql == [1] * B else np.concatenate([[0], np.cumsum(ql)]).tolist()
    size = qasc.kv_prefix_attn_workspace_bytes if n0 else qasc.kv_window_attn_workspace_bytes
    ws = qasc.alloc_workspace(size(sum(ql), B, Hq, Hkv, n_cap))

    def call(lens):
        out = torch.zeros((sum(ql), Hq, 128), dtype=torch.bfloat16, device="cuda")
        c, ln = batch_tensors(cu, lens)
        if n0:
            qasc.kv_prefix_attn_paged(q, K, V, pt, own, ln, out, ws, n_prefix=n0, cu_q=c)
        else:
            qasc.kv_window_attn_paged(q, K, V, own, ln, out, ws, local=1 << 30, cu_q=c)
        return out
    want = call([n_cap, 100, 0])
    qasc.qasc_device_error()
    got = call([n_cap + 70, 100, -3])
    with pytest.raises(qasc.QascError) as e:
        qasc.qasc_device_error()
    assert e.value.status == 6
    assert torch.equal(want, got)
    call([n_cap, 100, 0])
    qasc.qasc_device_error()


def test_window_bad_page_is_reported():
    Hq, Hkv, P = 8, 2, 64
    pages = Pages([200], Hkv, P, 4, seed=19)
    pages.table[0, 1] = pages.num_pages + 5
    K, V, table = pages.cuda()
    K.nan_to_num_(0.0)
    V.nan_to_num_(0.0)
    out = torch.empty((1, Hq, 128), dtype=torch.bfloat16, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(1, 1, Hq, Hkv, 256))
    qasc.kv_window_attn_paged(rand((1, Hq, 128), 1).cuda(), K, V, table, batch_tensors(None, [200])[1], out, ws,
                              local=256)
    with pytest.raises(qasc.QascError) as e:
        qasc.qasc_device_error()
    assert e.value.status == 6
    # a length beyond the cache is cut to it
    pages = Pages([256], Hkv, P, 4, seed=19)
    K, V, table = pages.cuda()
    q = rand((1, Hq, 128), 1).cuda()
    outs = [torch.empty((1, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    qasc.kv_window_attn_paged(q, K, V, table, batch_tensors(None, [256])[1], outs[0], ws, local=256)
    qasc.qasc_device_error()
    qasc.kv_window_attn_paged(q, K, V, table, batch_tensors(None, [300])[1], outs[1], ws, local=256)
    with pytest.raises(qasc.QascError):
        qasc.qasc_device_error()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("T,B,n", [(1, 1, 5000), (700, 1, 1400), (40, 40, 900)])
def test_window_is_deterministic_and_replays_in_a_graph(T, B, n):
    Hq, Hkv, P = 16, 4, 128
    lens = [n - 17 * b for b in range(B)]
    pages = Pages(lens, Hkv, P, cdiv(n, P), seed=21)
    K, V, table = pages.cuda()
    q = rand((T, Hq, 128), 22).cuda()
    cu = None if T == B else [0, T]
    c, ln = batch_tensors(cu, lens)
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(T, B, Hq, Hkv, pages.pps * P))

    def call(out, lse):
        qasc.kv_window_attn_paged(q, K, V, table, ln, out, ws, sink=4, local=700, cu_q=c, lse=lse)

    def fresh():
        return (torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((T, Hq), dtype=torch.float32, device="cuda"))
    a, b = fresh(), fresh()
    call(*a)
    call(*b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g_out = fresh()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(*g_out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], g_out[0]) and torch.equal(a[1], g_out[1])
    # the replay follows the lengths on the device
    ln.copy_(torch.tensor([max(1, x - 200) for x in lens], dtype=torch.int32))
    graph.replay()
    call(*a)
    torch.cuda.synchronize()
    assert torch.equal(a[0], g_out[0]) and not torch.equal(a[0], b[0])
    qasc.qasc_device_error()


def test_two_windows_on_two_streams():
    Hq, Hkv, P, n = 16, 4, 64, 2000
    pages = Pages([n, n - 3], Hkv, P, cdiv(n, P), seed=23)
    K, V, table = pages.cuda()
    q = rand((2, Hq, 128), 24).cuda()
    ln = batch_tensors(None, [n, n - 3])[1]
    size = qasc.kv_window_attn_workspace_bytes(2, 2, Hq, Hkv, pages.pps * P)
    outs = [torch.zeros((2, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    wss = [qasc.alloc_workspace(size) for _ in range(3)]
    qasc.kv_window_attn_paged(q, K, V, table, ln, outs[2], wss[2], local=n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            qasc.kv_window_attn_paged(q, K, V, table, ln, outs[i], wss[i], local=n, stream=s)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_a_workspace_of_the_prompt_serves_every_smaller_call():
    Hq, Hkv, P, n = 64, 8, 64, 5000             # more rows than a shared call can have
    pages = Pages([n], Hkv, P, cdiv(n, P), seed=25)
    K, V, table = pages.cuda()
    q = rand((n, Hq, 128), 26).cuda()
    size = lambda m: qasc.kv_window_attn_workspace_bytes(m, 1, Hq, Hkv, pages.pps * P)
    shared = qasc.alloc_workspace(size(n))

    def call(m, ws):
        out = torch.zeros((m, Hq, 128), dtype=torch.bfloat16, device="cuda")
        c, ln = batch_tensors([0, m], [n])
        qasc.kv_window_attn_paged(q[:m], K, V, table, ln, out, ws, local=n, cu_q=c)
        return out
    for m in (n, 1, 300, 4064, 7):
        own = call(m, qasc.alloc_workspace(size(m)))
        assert torch.equal(call(m, shared), own)
    # no rows are shared: the least workspace is enough; one token's are, and it is not
    least = qasc.alloc_workspace(size(0))
    assert torch.equal(call(n, least), call(n, shared))
    with pytest.raises(qasc.QascError) as e:
        call(1, least)
    assert e.value.status == 3
    qasc.qasc_device_error()


# --------------------------------------------------------------------- prefix
PREFIX = [
    # Hq, Hkv, P, n_prefix, q_lens, lens
    (8, 2, 64, 1, [1], [1]),
    (8, 2, 64, 64, [1, 1], [1, 65]),
    (8, 2, 64, 1000, [1, 1, 1, 1], [1, 37, 0, 130]),      # sequence 2 has the prefix alone
    (4, 4, 128, 300, [1] * 9, list(range(9))),
    (8, 1, 64, 129, [1] * 33, [1 + 7 * i for i in range(33)]),
    (64, 8, 256, 700, [3, 1, 0, 2], [3, 9, 4, 300]),
    (8, 2, 64, 500, [70, 5], [70, 2]),                     # three tokens stand in front of their own cache
    (16, 8, 64, 0, [2, 1], [90, 4]),
    (8, 2, 64, 90, [150], [200]),
]


@pytest.mark.parametrize("Hq,Hkv,P,n0,ql,lens", PREFIX)
def test_prefix(Hq, Hkv, P, n0, ql, lens):
    T, B = sum(ql), len(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    both = Pages([n0] + lens, Hkv, P, cdiv(max([n0] + lens), P) + 1, seed=31)
    q = rand((T, Hq, 128), 32)
    Kc, Vc = both.caches()
    ref = osv.prefix_attention(f64(q), Kc[0], Vc[0], Kc[1:], Vc[1:], cu, lens)
    K, V, table = both.cuda()
    ptable = table[0, :cdiv(n0, P)].contiguous()
    stable = table[1:].contiguous()
    out = torch.full((T, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), CANARY, dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(T, B, Hq, Hkv, both.pps * P))
    ws.fill_(255)
    c, ln = batch_tensors(None if ql == [1] * B else cu, lens)
    qasc.kv_prefix_attn_paged(q.cuda(), K, V, ptable, stable, ln, out, ws, n_prefix=n0, cu_q=c, lse=lse)
    qasc.qasc_device_error()
    check_rows(out, lse, ref, n0 + max(lens))


# long prefixes, whose items blocks share, and short ones, which every item walks
@pytest.mark.parametrize("Hq,Hkv,P,n0,ql,lens", [
    (8, 2, 64, 6000, [1] * 5, [1, 300, 0, 130, 64]),
    (16, 2, 64, 5000, [100, 40, 0, 1], [100, 333, 0, 1]),
    (64, 8, 64, 4100, [9, 1, 3], [9, 700, 3]),
    (8, 1, 128, 4000, [40, 60, 0, 5], [40, 1200, 3, 5]),
    (16, 2, 64, 130, [100, 40, 0, 1], [100, 333, 0, 1]),
    (8, 2, 64, 200, [300] * 4, [300, 411, 350, 299]),      # a token stands in front of its own cache
    (32, 8, 64, 65, [1] * 40, [(17 * i) % 200 for i in range(40)]),
])
def test_prefix_long_and_short(Hq, Hkv, P, n0, ql, lens):
    test_prefix(Hq, Hkv, P, n0, ql, lens)


# several items of the prefix to a KV head (their shares go around), KV heads in twos and an odd one
@pytest.mark.parametrize("B,Hq,Hkv,n0", [(70, 32, 4, 9000), (90, 24, 3, 5000), (64, 24, 3, 100)])
def test_prefix_of_several_items(B, Hq, Hkv, n0):
    P = 64
    lens = [(29 * b) % 260 for b in range(B)]
    both = Pages([n0] + lens, Hkv, P, max(5, cdiv(n0, P)), seed=85)
    q = rand((B, Hq, 128), 86)
    some = sorted({0, 1, 9, 10, B - 1, *range(2, B, 7)})
    Kc, Vc = both.caches()
    ref = osv.prefix_attention(f64(q), Kc[0], Vc[0], Kc[1:], Vc[1:], list(range(B + 1)), lens, tokens=some)
    K, V, table = both.cuda()
    own = table[1:, :5].contiguous()                     # 5 pages hold 260 tokens
    out = torch.full((B, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq), float("nan"), dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(B, B, Hq, Hkv, 5 * P))
    ws.fill_(255)
    qasc.kv_prefix_attn_paged(q.cuda(), K, V, table[0, :cdiv(n0, P)].contiguous(), own, batch_tensors(None, lens)[1], out,
                              ws, n_prefix=n0, lse=lse)
    qasc.qasc_device_error()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    check_rows(out, lse, ref, n0 + 260, rows=some)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (24, 3), (16, 16)])
def test_window_of_short_and_empty_sequences(Hq, Hkv):
    # many short items, some without any token (the query stands in front of an empty cache)
    B = 240 // Hkv + 60
    lens = [(13 * b) % 170 for b in range(B)]
    pages = Pages(lens, Hkv, 64, 3, seed=87)
    q = rand((B, Hq, 128), 88)
    ref = osv.window_attention(f64(q), *pages.caches(), list(range(B + 1)), lens, 4, 100)
    out, lse = window(q, pages, None, lens, 4, 100, Hkv)
    check_rows(out, lse, ref, 170)


@pytest.mark.parametrize("n0,ql", [(100, [1] * 30), (6000, [1] * 30), (6000, [40, 3, 90])])
def test_prefix_replays_in_a_graph(n0, ql):
    Hq, Hkv, P, B, T = 16, 4, 64, len(ql), sum(ql)
    lens = [m + (37 * b) % 200 for b, m in enumerate(ql)]
    both = Pages([n0] + lens, Hkv, P, max(5, cdiv(n0, P)), seed=93)
    K, V, table = both.cuda()
    own, pt = table[1:, :5].contiguous(), table[0, :cdiv(n0, P)].contiguous()
    q = rand((T, Hq, 128), 94).cuda()
    c, ln = batch_tensors(None if T == B else np.concatenate([[0], np.cumsum(ql)]).tolist(), lens)
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(T, B, Hq, Hkv, 5 * P))

    def call(out, lse):
        qasc.kv_prefix_attn_paged(q, K, V, pt, own, ln, out, ws, n_prefix=n0, cu_q=c, lse=lse)

    def fresh():
        return (torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((T, Hq), dtype=torch.float32, device="cuda"))
    a, b, g_out = fresh(), fresh(), fresh()
    call(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(*g_out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], g_out[0]) and torch.equal(a[1], g_out[1])
    ln.copy_(torch.tensor([max(0, x - 60) for x in lens], dtype=torch.int32))   # the replay follows the lengths
    graph.replay()
    call(*b)
    torch.cuda.synchronize()
    assert torch.equal(b[0], g_out[0]) and torch.equal(b[1], g_out[1]) and not torch.equal(a[0], b[0])
    qasc.qasc_device_error()


def test_prefix_leaves_other_rows_alone():
    Hq, Hkv, P = 8, 2, 64
    both = Pages([100, 20, 30], Hkv, P, 2, seed=33)
    K, V, table = both.cuda()
    q = rand((9, Hq, 128), 34).cuda()
    out = torch.full((9, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, Hq), CANARY, dtype=torch.float32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(9, 2, Hq, Hkv, 128))
    c, ln = batch_tensors([2, 3, 6], [20, 30])
    qasc.kv_prefix_attn_paged(q, K, V, table[0].contiguous(), table[1:].contiguous(), ln, out, ws, n_prefix=100,
                              cu_q=c, lse=lse)
    qasc.qasc_device_error()
    outside = [0, 1, 6, 7, 8]
    assert bool((out[outside] == CANARY).all()) and bool((lse[outside] == CANARY).all())
    assert not bool((out[2:6] == CANARY).any())


# ------------------------------------------------------- the calls as they are used
def test_prefill_in_chunks_then_decode():
    """A prompt appended and attended in chunks equals the prompt at once, and
    the token-selection decode step reads the cache that they filled."""
    Hq, Hkv, P, n, sink, local = 8, 2, 64, 600, 4, 256
    pps = cdiv(n + 1, P)
    table = torch.randperm(pps + 2, generator=torch.Generator().manual_seed(1))[:pps].to(torch.int32)[None].cuda()
    inv = freqs(128).cuda()
    qkv = rand((n + 1, Hq + 2 * Hkv, 128), 41).cuda()
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(n, 1, Hq, Hkv, pps * P))

    def prefill(chunks):
        K = torch.zeros((pps + 2, Hkv, P, 128), dtype=torch.bfloat16, device="cuda")
        V = torch.zeros_like(K)
        outs, at = [], 0
        for m in chunks:
            q, k, v = qkv[at:at + m].split([Hq, Hkv, Hkv], dim=1)
            q_rot = torch.empty((m, Hq, 128), dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q_rot)
            c, ln = batch_tensors([0, m], [at + m])
            qasc.kv_rope_append_paged(q, k, v, q_rot, K, V, table, ln, inv, cu_q=c)
            qasc.kv_window_attn_paged(q_rot, K, V, table, ln, out, ws, sink=sink, local=n, cu_q=c)
            outs.append(out)
            at += m
        return K, V, torch.cat(outs)

    K, V, whole = prefill([n])
    K2, V2, parts = prefill([100, 1, 299, 200])
    assert torch.equal(K.view(torch.int16), K2.view(torch.int16))
    assert torch.equal(V.view(torch.int16), V2.view(torch.int16))
    # two orders of the same fp32 sums and two roundings of the probabilities: A <= max |V| <= 6
    assert float((whole.float() - parts.float()).abs().max()) <= 2 * 2.0 ** -8 * (float(whole.float().abs().max()) + 6)
    # one decode step: append, index, select, sparse attention
    q, k, v = qkv[n:].split([Hq, Hkv, Hkv], dim=1)
    q_rot = torch.empty((1, Hq, 128), dtype=torch.bfloat16, device="cuda")
    ln = batch_tensors(None, [n + 1])[1]
    qasc.kv_rope_append_paged(q, k, v, q_rot, K, V, table, ln, inv)
    W = synth.projection(1, 0, Hkv, "cuda")
    index = torch.zeros((pps + 2, Hkv, P, 32), dtype=torch.bfloat16, device="cuda")
    qasc.ts_index_append_paged(K, W, index, table, 0, n + 1)
    nc = n + 1 - sink - local
    sel = torch.empty((1, nc), dtype=torch.int32, device="cuda")
    wss = qasc.alloc_workspace(qasc.ts_select_workspace_bytes(1, Hq, Hkv, n + 1, pps * P, nc, sink, local))
    qasc.ts_score_vote_select_paged(q_rot, W, index, table, sel, wss, n=n + 1, K=nc, sink=sink, local=local)
    ref = torch.empty((1, Hq, 128), dtype=torch.float32, device="cuda")
    wsa = qasc.alloc_workspace(qasc.ts_attn_workspace_bytes(1, Hq, Hkv, n + 1, pps * P, nc, sink, local))
    qasc.ts_sparse_attn_paged(q_rot, K, V, table, sel, ref, wsa, n=n + 1, sink=sink, local=local)
    out = torch.empty((1, Hq, 128), dtype=torch.bfloat16, device="cuda")
    qasc.kv_window_attn_paged(q_rot, K, V, table, ln, out, ws, sink=sink, local=n + 1)
    qasc.qasc_device_error()
    # every candidate selected: both attend to all tokens
    assert float((out.float() - ref).abs().max()) <= 2.0 ** -8 * (float(ref.abs().max()) + 6) + 1e-3


def test_shared_prefix_equals_private_copies():
    """Sequences that share a prefix, their own tokens rotated behind it,
    against the same tokens in one cache per sequence."""
    Hq, Hkv, P, n0, B, m = 8, 2, 64, 192, 3, 5
    inv = freqs(128).cuda()
    pre = rand((n0, 2 * Hkv, 128), 51).cuda()
    own_qkv = rand((B * m, Hq + 2 * Hkv, 128), 52).cuda()
    q, k, v = own_qkv.split([Hq, Hkv, Hkv], dim=1)
    cu = [0, m, 2 * m, 3 * m]
    pages0, num_pages = n0 // P, n0 // P + B
    K = torch.full((num_pages, Hkv, P, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    ptable = torch.arange(pages0, dtype=torch.int32, device="cuda")
    stable = (pages0 + torch.arange(B, dtype=torch.int32, device="cuda"))[:, None].contiguous()
    c0, ln0 = batch_tensors([0, n0], [n0])
    qasc.kv_rope_append_paged(None, pre[:, :Hkv], pre[:, Hkv:], None, K, V, ptable[None].contiguous(), ln0, inv,
                              cu_q=c0)
    c, ln = batch_tensors(cu, [m] * B)
    behind = (n0 + torch.arange(m, dtype=torch.int32)).repeat(B).cuda()
    q_rot = torch.empty((B * m, Hq, 128), dtype=torch.bfloat16, device="cuda")
    qasc.kv_rope_append_paged(q, k, v, q_rot, K, V, stable, ln, inv, cu_q=c, positions=behind)
    out = torch.empty_like(q_rot)
    ws = qasc.alloc_workspace(qasc.kv_prefix_attn_workspace_bytes(B * m, B, Hq, Hkv, P))
    qasc.kv_prefix_attn_paged(q_rot, K, V, ptable, stable, ln, out, ws, n_prefix=n0, cu_q=c)
    table = torch.cat([ptable.expand(B, -1), stable], dim=1).contiguous()
    ref = torch.empty_like(out)
    ws2 = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(B * m, B, Hq, Hkv, table.shape[1] * P))
    qasc.kv_window_attn_paged(q_rot, K, V, table, batch_tensors(None, [n0 + m] * B)[1], ref, ws2, sink=0,
                              local=n0 + m, cu_q=c)
    qasc.qasc_device_error()
    assert float((out.float() - ref.float()).abs().max()) <= 2 * 2.0 ** -8 * (float(ref.float().abs().max()) + 6)
