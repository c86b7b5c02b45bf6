"""GPU parity of the 4-bit cache's calls (kv4_rope_append*, kv4_read*, kv4_window_attn*,
kv4_sparse_attn*) against the fp64 oracle.

Tolerances, fixed before the first run (A = sum_j p_j |V_j|, from the oracle):
  codes, scales   equal: the oracle quantises the fp64 rotation rounded to bf16, which
                  the kernel has to 2^-38
  values read     equal
  rotated query   2^-8 |y| (one rounding to bf16: half a step) + 2^-20 (|x_a| + |x_b|)
  logit           e = 2^-17 max_j sum_e |q_e K_e| / sqrt(d) (128 fp32 additions of
                  exact products, 128 2^-24 each relative to the sum of magnitudes)
  output          2^-8 |out| (one rounding) + 2^-11 A (each fp16 probability: half a
                  step is 2^-11 relative) + n 2^-35 max |V| (those below fp16's normal range:
                  2^-25 absolute where the largest is 2^10); 2^-8 A where a sequence has
                  more than 128 rows in a group (token, head) and goes by the bf16 copy and
                  its bf16 probabilities (half a step 2^-8)
                  + 2 (e + 2^-18) A (a logit's error moves a weight and the sum)
                  + (n 2^-24 + 2^-20) A (fp32 sums over n keys)
  lse             e + n 2^-24 + 2^-20 + 2^-22 |lse|
Rows of the cache that nothing attends to hold NaN scales, block-table entries that
must not be read lie outside the pool, and outputs are canaries beforehand.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import kv4 as okv4
from oracle import serving as osv
from oracle import tokenselect as ots
from oracle.bf16 import round_bf16

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


def packed(x, t=1.0):
    """Codes and scale bytes (CPU uint8 tensors) of fp64 rows, and their values."""
    codes, sf = okv4.quantise(x, t)
    return torch.from_numpy(codes), torch.from_numpy(sf), okv4.values(codes, sf, t)


class Pages4:
    """4-bit pools with the caches of several sequences: NaN scales everywhere else, and
    a table whose unused entries lie outside the pool.  random: codes and scales drawn
    at once (large caches)."""

    def __init__(self, lens, Hkv, P, pps, seed, extra=3, t=(1.0, 1.0), kscale=1.0, random=False):
        self.lens, self.Hkv, self.P, self.pps, self.t = list(lens), Hkv, P, pps, t
        self.num_pages = sum(cdiv(n, P) for n in lens) + extra
        order = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((len(lens), pps), POISON, dtype=torch.int32)
        self.codes = torch.full((2, self.num_pages, Hkv, P, 64), 255, dtype=torch.uint8)
        self.sf = torch.full((2, self.num_pages, Hkv, P, 8), 127, dtype=torch.uint8)
        self.logical = []
        for b, n in enumerate(lens):
            held = []
            for side in range(2):
                if random:
                    g = torch.Generator().manual_seed(seed + 10 * b + side)
                    c = torch.randint(0, 256, (Hkv, n, 64), generator=g, dtype=torch.uint8)
                    s = torch.randint(40, 56, (Hkv, n, 8), generator=g, dtype=torch.uint8)   # 0.25 .. 0.94
                    v = None
                else:
                    x = f64(rand((Hkv, n, 128), seed + 10 * b + side + 1, kscale if side == 0 else 1.0))
                    c, s, v = packed(x * t[side], t[side])
                held.append((c, s, v))
            for i in range(cdiv(n, P)):
                page = order.pop()
                self.table[b, i] = page
                m = min(P, n - i * P)
                for side, (c, s, _) in enumerate(held):
                    self.codes[side, page, :, :m] = c[:, i * P:i * P + m]
                    self.sf[side, page, :, :m] = s[:, i * P:i * P + m]
            self.logical.append(held)

    def hide(self, b, lo, hi):
        """Rows [lo, hi) of sequence b get NaN scales; pages wholly inside them
        leave the table."""
        for t in range(lo, hi):
            page = int(self.table[b, t // self.P])
            if page >= 0:
                self.sf[:, page, :, t % self.P] = 127
        for i in range(cdiv(lo, self.P), hi // self.P):
            self.table[b, i] = POISON

    def cache(self):
        c, s = self.codes.cuda(), self.sf.cuda().view(torch.float8_e4m3fn)
        return qasc.KV4(c[0], s[0], c[1], s[1], *self.t)

    def contiguous(self, n_cap):
        B = len(self.lens)
        codes = torch.full((2, B, self.Hkv, n_cap, 64), 255, dtype=torch.uint8)
        sf = torch.full((2, B, self.Hkv, n_cap, 8), 127, dtype=torch.uint8)
        for b, n in enumerate(self.lens):
            for t in range(n):
                page = int(self.table[b, t // self.P])
                if page >= 0:
                    codes[:, b, :, t] = self.codes[:, page, :, t % self.P]
                    sf[:, b, :, t] = self.sf[:, page, :, t % self.P]
        c, s = codes.cuda(), sf.cuda().view(torch.float8_e4m3fn)
        return qasc.KV4(c[0], s[0], c[1], s[1], *self.t)

    def values(self, side):
        return [held[side][2] if held[side][2] is not None else
                okv4.values(held[side][0].numpy(), held[side][1].numpy(), self.t[side]) for held in self.logical]


def batch_tensors(cu, lens):
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return c, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_rows(out, lse, ref, n_keys, vmax, rows=None, p=2.0 ** -11):
    want, want_lse, A, zabs = ref
    got, got_lse = f64(out), lse.cpu().numpy().astype(np.float64)
    if rows is not None:
        got, got_lse, want, want_lse, A, zabs = (x[rows] for x in (got, got_lse, want, want_lse, A, zabs))
        p = p if np.isscalar(p) else p[rows]
    e = 2.0 ** -17 * zabs
    sums = n_keys * 2.0 ** -24 + 2.0 ** -20
    tol = (2.0 ** -8 * np.abs(want) + (p + 2 * (e[..., None] + 2.0 ** -18) + sums) * A
           + n_keys * 2.0 ** -35 * vmax + 1e-30)
    bad = np.abs(got - want) / tol
    assert np.all(np.isfinite(got)), "output not finite"
    assert bad.max() <= 1.0, "output off by %.2f tolerances at %s" % (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    ltol = e + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, want_lse))
    ldiff = np.abs(np.where(empty, 0, got_lse) - np.where(empty, 0, want_lse))
    assert np.all(ldiff <= ltol), "lse off by %.2f tolerances" % (ldiff / ltol).max()


def p_error(ql, gq):
    """Per token [T, 1, 1]: the relative error of its probabilities."""
    return np.concatenate([np.full((m, 1, 1), 2.0 ** -8 if m * gq > 128 else 2.0 ** -11) for m in ql])


def outputs(T, Hq):
    return (torch.full((T, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda"),
            torch.full((T, Hq), CANARY, dtype=torch.float32, device="cuda"))


def window_ws(T, B, Hq, Hkv, n_cap, local, sink=4, max_q=None):
    ws = qasc.alloc_workspace(qasc.kv4_window_attn_workspace_bytes(T, B, Hq, Hkv, n_cap, local=local, sink=sink,
                                                                   max_q=max_q))
    ws.fill_(255)
    return ws


def window(q, pages, cu, lens, sink, local, max_q=None):
    """kv4_window_attn_paged into canary outputs."""
    T, Hq, _ = q.shape
    out, lse = outputs(T, Hq)
    ws = window_ws(T, len(lens), Hq, pages.Hkv, pages.pps * pages.P, local, sink, max_q)
    c, ln = batch_tensors(cu, lens)
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, ws, sink=sink, local=local, cu_q=c,
                               max_q=max_q, lse=lse)
    qasc.qasc_device_error()
    return out, lse


def goes_over_a_copy(T, B, Hq, Hkv, n_cap, local, sink, max_q):
    size = qasc.kv4_window_attn_workspace_bytes
    return size(T, B, Hq, Hkv, n_cap, local=local, sink=sink, max_q=max_q) > size(T, B, Hq, Hkv, n_cap, local=local, sink=sink, max_q=1)


def vmax_of(pages):
    return max(np.abs(v).max() if v.size else 0.0 for v in pages.values(1))


# --------------------------------------------------------------------- append
APPEND = [
    # Hq, Hkv, P, new tokens, lens, rot, interleaved, override of positions, factors
    (8, 2, 64, [1, 1, 1], [1, 64, 130], 128, False, False, (1.0, 1.0)),
    (8, 2, 64, [70, 0, 3, 129], [70, 9, 67, 400], 64, True, False, (1.0, 0.25)),
    (8, 8, 128, [33], [300], 128, True, False, (4.0, 2.0 ** -20)),
    (16, 8, 64, [5, 6], [4000, 90], 48, False, True, (1.0, 1.0)),
    (8, 1, 64, [40], [64], 16, False, False, (2.0 ** -9, 1.0)),
    (64, 8, 256, [700], [700], 128, False, True, (1.0, 1.0)),
    (4, 4, 64, [9, 2], [9, 2], 0, False, False, (1.0, 1.0)),
    (8, 2, 64, [20], [25], 112, False, False, (1.0, 1.0)),
    (8, 2, 64, [20], [25], 80, True, False, (1.0, 1.0)),
]


def special_rows(k, v):
    """Groups whose quotients stand on the codes' borders, zeros of both signs, the ends
    of the scales' range, infinities and NaN (in v; k where it is not rotated)."""
    x = torch.tensor([12, -12, 0.5, 1.5, 2.5, 3.5, 5, 7, 10, -0.5, 1, -0.0, 3, 0, 6, 8])
    v[0, 0, :16] = x.bfloat16()
    v[0, 0, 16:32] = x.bfloat16() * 2.0 ** -9
    v[0, 0, 32:48] = 0
    v[0, 0, 48:64] = 6 * 2.0 ** -10
    v[0, 0, 64:80] = 6.375                                 # its scale stands between two
    v[0, -1, 80:96] = torch.tensor([float("inf"), -float("inf"), 3e38, -1.0] * 4).bfloat16()
    v[0, -1, 96] = float("nan")
    v[0, -1, 112:128] = torch.tensor([2800.0, -2800.0, 2688.0, 100.0] * 4).bfloat16()
    k[-1, 0] *= 300


@pytest.mark.parametrize("Hq,Hkv,P,ql,lens,rot,inter,override,t", APPEND)
@pytest.mark.parametrize("paged", [True, False])
def test_append(Hq, Hkv, P, ql, lens, rot, inter, override, t, paged):
    T, B = sum(ql), len(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    single = ql == [1] * B
    extra = 0 if single else 2                             # tokens of no sequence
    qkv = rand((T + extra, Hq + 2 * Hkv, 128), 5)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    special_rows(k, v)
    k, v = k * t[0], v * t[1]
    qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:] = k, v
    f = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float()
    pos = torch.randint(0, 1 << 24, (T + extra,), generator=torch.Generator().manual_seed(6)).int() if override else None
    seq, cpos = osv.positions(cu, lens, T)
    rpos = cpos if pos is None else pos[:T].numpy()
    krot = round_bf16(osv.rotate(f64(k[:T]), rpos, f.numpy(), inter))
    qrot = osv.rotate(f64(q[:T]), rpos, f.numpy(), inter)
    want = [okv4.quantise(krot, t[0]), okv4.quantise(f64(v[:T]), t[1])]

    n_cap = cdiv(max(lens), P) * P + P
    num_pages = B * n_cap // P + 2
    rows = num_pages if paged else B
    codes = torch.full((2, rows, Hkv, P if paged else n_cap, 64), 0x5a, dtype=torch.uint8)
    sf = torch.full((2, rows, Hkv, P if paged else n_cap, 8), 0x11, dtype=torch.uint8)
    table = torch.randperm(num_pages, generator=torch.Generator().manual_seed(8))[:B * n_cap // P].reshape(B, -1).int()
    for b in range(B):                                     # pages that nothing is written to must not be read
        first = max(0, lens[b] - ql[b]) // P
        table[b, :first] = POISON
        table[b, cdiv(lens[b], P) if ql[b] else 0:] = POISON
    exp_codes, exp_sf = codes.numpy().copy(), sf.numpy().copy()
    for i in range(T):
        p = int(cpos[i])
        at = (int(table[seq[i], p // P]), slice(None), p % P) if paged else (seq[i], slice(None), p)
        for side in range(2):
            exp_codes[side][at], exp_sf[side][at] = want[side][0][i], want[side][1][i]
    dc, ds = codes.cuda(), sf.cuda()
    kv = qasc.KV4(dc[0], ds[0].view(torch.float8_e4m3fn), dc[1], ds[1].view(torch.float8_e4m3fn), *t)
    c, ln = batch_tensors(None if single else cu, lens)
    d = qkv.cuda()
    q_out = torch.full((T + extra, Hq, 128), CANARY, dtype=torch.bfloat16, device="cuda")
    args = (d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], q_out, kv)
    kw = dict(cu_q=c, positions=None if pos is None else pos.cuda(), interleaved=inter)
    freq = f.cuda() if rot else None
    if paged:
        qasc.kv4_rope_append_paged(*args, table.cuda(), ln, freq, **kw)
    else:
        qasc.kv4_rope_append(*args, ln, freq, **kw)
    qasc.qasc_device_error()
    got_codes, got_sf = dc.cpu().numpy(), ds.cpu().numpy()
    assert np.array_equal(got_sf, exp_sf)
    broken = np.repeat(exp_sf == 127, 8, axis=-1)          # a NaN group's codes may be any
    assert np.array_equal(np.where(broken, 0, got_codes), np.where(broken, 0, exp_codes))
    mag = np.zeros_like(qrot)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        mag[..., a] = mag[..., b] = np.abs(f64(q[:T]))[..., a] + np.abs(f64(q[:T]))[..., b]
    assert np.all(np.abs(f64(q_out[:T]) - qrot) <= 2.0 ** -8 * np.abs(qrot) + 2.0 ** -20 * mag)
    assert bool((q_out[T:] == CANARY).all())


def test_append_of_a_long_prompt_is_exact():
    """2048 tokens at far positions: 4 million rotated keys, each rounded as the fp64 rotation is."""
    T, Hkv, P = 2048, 16, 64
    k, v = rand((T, Hkv, 128), 9), rand((T, Hkv, 128), 10)
    f = (500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    pos = (torch.arange(T) * 61 + 3).int()
    want = okv4.quantise(round_bf16(osv.rotate(f64(k), pos.numpy(), f.numpy(), False)))
    kv = qasc.alloc_kv4(1, Hkv, T)
    c, ln = batch_tensors([0, T], [T])
    qasc.kv4_rope_append(None, k.cuda(), v.cuda(), None, kv, ln, f.cuda(), cu_q=c, positions=pos.cuda())
    qasc.qasc_device_error()
    assert np.array_equal(kv.K_sf.view(torch.uint8)[0].cpu().numpy().transpose(1, 0, 2), want[1])
    assert np.array_equal(kv.K[0].cpu().numpy().transpose(1, 0, 2), want[0])


# Position, frequency, and a pair (a, b) one of whose rotated values stands 2^-33 to 2^-28 beside the middle
# between a border of two codes of scale 1 and the next bf16 value: the angle has to be better than
# that at these positions for the code to be right (a product of 53 bits is 2^-29 off there).
BORDERS = [
    (16774594, 0.8815479278564453, -1.6953125, 3.640625),
    (16777213, 0.6797472238540649, 3.453125, 0.5390625),
    (16775826, 0.6150959730148315, 0.84765625, 1.65625),
    (15199687, 0.8867228031158447, -1.4453125, 1.359375),
    (16774875, 0.8313730955123901, -1.484375, 1.9296875),
    (16776500, 0.6090608835220337, -2.921875, 1.0390625),
]


@pytest.mark.parametrize("sign", [1, -1])
def test_append_beside_the_codes_borders_at_far_positions(sign):
    """A value of 6 that does not turn makes the scale 1; the pair turns at its own frequency."""
    T = len(BORDERS)
    k = torch.zeros((T, 1, 128))
    f = torch.zeros(64)
    k[:, 0, 0] = 6
    for t, (_, freq, a, b) in enumerate(BORDERS):
        f[1 + t] = freq
        k[t, 0, 2 + 2 * t], k[t, 0, 3 + 2 * t] = a, sign * b    # (the angle's sign turned with b's: the same values)
    k, f = k.bfloat16(), f * sign
    pos = torch.tensor([p for p, *_ in BORDERS], dtype=torch.int32)
    want = okv4.quantise(round_bf16(osv.rotate(f64(k), pos.numpy(), f.numpy(), True)))
    kv = qasc.alloc_kv4(1, 1, T)
    c, ln = batch_tensors([0, T], [T])
    qasc.kv4_rope_append(None, k.cuda(), k.cuda(), None, kv, ln, f.cuda(), cu_q=c, positions=pos.cuda(), interleaved=True)
    qasc.qasc_device_error()
    assert np.array_equal(kv.K_sf.view(torch.uint8)[0].cpu().numpy().transpose(1, 0, 2), want[1])
    assert np.array_equal(kv.K[0].cpu().numpy().transpose(1, 0, 2), want[0])


def test_append_at_far_positions():
    """4 million rotated keys below position 2^24, and in front of position 0."""
    T, Hkv = 2048, 16
    k = rand((T, Hkv, 128), 73)
    f = (500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    pos = ((1 << 24) - 1 - 3 * torch.arange(T)).int()
    pos[::16] = -pos[::16]
    want = okv4.quantise(round_bf16(osv.rotate(f64(k), pos.numpy(), f.numpy(), False)))
    kv = qasc.alloc_kv4(1, Hkv, T)
    c, ln = batch_tensors([0, T], [T])
    qasc.kv4_rope_append(None, k.cuda(), k.cuda(), None, kv, ln, f.cuda(), cu_q=c, positions=pos.cuda())
    qasc.qasc_device_error()
    assert np.array_equal(kv.K_sf.view(torch.uint8)[0].cpu().numpy().transpose(1, 0, 2), want[1])
    assert np.array_equal(kv.K[0].cpu().numpy().transpose(1, 0, 2), want[0])


@pytest.mark.parametrize("inter", [True, False])
def test_append_rotates_infinities_and_nan(inter):
    """Infinite, huge and NaN keys under rotation, at position 0 as well (where infinity times sin 0 is NaN)."""
    T, Hkv = 40, 2
    k = rand((T, Hkv, 128), 82)
    g = torch.Generator().manual_seed(83)
    for value in (float("inf"), -float("inf"), float("nan"), 3.3e38, -3.3e38, 3e-39):
        at = torch.randint(0, T * Hkv * 128, (12,), generator=g)
        k.reshape(-1)[at] = value
    k[0, 0, 0], k[0, 1, 70] = float("inf"), float("nan")
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    with np.errstate(invalid="ignore", over="ignore"):
        want = okv4.quantise(round_bf16(osv.rotate(f64(k), np.arange(T), f.numpy(), inter)))
    kv = qasc.alloc_kv4(1, Hkv, T)
    c, ln = batch_tensors([0, T], [T])
    qasc.kv4_rope_append(None, k.cuda(), k.cuda(), None, kv, ln, f.cuda(), cu_q=c, interleaved=inter)
    qasc.qasc_device_error()
    codes, sf = kv.K[0].cpu().numpy().transpose(1, 0, 2), kv.K_sf.view(torch.uint8)[0].cpu().numpy().transpose(1, 0, 2)
    assert np.array_equal(sf, want[1]) and (sf == 127).any() and (sf == 126).any()
    broken = np.repeat(sf == 127, 8, axis=-1)              # a NaN group's codes may be any
    assert np.array_equal(np.where(broken, 0, codes), np.where(broken, 0, want[0]))


@pytest.mark.parametrize("inter", [True, False])
def test_append_of_zeros_keeps_their_signs(inter):
    """Pairs of zeros of either sign at angles of every quadrant: the code's sign bit is that of the rotation."""
    T = 64
    k = torch.zeros((T, 2, 128))
    k[:, 1] = -0.0
    k[:, :, 3::7] *= -1
    f = (torch.arange(64) * 0.37 + 0.1).float()
    want = okv4.quantise(round_bf16(osv.rotate(f64(k.bfloat16()), np.arange(T), f.numpy(), inter)))
    kv = qasc.alloc_kv4(1, 2, T)
    c, ln = batch_tensors([0, T], [T])
    kd = k.bfloat16().cuda()
    qasc.kv4_rope_append(None, kd, kd, None, kv, ln, f.cuda(), cu_q=c, interleaved=inter)
    qasc.qasc_device_error()
    assert np.array_equal(kv.K[0].cpu().numpy().transpose(1, 0, 2), want[0])
    assert 8 in want[0] and 128 in want[0]                 # signs of either value of a byte
    assert np.array_equal(kv.V[0].cpu().numpy().transpose(1, 0, 2), okv4.quantise(f64(kd))[0])


def test_append_does_not_depend_on_the_cut():
    """Token by token, in chunks and at once: the same cache, bit for bit."""
    T, Hkv = 900, 4
    k, v = rand((T, Hkv, 128), 11).cuda(), rand((T, Hkv, 128), 12).cuda()
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    caches = []
    for cuts in ([0, T], [0, 1, 2, 3, 500, 501, 899, T]):
        kv = qasc.alloc_kv4(1, Hkv, T + 3)
        for lo, hi in zip(cuts, cuts[1:]):
            c, ln = batch_tensors([0, hi - lo], [hi])
            qasc.kv4_rope_append(None, k[lo:hi], v[lo:hi], None, kv, ln, f, cu_q=c)
        caches.append(kv)
    qasc.qasc_device_error()
    for name in ("K", "K_sf", "V", "V_sf"):
        a, b = (getattr(kv, name).view(torch.uint8) for kv in caches)
        assert torch.equal(a, b)


def test_append_in_place_and_without_queries():
    T, Hq, Hkv = 300, 16, 4
    q, k, v = (rand((T, h, 128), 16 + h).cuda() for h in (Hq, Hkv, 2 * Hkv))
    v = v[:, ::2].contiguous()
    f = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    c, ln = batch_tensors([0, T], [T + 5])
    caches, outs = [], []
    for way in ("apart", "in place", "none"):
        kv = qasc.alloc_kv4(1, Hkv, T + 5)
        qq = q.clone()
        out = {"apart": torch.zeros_like(q), "in place": qq, "none": None}[way]
        qasc.kv4_rope_append(None if out is None else qq, k, v, out, kv, ln, f, cu_q=c)
        caches.append(kv)
        outs.append(out)
    qasc.qasc_device_error()
    assert torch.equal(outs[0], outs[1])
    for kv in caches[1:]:
        assert torch.equal(kv.K, caches[0].K) and torch.equal(kv.V_sf.view(torch.uint8), caches[0].V_sf.view(torch.uint8))


@pytest.mark.parametrize("ql", [[1, 1, 1], [300, 2, 400]])
def test_append_and_read_replay_in_a_graph(ql):
    """A captured call follows the lengths and offsets on the device."""
    T, Hkv, P = sum(ql), 2, 64
    single = ql == [1] * 3
    k, v = rand((T, Hkv, 128), 17).cuda(), rand((T, Hkv, 128), 18).cuda()
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    table = torch.arange(30, dtype=torch.int32).reshape(3, 10).cuda()
    c, ln = batch_tensors(None if single else np.concatenate([[0], np.cumsum(ql)]).tolist(), [m + 5 for m in ql])

    def call(kv, K, V):
        qasc.kv4_rope_append_paged(None, k, v, None, kv, table, ln, f, cu_q=c)
        qasc.kv4_read_paged(kv, table, ln, K, V, cu_q=c)

    def fresh():
        return qasc.alloc_kv4(30, Hkv, P), torch.zeros_like(k), torch.zeros_like(v)
    one, two = fresh(), fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(*one)
    for shift in (0, 40):
        ln.copy_(torch.tensor([m + 5 + shift for m in ql], dtype=torch.int32))
        graph.replay()
        call(*two)
        torch.cuda.synchronize()
        assert torch.equal(one[0].K, two[0].K) and torch.equal(one[0].V, two[0].V)
        assert torch.equal(one[1], two[1]) and torch.equal(one[2], two[2]) and bool(one[1].any())
    qasc.qasc_device_error()


@pytest.mark.parametrize("bad", ["page", "position", "length"])
def test_append_and_read_skip_what_lies_outside(bad):
    P, Hkv = 64, 2
    lens, ql = [70, 130], [70, 5]
    cu = [0, 70, 75]
    table = torch.tensor([[1, 2, 5], [3, 4, 0]], dtype=torch.int32)
    if bad == "page":
        table[0, 1] = 9                                    # tokens 64 .. 69 of sequence 0
        lost = range(64, 70)
    elif bad == "position":
        lens[1] = 3                                        # its first two stand in front of the cache
        lost = range(70, 72)
    else:
        lens[1] = 3 * P + 2                                # its last two behind it
        lost = range(73, 75)
    k, v = rand((75, Hkv, 128), 13).cuda(), rand((75, Hkv, 128), 14).cuda()
    kv = qasc.alloc_kv4(6, Hkv, P)
    c, ln = batch_tensors(cu, lens)
    qasc.kv4_rope_append_paged(None, k, v, None, kv, table.cuda(), ln, None, cu_q=c)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    K, V = (torch.full((75, Hkv, 128), CANARY, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qasc.kv4_read_paged(kv, table.cuda(), ln, K, V, cu_q=c)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    keep = torch.ones(75, dtype=torch.bool)
    keep[list(lost)] = False
    assert bool((K[~keep] == CANARY).all()) and bool((V[~keep] == CANARY).all())
    assert np.array_equal(f64(K[keep]), okv4.values(*okv4.quantise(f64(k[keep]))))
    assert np.array_equal(f64(V[keep]), okv4.values(*okv4.quantise(f64(v[keep]))))


# ----------------------------------------------------------------------- read
@pytest.mark.parametrize("Hkv,P,ql,lens,t", [
    (2, 64, [5, 0, 64, 130], [5, 9, 64, 300], (1.0, 1.0)),
    (8, 128, [1], [1000], (2.0 ** -6, 8.0)),
    (1, 64, [257], [257], (1.0, 2.0 ** 30)),
])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("split_heads", [True, False])
def test_read(Hkv, P, ql, lens, t, paged, split_heads):
    T = sum(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P) + 1, 15, t=t)
    for b, n in enumerate(lens):
        pages.hide(b, 0, n - ql[b])
    c, ln = batch_tensors(cu, lens)
    if split_heads:                                        # heads first, tokens behind each other, with room between
        K, V = (torch.full((Hkv, T + 9, 128), CANARY, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        outs = K.transpose(0, 1)[:T + 2], V.transpose(0, 1)[:T + 2]
    else:
        K, V = (torch.full((T + 2, Hkv, 128), CANARY, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        outs = K, V
    if paged:
        qasc.kv4_read_paged(pages.cache(), pages.table.cuda(), ln, *outs, cu_q=c)
    else:
        qasc.kv4_read(pages.contiguous(max(lens) + 3), ln, *outs, cu_q=c)
    qasc.qasc_device_error()
    for side, out in enumerate(outs):
        want = np.concatenate([x[:, n - m:n] for x, n, m in zip(pages.values(side), lens, ql)], axis=1)
        assert np.array_equal(f64(out[:T]).transpose(1, 0, 2), want)
        assert bool((out[T:] == CANARY).all())
    if split_heads:
        assert bool((K[:, T + 2:] == CANARY).all())


def test_read_of_every_code_and_scale():
    kv = qasc.alloc_kv4(1, 1, 256)
    kv.K.copy_(torch.arange(256, dtype=torch.uint8).reshape(1, 1, 256, 1).expand(1, 1, 256, 64))
    kv.K_sf.view(torch.uint8).copy_(torch.arange(256, dtype=torch.uint8).reshape(1, 1, 256, 1).expand(1, 1, 256, 8))
    kv.V.copy_(kv.K.flip(2))
    kv.V_sf.view(torch.uint8).copy_(kv.K_sf.view(torch.uint8).flip(2).roll(1, 2))
    K, V = (torch.zeros((256, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c, ln = batch_tensors([0, 256], [256])
    qasc.kv4_read(kv, ln, K, V, cu_q=c)
    for out, codes, sf in ((K, kv.K, kv.K_sf), (V, kv.V, kv.V_sf)):
        want = okv4.values(codes[0, 0].cpu().numpy(), sf.view(torch.uint8)[0, 0].cpu().numpy())
        assert np.array_equal(f64(out[:, 0]), want, equal_nan=True)


# --------------------------------------------------------------------- window
WINDOW = [
    # Hq, Hkv, P, new tokens, lens, sink, local
    (8, 2, 64, [1, 1, 1, 1], [1, 31, 64, 300], 4, 1000),
    (32, 8, 64, [1, 1], [200, 517], 4, 64),
    (8, 8, 64, [1, 1], [33, 700], 3, 5000),
    (16, 8, 128, [1], [1500], 0, 400),
    (64, 8, 256, [1], [600], 4, 600),
    (8, 2, 64, [131, 1, 0, 40], [131, 90, 77, 400], 4, 100),
    (8, 1, 128, [33, 2], [33, 257], 130, 17),
    (8, 4, 64, [64, 65], [64, 321], 0, 128),
    (64, 8, 64, [9], [140], 1, 139),
    (8, 2, 64, [5, 3], [2, 3], 4, 9),          # three tokens stand in front of their cache
    (8, 2, 64, [300], [300], 0, 300),
    (8, 2, 64, [3, 0, 2], [0, 0, 130], 2, 1),
    (32, 8, 64, [5, 5, 5], [700, 5, 64], 4, 90),
]


@pytest.mark.parametrize("Hq,Hkv,P,ql,lens,sink,local", WINDOW)
@pytest.mark.parametrize("paged", [True, False])
def test_window(Hq, Hkv, P, ql, lens, sink, local, paged):
    T, B = sum(ql), len(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P) + 1, seed=21, t=(0.5, 4.0) if paged else (1.0, 1.0))
    single = ql == [1] * B
    q = rand((T + (0 if single else 2), Hq, 128), 22)      # two tokens of no sequence
    ref = osv.window_attention(f64(q[:T]), pages.values(0), pages.values(1), cu, lens, sink, local)
    for b, n in enumerate(lens):                           # what no query attends to
        first = max(0, n - ql[b])
        if ql[b] == 0:
            pages.hide(b, 0, n)
        elif first - local + 1 > sink:
            pages.hide(b, sink, first - local + 1)
    cu_arg = None if single else cu
    if paged:
        out, lse = window(q, pages, cu_arg, lens, sink, local, max_q=max(ql))
    else:
        n_cap = max(lens) + 5
        out, lse = outputs(q.shape[0], Hq)
        c, ln = batch_tensors(cu_arg, lens)
        ws = window_ws(q.shape[0], B, Hq, Hkv, n_cap, local, sink)
        qasc.kv4_window_attn(q.cuda(), pages.contiguous(n_cap), ln, out, ws, sink=sink, local=local, cu_q=c, lse=lse)
        qasc.qasc_device_error()
    check_rows(out[:T], lse[:T], ref, max(lens), vmax_of(pages), p=p_error(ql, Hq // Hkv))
    assert bool((out[T:] == CANARY).all()) and bool((lse[T:] == CANARY).all())


@pytest.mark.parametrize("max_q", [1, 2, 7, 60])
def test_window_max_q_changes_no_answer(max_q):
    """A number that is too small or too large: other kernels, the same rows."""
    ql, lens = [7, 1, 50, 2], [300, 77, 400, 2]
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, 2, 64, 8, seed=23)
    q = rand((60, 8, 128), 24)
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), cu, lens, 4, 120)
    out, lse = window(q, pages, cu, lens, 4, 120, max_q=max_q)
    check_rows(out, lse, ref, 400, vmax_of(pages), p=p_error(ql, 4))


@pytest.mark.parametrize("qscale", [0.0, 1e-30, 20.0, 1e4])
def test_window_flat_and_peaked_logits(qscale):
    lens, P = [900, 33], 64
    pages = Pages4(lens, 2, P, 16, seed=25)
    q = rand((2, 8, 128), 26, qscale)
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), [0, 1, 2], lens, 4, 5000)
    out, lse = window(q, pages, None, lens, 4, 5000)
    check_rows(out, lse, ref, 900, vmax_of(pages))


def test_window_queries_of_very_different_values():
    """One value of a query row 2^20 times the others: those keep their bits as well."""
    pages = Pages4([500], 2, 64, 9, seed=27)
    q = rand((1, 8, 128), 28)
    q[0, :, 5] = 2.0 ** -20
    q[0, ::2, 7] = 2.0 ** 12
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), [0, 1], [500], 4, 5000)
    out, lse = window(q, pages, None, [500], 4, 5000)
    check_rows(out, lse, ref, 500, vmax_of(pages))


def test_window_growing_maximum():
    """Keys whose logits grow along the sequence: the base moves again and again."""
    n, Hkv = 3000, 2
    pages = Pages4([n], Hkv, 64, cdiv(n, 64), seed=29)
    q = rand((1, 8, 128), 30)
    ramp = np.linspace(0, 30, n)[None, :, None] * np.sign(f64(q)[0, ::4])[:, None, :] / 16
    held = pages.logical[0]
    c, s, v = packed(ramp + held[0][2] * 0.1)
    held[0] = (c, s, v)
    for i in range(cdiv(n, 64)):
        page, m = int(pages.table[0, i]), min(64, n - 64 * i)
        pages.codes[0, page, :, :m], pages.sf[0, page, :, :m] = c[:, 64 * i:64 * i + m], s[:, 64 * i:64 * i + m]
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), [0, 1], [n], 4, n)
    out, lse = window(q, pages, None, [n], 4, n)
    check_rows(out, lse, ref, n, vmax_of(pages))


LONG = [
    # Hq, Hkv, new tokens, lens, sink, local: shared between blocks
    (8, 2, [1], [40000], 4, 40000),
    (64, 8, [1, 1], [9000, 20001], 4, 19000),
    (8, 8, [1] * 5, [7000, 1, 300, 12345, 64], 0, 100000),
    (32, 8, [3, 2], [9000, 8999], 4, 100000),
    (8, 1, [40], [6000], 4, 5500),
]


@pytest.mark.parametrize("Hq,Hkv,ql,lens,sink,local", LONG)
def test_window_shared_between_blocks(Hq, Hkv, ql, lens, sink, local):
    T, P = sum(ql), 128
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P), seed=31, random=True)
    q = rand((T, Hq, 128), 32)
    out, lse = window(q, pages, cu, lens, sink, local, max_q=max(ql))
    K, V = pages.values(0), pages.values(1)
    tokens = sorted({0, T // 2, T - 1})
    ref = osv.window_attention(f64(q), K, V, cu, lens, sink, local, tokens=tokens)
    check_rows(out, lse, ref, max(lens), 6.0, rows=tokens, p=p_error(ql, Hq // Hkv))


def test_window_of_many_sequences():
    B, Hq, Hkv, P = 2048, 4, 2, 64
    lens = [1 + (37 * b) % 150 for b in range(B)]
    pages = Pages4(lens, Hkv, P, 3, seed=33, random=True)
    q = rand((B, Hq, 128), 34)
    out, lse = window(q, pages, None, lens, 4, 100)
    tokens = list(range(0, B, 61)) + [B - 1]
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), list(range(B + 1)), lens, 4, 100, tokens=tokens)
    check_rows(out, lse, ref, 150, 6.0, rows=tokens)


@pytest.mark.parametrize("ql,local", [(1, 400), (1, 100), (3, 400)])
def test_window_of_more_short_items_than_warps(ql, local):
    """Items of a few hundred tokens, which blocks then share."""
    B, Hq, Hkv, n = 240, 16, 8, 620
    pages = Pages4([n], Hkv, 64, 10, seed=69, random=True)
    pages.table = pages.table.repeat(B, 1)                 # all sequences over the same pages
    lens = [n - (7 * b) % 300 for b in range(B)]
    K, V = ([pages.values(side)[0][:, :m] for m in lens] for side in range(2))
    T, cu = ql * B, list(range(0, ql * B + 1, ql))
    q = rand((T, Hq, 128), 70)
    out, lse = outputs(T, Hq)
    c, ln = batch_tensors(cu if ql > 1 else None, lens)
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, window_ws(T, B, Hq, Hkv, 640, local, 4, ql),
                               local=local, cu_q=c, max_q=ql, lse=lse)
    qasc.qasc_device_error()
    tokens = list(range(0, T, 17)) + [T - 1]
    ref = osv.window_attention(f64(q), K, V, cu, lens, 4, local, tokens=tokens)
    check_rows(out, lse, ref, n, 6.0, rows=tokens)


def test_window_equals_the_bf16_call_on_the_cache_read_back():
    """What kv4_read gives, attended to by kv_window_attn: the same up to both calls' roundings."""
    lens, ql, Hq, Hkv, n_cap = [700, 64], [90, 1], 16, 4, 704
    pages = Pages4(lens, Hkv, 64, 11, seed=35)
    kv = pages.contiguous(n_cap)
    q = rand((91, Hq, 128), 36).cuda()
    c, ln = batch_tensors([0, 90, 91], lens)
    K, V = (torch.zeros((2, Hkv, n_cap, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        one = qasc.KV4(*(x[b:b + 1] for x in (kv.K, kv.K_sf, kv.V, kv.V_sf)))
        cb, lb = batch_tensors([0, n], [n])
        qasc.kv4_read(one, lb, K[b, :, :n].transpose(0, 1), V[b, :, :n].transpose(0, 1), cu_q=cb)
    want, want_lse = outputs(91, Hq)
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(91, 2, Hq, Hkv, n_cap))
    qasc.kv_window_attn(q, K, V, ln, want, ws, local=300, cu_q=c, lse=want_lse)
    out, lse = outputs(91, Hq)
    qasc.kv4_window_attn(q, kv, ln, out, window_ws(91, 2, Hq, Hkv, n_cap, 300), local=300, cu_q=c, lse=lse)
    qasc.qasc_device_error()
    A = float(np.abs(pages.values(1)[0]).max())
    # bf16 outputs (2^-8 each) and probabilities (2^-8 and 2^-11) of values up to A
    assert float((out.float() - want.float()).abs().max()) <= A * (2 * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)
    assert float((lse - want_lse).abs().max()) <= 1e-4


@pytest.mark.parametrize("tk,tv", [(-32, 32), (32, -32)])
@pytest.mark.parametrize("Hq,Hkv,ql,lens,local", [
    (8, 2, [1, 1], [700, 33], 300),                        # whole items
    (8, 1, [3], [6000], 6000),                             # shared between blocks
    (64, 8, [300, 2], [900, 80], 1000),                    # over a copy
])
def test_window_of_factors_at_the_ends_of_their_range(Hq, Hkv, ql, lens, local, tk, tv):
    T, P, cu = sum(ql), 64, np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P), seed=84, random=True, t=(2.0 ** tk, 2.0 ** tv))
    q = rand((T, Hq, 128), 85, 0.3 * 2.0 ** -tk)
    assert goes_over_a_copy(T, len(ql), Hq, Hkv, pages.pps * P, local, 4, max(ql)) == (max(ql) == 300)
    out, lse = window(q, pages, cu, lens, 4, local, max_q=max(ql))
    tokens = sorted({0, T // 2, T - 1})
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), cu, lens, 4, local, tokens=tokens)
    check_rows(out, lse, ref, max(lens), 6.0 * 2.0 ** tv, rows=tokens, p=p_error(ql, Hq // Hkv))


def test_window_rows_that_are_not_copied_keep_fp16_probabilities():
    """More than 128 rows of a sequence, on the 4-bit cache because the call says so (max_q) or has no room for a copy:
    the smaller of the two errors."""
    Hq, Hkv, P, ql, lens, local = 64, 8, 64, [200, 40], [1500, 700], 1000
    T, cu = sum(ql), [0, 200, 240]
    pages = Pages4(lens, Hkv, P, 24, seed=86, random=True)
    q = rand((T, Hq, 128), 87, 0.3)
    tokens = [0, 77, 199, 200, 239]
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), cu, lens, 4, local, tokens=tokens)
    assert goes_over_a_copy(T, 2, Hq, Hkv, 24 * P, local, 4, 200)
    c, ln = batch_tensors(cu, lens)
    for max_q in (1, 16, 200):
        ws = window_ws(T, 2, Hq, Hkv, 24 * P, local, 4, 1)
        out, lse = outputs(T, Hq)
        qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, ws, local=local, cu_q=c, max_q=max_q, lse=lse)
        qasc.qasc_device_error()
        check_rows(out, lse, ref, 1500, 6.0, rows=tokens)


@pytest.mark.parametrize("n,m", [(1900, 1), (900, 40)])
@pytest.mark.parametrize("side", [0, 1])
def test_window_not_a_number_stays_visible(n, m, side):
    Hq, Hkv = 8, 2
    pages = Pages4([n], Hkv, 64, cdiv(n, 64), seed=37, random=True)
    at = n - m                                             # the first new token: all new ones see it
    pages.sf[side, int(pages.table[0, at // 64]), 1, at % 64, 3] = 127
    q = rand((m, Hq, 128), 38)
    out, lse = window(q, pages, [0, m], [n], 4, n, max_q=m)
    assert bool(torch.isfinite(out[:, :4].float()).all()) and bool(torch.isfinite(lse[:, :4]).all())
    if side == 0:
        assert bool(torch.isnan(out[:, 4:].float()).all()) and bool(torch.isnan(lse[:, 4:]).all())
    else:
        assert bool(torch.isnan(out[:, 4:, 48:64].float()).all()) and bool(torch.isfinite(lse).all())
        assert bool(torch.isfinite(out[:, 4:, :48].float()).all()) and bool(torch.isfinite(out[:, 4:, 64:].float()).all())


@pytest.mark.parametrize("ql,n_cap", [([1, 1, 1], 256), ([9, 2, 40], 512)])
def test_window_lengths_outside_are_clamped_and_reported(ql, n_cap):
    P, Hkv = 64, 2
    T, cu = sum(ql), np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4([n_cap] * 3, Hkv, P, n_cap // P, seed=39, random=True)
    q = rand((T, 8, 128), 40)
    ref = window(q, pages, cu, [n_cap, 0, 100], 4, 90)
    out, lse = outputs(T, 8)
    c, ln = batch_tensors(cu, [n_cap + 5, -3, 100])
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out,
                               window_ws(T, 3, 8, Hkv, n_cap, 90), local=90, cu_q=c, lse=lse)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_window_bad_page_is_reported():
    pages = Pages4([300], 2, 64, 5, seed=41, random=True)
    pages.table[0, 2] = pages.num_pages
    out, lse = outputs(1, 8)
    q = rand((1, 8, 128), 42)
    ln = batch_tensors(None, [300])[1]
    ws = window_ws(1, 1, 8, 2, 320, 300)
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, ws, local=300, lse=lse)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    K, V = pages.values(0), pages.values(1)
    K[0][:, 128:192], V[0][:, 128:192] = 0, 0              # rows of zeros
    check_rows(out, lse, osv.window_attention(f64(q), K, V, [0, 1], [300], 4, 300), 300, 6.0)
    # behind the window it is not read
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, ws, local=100, lse=lse)
    qasc.qasc_device_error()


@pytest.mark.parametrize("T,B,n", [(1, 1, 5000), (300, 1, 1400), (40, 40, 900)])
def test_window_is_deterministic_and_replays_in_a_graph(T, B, n):
    Hq, Hkv, P = 16, 4, 128
    lens = [n - 17 * b for b in range(B)]
    pages = Pages4(lens, Hkv, P, cdiv(n, P), seed=43, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    q = rand((T, Hq, 128), 44).cuda()
    c, ln = batch_tensors(None if T == B else [0, T], lens)
    ws = window_ws(T, B, Hq, Hkv, pages.pps * P, 700)

    def call(out, lse):
        qasc.kv4_window_attn_paged(q, kv, table, ln, out, ws, local=700, cu_q=c, lse=lse)

    a, b, g_out = outputs(T, Hq), outputs(T, Hq), outputs(T, Hq)
    call(*a)
    ws.fill_(255)
    call(*b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(*g_out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], g_out[0]) and torch.equal(a[1], g_out[1])
    ln.copy_(torch.tensor([max(1, x - 200) for x in lens], dtype=torch.int32))   # the replay follows the lengths
    graph.replay()
    call(*a)
    torch.cuda.synchronize()
    assert torch.equal(a[0], g_out[0]) and not torch.equal(a[0], b[0])
    qasc.qasc_device_error()


@pytest.mark.parametrize("kind", ["single", "packed", "listed"])
def test_short_items_of_several_warps_keep_every_part(kind):
    """One item for the warps of a block, a tile or two each, joined at its end: in thousands of
    launches none of the warps' parts is left out."""
    Hq, Hkv, P, n = 8, 1, 64, 380
    pages = Pages4([n], Hkv, P, cdiv(n, P), seed=71, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    q = rand((1, Hq, 128), 72).cuda()
    c, ln = batch_tensors([0, 1] if kind == "packed" else None, [n])
    sel = torch.arange(4, n - 64, dtype=torch.int32, device="cuda").reshape(1, -1)
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), [0, 1], [n], 4, n)
    outs = [torch.full((2000, 1, Hq, w), CANARY, dtype=t, device="cuda") for w, t in ((128, torch.bfloat16), (1, torch.float32))]
    wss = [window_ws(1, 1, Hq, Hkv, pages.pps * P, n) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2000):
        out, lse, s = outs[0][i], outs[1][i, :, :, 0], streams[i % 2]
        if kind == "listed":
            qasc.kv4_sparse_attn_paged(q, kv, table, sel, out, wss[i % 2], n=n, local=64, lse=lse, stream=s)
        else:
            qasc.kv4_window_attn_paged(q, kv, table, ln, out, wss[i % 2], local=n, cu_q=c, lse=lse, stream=s)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    check_rows(outs[0][0], outs[1][0, :, :, 0], ref, n, 6.0)
    for o in outs:
        assert torch.equal(o, o[:1].expand_as(o))


def test_two_windows_on_two_streams():
    Hq, Hkv, P, n = 16, 4, 64, 6000
    pages = Pages4([n, n - 3], Hkv, P, cdiv(n, P), seed=45, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    q = rand((2, Hq, 128), 46).cuda()
    ln = batch_tensors(None, [n, n - 3])[1]
    outs = [outputs(2, Hq)[0] for _ in range(3)]
    wss = [window_ws(2, 2, Hq, Hkv, pages.pps * P, n) for _ in range(3)]
    qasc.kv4_window_attn_paged(q, kv, table, ln, outs[2], wss[2], local=n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            qasc.kv4_window_attn_paged(q, kv, table, ln, outs[i], wss[i], local=n, stream=s)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("ql,lens,local", [([300, 1, 200], [900, 700, 800], 300), ([300, 1, 200], [4000, 3000, 2500], 5000)])
def test_two_windows_over_copies_on_two_streams(ql, lens, local):
    """The rest and the copy beside it, or one behind the other, of two calls at once, each with a workspace of its own."""
    Hq, Hkv, P, T = 64, 8, 64, sum(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P), seed=88, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    assert goes_over_a_copy(T, 3, Hq, Hkv, pages.pps * P, local, 4, 300)
    qs = [rand((T, Hq, 128), 89 + i, 0.3).cuda() for i in range(2)]
    c, ln = batch_tensors(cu, lens)
    wss = [window_ws(T, 3, Hq, Hkv, pages.pps * P, local, 4, 300) for _ in range(2)]
    wants, gots = ([outputs(T, Hq) for _ in range(2)] for _ in range(2))
    for q, want, ws in zip(qs, wants, wss):
        qasc.kv4_window_attn_paged(q, kv, table, ln, want[0], ws, local=local, cu_q=c, max_q=300, lse=want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, got, ws, s in zip(qs, gots, wss, streams):
            qasc.kv4_window_attn_paged(q, kv, table, ln, got[0], ws, local=local, cu_q=c, max_q=300, lse=got[1], stream=s)
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    for want, got in zip(wants, gots):
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_two_graphs_take_turns_with_one_workspace():
    """Nothing of a call stays in its workspace: a call shared between blocks, one that is not
    and two over a copy, captured with the same one and replayed in turn."""
    Hq, Hkv, P, n = 16, 2, 64, 5000
    pages = Pages4([n, n - 9], Hkv, P, cdiv(n, P), seed=47, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    kinds = [([0, 1, 2], 2, n, 1), ([0, 1, 2], 2, 300, 1), ([0, 400, 560], 560, 2000, 400), ([0, 550, 560], 560, 1000, 550)]
    assert all(goes_over_a_copy(560, 2, Hq, Hkv, pages.pps * P, local, 4, m) for _, _, local, m in kinds[2:])
    ws = qasc.alloc_workspace(max(qasc.kv4_window_attn_workspace_bytes(T, 2, Hq, Hkv, pages.pps * P, local=local, max_q=m)
                                  for _, T, local, m in kinds))
    ln = batch_tensors(None, [n, n - 9])[1]
    graphs, outs, wants = [], [], []
    for cu, T, local, m in kinds:
        q, c = rand((T, Hq, 128), 48 + T).cuda(), batch_tensors(cu, [0])[0]
        out, want = outputs(T, Hq), outputs(T, Hq)

        def call(o, ws=ws, q=q, c=c, local=local, m=m):
            qasc.kv4_window_attn_paged(q, kv, table, ln, o[0], ws, local=local, cu_q=c, max_q=m, lse=o[1])
        call(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            call(out)
        graphs.append((graph, call))
        outs.append(out)
        wants.append(want)
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    qasc.qasc_device_error()
    for out, want in zip(outs, wants):
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def repeated(n, Hkv, P, seed):
    """A sequence of n tokens whose pages come around again: a long context in a small pool."""
    pages = Pages4([8 * P], Hkv, P, 8, seed=seed, random=True)
    first = pages.table[0].clone()
    pages.pps = cdiv(n, P)
    pages.table = first.repeat(cdiv(pages.pps, 8))[:pages.pps].reshape(1, -1).contiguous()
    reps = cdiv(n, 8 * P)
    values = [np.concatenate([pages.values(side)[0]] * reps, axis=1)[:, :n] for side in range(2)]
    return pages, values


def test_window_places_of_more_than_a_tile():
    """So many row blocks of so wide a table that a place of the line is several tiles."""
    T, Hq, Hkv, P, n = 8200, 8, 1, 64, 9000
    pages, values = repeated(n, Hkv, P, 49)
    wide = 1 << 17                                          # n_cap = 2^23
    table = torch.full((1, wide), POISON, dtype=torch.int32)
    table[0, :pages.pps] = pages.table[0]
    q = rand((T, Hq, 128), 50)
    out, lse = outputs(T, Hq)
    c, ln = batch_tensors([0, T], [n])
    ws = window_ws(T, 1, Hq, Hkv, wide * P, 64, max_q=1)
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), table.cuda(), ln, out, ws, local=64, cu_q=c, max_q=1, lse=lse)
    qasc.qasc_device_error()
    tokens = [0, 3, 700, 4099, T - 1]
    ref = osv.window_attention(f64(q), values[:1], values[1:], [0, T], [n], 4, 64, tokens=tokens)
    check_rows(out, lse, ref, 68, 6.0, rows=tokens)


def test_window_longer_than_the_copy():
    """A chunk of a context that the copy has no room for stands beside one that it has."""
    Hq, Hkv, P, ql = 64, 64, 64, [130, 131]
    lens = [140000, 300]
    long, values = repeated(lens[0], Hkv, P, 51)
    pps = long.pps
    table = torch.cat([long.table, long.table[:, :8].repeat(1, cdiv(pps, 8))[:, :pps]])
    q = rand((261, Hq, 128), 52)
    c, ln = batch_tensors([0, 130, 261], lens)
    out, lse = outputs(261, Hq)
    ws = window_ws(261, 2, Hq, Hkv, pps * P, lens[0], max_q=131)
    assert goes_over_a_copy(261, 2, Hq, Hkv, pps * P, lens[0], 4, 131) and ws.numel() < 5 << 30   # 4 GiB of a copy at most
    qasc.kv4_window_attn_paged(q.cuda(), long.cache(), table.cuda(), ln, out, ws, local=lens[0], cu_q=c, max_q=131, lse=lse)
    qasc.qasc_device_error()
    for t, h in ((0, 0), (77, 63), (129, 31), (130, 5), (260, 63)):
        b = t >= 130
        n = lens[b] - ql[b] + t - (130 if b else 0) + 1
        want = osv.attend(f64(q)[t, h], values[0][h, :n], values[1][h, :n])
        ref = tuple(np.asarray(x)[None, None] for x in want)
        check_rows(out[t:t + 1, h:h + 1].contiguous(), lse[t:t + 1, h:h + 1], ref, n, 6.0, p=2.0 ** -8)


COPIED = [
    # Hq, Hkv, P, new tokens, lens, sink, local: calls that go over a copy
    (64, 8, 64, [200, 1, 300, 2], [1500, 900, 800, 77], 4, 100000),
    (64, 8, 128, [400, 30, 0, 1], [1300, 700, 50, 1], 4, 300),
    (64, 8, 64, [700], [5000], 200, 90),
    (8, 8, 64, [1000, 129], [1000, 4000], 0, 2500),
    (64, 8, 64, [150, 16, 17, 400], [100, 2000, 2000, 401], 4, 1000),   # more new tokens than cached ones
]


@pytest.mark.parametrize("Hq,Hkv,P,ql,lens,sink,local", COPIED)
def test_window_over_a_copy(Hq, Hkv, P, ql, lens, sink, local):
    T, B = sum(ql), len(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, P, cdiv(max(lens), P) + 1, seed=61, random=True, t=(0.5, 4.0))
    K, V = pages.values(0), pages.values(1)
    for b, n in enumerate(lens):                           # what no query attends to
        first = max(0, n - ql[b])
        if ql[b] == 0:
            pages.hide(b, 0, n)
        elif first - local + 1 > sink:
            pages.hide(b, sink, first - local + 1)
    assert goes_over_a_copy(T + 2, B, Hq, Hkv, pages.pps * P, local, sink, max(ql))
    q = rand((T + 2, Hq, 128), 62, 0.3)                    # two tokens of no sequence
    out, lse = window(q, pages, cu, lens, sink, local, max_q=max(ql))
    tokens = sorted({t for a, z in zip(cu, cu[1:]) if z > a for t in (a, (a + z) // 2, z - 1)})
    ref = osv.window_attention(f64(q[:T]), K, V, cu, lens, sink, local, tokens=tokens)
    check_rows(out[:T], lse[:T], ref, max(lens), 24.0, rows=tokens, p=p_error(ql, Hq // Hkv))
    # and every row against the calls without a copy, with both roundings
    out1, lse1 = window(q, pages, cu, lens, sink, local, max_q=1)
    assert float((out[:T].float() - out1[:T].float()).abs().max()) <= 24.0 * (2 * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)
    finite = torch.isfinite(lse1[:T])
    assert torch.equal(finite, torch.isfinite(lse[:T]))
    assert float((lse[:T][finite] - lse1[:T][finite]).abs().max()) <= 1e-3
    assert bool((out[T:] == CANARY).all()) and bool((lse[T:] == CANARY).all())


@pytest.mark.parametrize("pages", [0, 5, 6, 9, 11])
def test_window_with_less_workspace_than_the_whole_copy(pages):
    """Room for no page, for less than, just as much as and more than the longest sequence takes, and for nearly all of
    them: the same rows, from a copy or from the 4-bit cache."""
    Hq, Hkv, P, ql, lens, local = 64, 8, 64, [200, 1, 300, 2], [1500, 900, 800, 77], 1200
    T, cu = sum(ql), np.concatenate([[0], np.cumsum(ql)]).tolist()
    caches = Pages4(lens, Hkv, P, 24, seed=78, random=True)
    size = qasc.kv4_window_attn_workspace_bytes
    full = size(T, 4, Hq, Hkv, 24 * P, local=local, max_q=300)
    least = size(1, 4, Hq, Hkv, 24 * P, local=local, max_q=1)
    page = 2 * Hkv * 256 * 256                              # of 256 tokens; sequences of up to 1503 tokens take 6
    assert full - least > 24 * page and goes_over_a_copy(T, 4, Hq, Hkv, 24 * P, local, 4, 300)
    ws = qasc.alloc_workspace(full - (24 - pages) * page if pages else least)
    ws.fill_(255)
    q = rand((T, Hq, 128), 79, 0.3)
    c, ln = batch_tensors(cu, lens)
    out, lse = outputs(T, Hq)
    qasc.kv4_window_attn_paged(q.cuda(), caches.cache(), caches.table.cuda(), ln, out, ws, local=local, cu_q=c, max_q=300, lse=lse)
    qasc.qasc_device_error()
    tokens = [0, 100, 199, 200, 201, 350, 500, 501, 502]
    ref = osv.window_attention(f64(q), caches.values(0), caches.values(1), cu, lens, 4, local, tokens=tokens)
    check_rows(out, lse, ref, 1500, 6.0, rows=tokens, p=p_error(ql, Hq // Hkv))
    whole, whole_lse = window(q, caches, cu, lens, 4, local, max_q=300)
    assert float((out.float() - whole.float()).abs().max()) <= 6.0 * (2 * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)
    assert float((lse - whole_lse).abs().max()) <= 1e-3


@pytest.mark.parametrize("T,m", [(103, 53), (96, 53), (53, 53), (16, 1)])
def test_window_smaller_calls_take_the_largest_ones_workspace(T, m):
    """A workspace sized once, at 103 tokens of up to 53, where a call does not copy and a smaller one does."""
    B, Hq, Hkv, P, n = 16, 32, 8, 256, 131072
    pages = Pages4([2000], Hkv, P, 8, seed=80, random=True)
    table = torch.full((B, n // P), POISON, dtype=torch.int32)
    table[:, :8] = pages.table
    ws = qasc.alloc_workspace(qasc.kv4_window_attn_workspace_bytes(103, B, Hq, Hkv, n, local=4096, max_q=53))
    ql = [m] + [1] * (T - m) + [0] * (B - 1 - (T - m)) if T - m < B else [m, T - m - (B - 2)] + [1] * (B - 2)
    cu, lens = np.concatenate([[0], np.cumsum(ql)]).tolist(), [2000 - b for b in range(B)]
    q = rand((T, Hq, 128), 81, 0.3)
    c, ln = batch_tensors(cu, lens)
    out, lse = outputs(T, Hq)
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), table.cuda(), ln, out, ws, local=4096, cu_q=c, max_q=m, lse=lse)
    qasc.qasc_device_error()
    K, V = ([pages.values(side)[0][:, :x] for x in lens] for side in range(2))
    tokens = sorted({0, T // 2, T - 1})
    check_rows(out, lse, osv.window_attention(f64(q), K, V, cu, lens, 4, 4096, tokens=tokens), 2000, 6.0, rows=tokens,
               p=p_error(ql, Hq // Hkv))


def test_window_over_a_copy_of_a_contiguous_cache():
    Hq, Hkv, ql, lens, n_cap, sink, local = 64, 8, [300, 2, 140], [900, 70, 333], 960, 4, 500
    T = sum(ql)
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    pages = Pages4(lens, Hkv, 64, n_cap // 64, seed=63, random=True)
    assert goes_over_a_copy(T, 3, Hq, Hkv, n_cap, local, sink, max(ql))
    q = rand((T, Hq, 128), 64, 0.3)
    out, lse = outputs(T, Hq)
    c, ln = batch_tensors(cu, lens)
    qasc.kv4_window_attn(q.cuda(), pages.contiguous(n_cap), ln, out, window_ws(T, 3, Hq, Hkv, n_cap, local, sink, max(ql)),
                         sink=sink, local=local, cu_q=c, max_q=max(ql), lse=lse)
    qasc.qasc_device_error()
    tokens = [0, 150, 299, 300, 301, 302, T - 1]
    ref = osv.window_attention(f64(q), pages.values(0), pages.values(1), cu, lens, sink, local, tokens=tokens)
    check_rows(out, lse, ref, max(lens), 6.0, rows=tokens, p=p_error(ql, Hq // Hkv))


@pytest.mark.parametrize("local,max_q", [(2000, 6), (2000, None), (100, 6)])
def test_window_offsets_that_do_not_ascend(local, max_q):
    """Each sequence as its own two offsets say; a token that two of them have is one's or the other's."""
    cu, lens, Hq, Hkv = [0, 5, 3, 9, 9], [1500, 50, 1700, 80], 8, 2
    pages = Pages4(lens, Hkv, 64, 27, seed=65, random=True)
    q = rand((9, Hq, 128), 66)
    out, lse = window(q, pages, cu, lens, 4, local, max_q=max_q)
    K, V = pages.values(0), pages.values(1)
    for b, lo, hi, own in ((0, 0, 5, slice(0, 3)), (2, 3, 9, slice(2, 6))):
        ref = osv.window_attention(f64(q)[lo:hi], K[b:b + 1], V[b:b + 1], [0, hi - lo], [lens[b]], 4, local)
        rows = list(range(hi - lo))[own]
        check_rows(out[lo:hi], lse[lo:hi], ref, lens[b], 6.0, rows=rows)


@pytest.mark.parametrize("lens", [[20000, 50, 19900], [300, 50, 400]])
def test_window_offsets_that_do_not_ascend_over_a_copy(lens):
    """Two long sequences where T tokens can have one, and the copy room for one of 20000 cached tokens: recorded.
    The next call over the same workspace is right again."""
    T, Hq, Hkv, P, n = 20, 64, 8, 64, 20000
    pages, values = repeated(n, Hkv, P, 76)
    q = rand((T, Hq, 128), 77, 0.3)
    kv, table = pages.cache(), pages.table.repeat(3, 1).cuda()
    ws = window_ws(T, 3, Hq, Hkv, pages.pps * P, n, 4, 17)
    assert goes_over_a_copy(T, 3, Hq, Hkv, pages.pps * P, n, 4, 17)

    def call(cu):
        out, lse = outputs(T, Hq)
        c, ln = batch_tensors(cu, lens)
        qasc.kv4_window_attn_paged(q.cuda(), kv, table, ln, out, ws, local=n, cu_q=c, max_q=17, lse=lse)
        return out, lse
    call([0, 17, 3, 20])
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    for cu in ([0, 17, 17, 20], [-5, 0, 3, 27]):            # (values outside [0, T] are clamped)
        out, lse = call(cu)
        qasc.qasc_device_error()
        cu = [min(max(x, 0), T) for x in cu]
        for b, t, h in ((0, 0, 0), (0, 16, 63), (1, 1, 3), (2, 17, 5), (2, 19, 40)):
            if not cu[b] <= t < cu[b + 1]:
                continue
            m = lens[b] - (cu[b + 1] - t) + 1
            want = osv.attend(f64(q)[t, h], values[0][h // 8, :m], values[1][h // 8, :m])
            check_rows(out[t:t + 1, h:h + 1].contiguous(), lse[t:t + 1, h:h + 1].contiguous(),
                       tuple(np.asarray(x)[None, None] for x in want), m, 6.0, p=2.0 ** -8)


def test_window_bad_page_of_a_copied_sequence():
    Hq, Hkv, n, m = 64, 8, 1500, 300
    pages = Pages4([n], Hkv, 64, 24, seed=53, random=True)
    pages.table[0, 2] = -1
    assert goes_over_a_copy(m, 1, Hq, Hkv, 24 * 64, n, 4, m)
    q = rand((m, Hq, 128), 54)
    out, lse = outputs(m, Hq)
    c, ln = batch_tensors([0, m], [n])
    qasc.kv4_window_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), ln, out, window_ws(m, 1, Hq, Hkv, 24 * 64, n), local=n,
                               cu_q=c, lse=lse)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    K, V = pages.values(0), pages.values(1)
    K[0][:, 128:192], V[0][:, 128:192] = 0, 0               # rows of zeros
    tokens = [0, 100, m - 1]
    check_rows(out, lse, osv.window_attention(f64(q), K, V, [0, m], [n], 4, n, tokens=tokens), n, 6.0, rows=tokens, p=2.0 ** -8)


# --------------------------------------------------------------------- sparse
def sparse_ref(q, pages, lists, n, sink, local):
    """lists[b][g]: listed tokens."""
    B, Hq, _ = q.shape
    out, lse = np.zeros((B, Hq, 128)), np.full((B, Hq), -np.inf)
    A, zabs = np.zeros_like(out), np.zeros_like(lse)
    K, V = pages.values(0), pages.values(1)
    end = min(n, sink)
    always = list(range(end)), list(range(max(end, n - local), n))
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // pages.Hkv)
            j = np.array(always[0] + list(lists[b][g]) + always[1], dtype=np.int64)
            out[b, h], lse[b, h], A[b, h], zabs[b, h] = osv.attend(q[b, h], K[b][g][j], V[b][g][j])
    return out, lse, A, zabs


SPARSE = [
    # B, Hq, Hkv, n, K, sink, local, per head, lengths
    (1, 8, 2, 600, 100, 4, 256, False, False),
    (2, 32, 8, 700, 77, 4, 64, True, True),
    (3, 8, 8, 300, 0, 4, 256, False, False),
    (2, 8, 1, 400, 200, 0, 0, False, True),
    (2, 16, 8, 900, 300, 0, 0, True, True),
    (1, 64, 8, 5, 0, 4, 256, False, False),
    (1, 8, 4, 20000, 9000, 4, 256, True, False),
]


@pytest.mark.parametrize("B,Hq,Hkv,n,K,sink,local,per_head,with_len", SPARSE)
@pytest.mark.parametrize("paged", [True, False])
def test_sparse(B, Hq, Hkv, n, K, sink, local, per_head, with_len, paged):
    P = 64
    pages = Pages4([n] * B, Hkv, P, cdiv(n, P) + 2, seed=51, random=n > 2000, t=(2.0, 0.25))
    g = torch.Generator().manual_seed(52)
    c1 = max(sink, n - local)
    rows = B * (Hkv if per_head else 1)
    sel = torch.stack([(sink + torch.randperm(c1 - sink, generator=g)[:K]) for _ in range(rows)]).int()
    lens = None
    if with_len:
        lens = torch.randint(0, K + 1, (rows,), generator=g).int()
        lens[0] = 0                                        # no entry; without sink and local no token at all
        lens[-1] = K + 9                                   # clamped
        for i in range(rows):
            sel[i, min(K, int(lens[i])):] = 1 << 30        # entries that are not in use
    lists = [[sel[b * Hkv + gg if per_head else b][:K if lens is None else min(K, int(lens[b * Hkv + gg if per_head else b]))].tolist()
              for gg in range(Hkv)] for b in range(B)]
    q = rand((B, Hq, 128), 53)
    ref = sparse_ref(f64(q), pages, lists, n, sink, local)
    # what no head attends to
    for b in range(B):
        used = set(range(min(n, sink))) | set(range(max(min(n, sink), n - local), n))
        used |= {t for gg in range(Hkv) for t in lists[b][gg]}
        if n <= 2000:
            for t in range(n):
                if t not in used:
                    pages.hide(b, t, t + 1)
    shape = (B, Hkv) if per_head else (B,)
    out, lse = outputs(B, Hq)
    args = dict(n=n, sink=sink, local=local, lengths=None if lens is None else lens.reshape(shape).cuda(),
                per_kv_head=per_head, lse=lse)
    sel_arg = sel.reshape(*shape, K).cuda() if K else None
    n_cap = pages.pps * P if paged else n + 7
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, n, n_cap, K, sink, local))
    ws.fill_(255)
    if paged:
        qasc.kv4_sparse_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), sel_arg, out, ws, **args)
    else:
        qasc.kv4_sparse_attn(q.cuda(), pages.contiguous(n_cap), sel_arg, out, ws, **args)
    qasc.qasc_device_error()
    check_rows(out, lse, ref, n, max(6.0, vmax_of(pages)))


@pytest.mark.parametrize("K", [40, 300])
def test_sparse_of_many_lists(K):
    B, Hq, Hkv, n, P = 300, 16, 8, 900, 64
    pages = Pages4([n], Hkv, P, cdiv(n, P), seed=57, random=True)
    table = pages.table.repeat(B, 1).cuda()                 # all sequences over the same pages
    g = torch.Generator().manual_seed(58)
    sel = torch.randint(4, n - 64, (B, Hkv, K), generator=g).int()      # in any order, some twice
    lens = torch.randint(0, K + 1, (B, Hkv), generator=g).int()
    q = rand((B, Hq, 128), 59)
    out, lse = outputs(B, Hq)
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, n, pages.pps * P, K, 4, 64))
    qasc.kv4_sparse_attn_paged(q.cuda(), pages.cache(), table, sel.cuda(), out, ws, n=n, local=64, lengths=lens.cuda(),
                               per_kv_head=True, lse=lse)
    qasc.qasc_device_error()
    rows = list(range(0, B, 37)) + [B - 1]
    K1, V1 = pages.values(0) * B, pages.values(1) * B

    class Held:
        values = staticmethod(lambda side: [(K1, V1)[side][b] for b in rows])
    Held.Hkv = Hkv
    ref = sparse_ref(f64(q)[rows], Held, [[sel[b, gg, :int(lens[b, gg])].tolist() for gg in range(Hkv)] for b in rows], n, 4, 64)
    check_rows(out[rows], lse[rows], ref, n, 6.0)


@pytest.mark.parametrize("tk,tv", [(-32, 32), (32, -32)])
def test_sparse_of_factors_at_the_ends_of_their_range(tk, tv):
    n, P = 900, 64
    pages = Pages4([n], 2, P, 15, seed=91, random=True, t=(2.0 ** tk, 2.0 ** tv))
    q = rand((1, 8, 128), 92, 0.3 * 2.0 ** -tk)
    sel = torch.arange(10, 710, 7, dtype=torch.int32).reshape(1, -1)
    out, lse = outputs(1, 8)
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, n, 960, 100, 4, 64))
    qasc.kv4_sparse_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), sel.cuda(), out, ws, n=n, local=64, lse=lse)
    qasc.qasc_device_error()
    check_rows(out, lse, sparse_ref(f64(q), pages, [[sel[0].tolist()] * 2], n, 4, 64), n, 6.0 * 2.0 ** tv)


def test_sparse_replays_in_a_graph():
    """The captured call follows the lists and their lengths; a list of the whole context is split."""
    B, Hq, Hkv, n, K, P = 2, 32, 8, 6000, 4000, 64
    pages = Pages4([n] * B, Hkv, P, cdiv(n, P), seed=55, random=True)
    kv, table = pages.cache(), pages.table.cuda()
    q = rand((B, Hq, 128), 56).cuda()
    sel = torch.arange(4, 4 + K, dtype=torch.int32).repeat(B, 1).cuda()
    lens = torch.full((B,), K, dtype=torch.int32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, n, pages.pps * P, K))

    def call(o):
        qasc.kv4_sparse_attn_paged(q, kv, table, sel, o[0], ws, n=n, lengths=lens, lse=o[1])
    got, want = outputs(B, Hq), outputs(B, Hq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(got)
    for use in ([K, K], [17, 3000], [0, K]):
        lens.copy_(torch.tensor(use, dtype=torch.int32))
        sel.copy_(sel.flip(1) if use[0] == 17 else sel)
        graph.replay()
        call(want)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qasc.qasc_device_error()


def test_sparse_entry_outside_is_reported():
    n, P = 400, 64
    pages = Pages4([n], 2, P, 7, seed=54, random=True)
    q = rand((1, 8, 128), 55)
    sel = torch.tensor([[10, n, -1, 40]], dtype=torch.int32)
    out, lse = outputs(1, 8)
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, n, 448, 4, 4, 64))
    qasc.kv4_sparse_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), sel.cuda(), out, ws, n=n, local=64, lse=lse)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    K, V = pages.values(0), pages.values(1)
    K[0][:, 11], V[0][:, 11], K[0][:, 12], V[0][:, 12] = 0, 0, 0, 0   # rows of zeros in their places
    pages.values = lambda side: (K, V)[side]
    check_rows(out, lse, sparse_ref(f64(q), pages, [[[10, 11, 12, 40]] * 2], n, 4, 64), n, 6.0)


@pytest.mark.parametrize("entry", [-2 ** 31, -2 ** 31 + 1, 2 ** 31 - 1])
def test_sparse_entry_far_outside_is_reported(entry):
    """One entry outside, the ends of its type: a row of zeros, and recorded."""
    n, P = 400, 64
    pages = Pages4([n], 2, P, 7, seed=74, random=True)
    q = rand((1, 8, 128), 75)
    sel = torch.tensor([[10, entry, 40]], dtype=torch.int32)
    out, lse = outputs(1, 8)
    ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, n, 448, 3, 4, 64))
    qasc.kv4_sparse_attn_paged(q.cuda(), pages.cache(), pages.table.cuda(), sel.cuda(), out, ws, n=n, local=64, lse=lse)
    with pytest.raises(qasc.QascError, match="BAD_TABLE"):
        qasc.qasc_device_error()
    K, V = pages.values(0), pages.values(1)
    K[0][:, 11], V[0][:, 11] = 0, 0                         # a row of zeros in its place
    pages.values = lambda side: (K, V)[side]
    check_rows(out, lse, sparse_ref(f64(q), pages, [[[10, 11, 40]] * 2], n, 4, 64), n, 6.0)


def test_decode_steps_over_a_4_bit_cache():
    """The run of a serving loop: a prompt in two chunks, then steps that append, select on the
    index and attend to the selected tokens, against the oracle on what the cache holds."""
    B, Hq, Hkv, P, n0, K = 2, 8, 2, 64, 500, 60
    n_cap = 640
    table = torch.randperm(22, generator=torch.Generator().manual_seed(60))[:20].reshape(2, 10).int().cuda()
    kv = qasc.alloc_kv4(22, Hkv, P)
    W = rand((Hkv, 128, 32), 61, 128 ** -0.5).cuda()
    index = torch.zeros((B, Hkv, n_cap, 32), dtype=torch.bfloat16, device="cuda")
    Kb = torch.zeros((B, Hkv, n_cap, 128), dtype=torch.bfloat16, device="cuda")     # bf16 keys of the index
    Vb = torch.zeros_like(Kb)
    f = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    log = []
    at = 0
    for step, m in enumerate([300, 200, 1, 1, 1]):
        n = at + m
        qkv = rand((B * m, Hq + 2 * Hkv, 128), 70 + step).cuda()
        q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
        log.append((m, f64(k), f64(v)))
        c, ln = batch_tensors(None if m == 1 else [0, m, 2 * m], [n] * B)
        q_rot, q_same = (torch.zeros((B * m, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qasc.kv4_rope_append_paged(q, k, v, q_rot, kv, table, ln, f.cuda(), cu_q=c)
        qasc.kv_rope_append(q, k, v, q_same, Kb, Vb, ln, f.cuda(), cu_q=c)
        qasc.ts_index_append(Kb, W, index, at, m, Hq=Hq)
        at = n
        out, lse = outputs(B * m, Hq)
        if m > 1:
            ws = window_ws(B * m, B, Hq, Hkv, n_cap, n_cap, max_q=m)
            qasc.kv4_window_attn_paged(q_rot, kv, table, ln, out, ws, local=n_cap, cu_q=c, max_q=m, lse=lse)
        else:
            sel = torch.empty((B, K), dtype=torch.int32, device="cuda")
            ws = qasc.alloc_workspace(qasc.ts_select_workspace_bytes(B, Hq, Hkv, n, n_cap, K))
            qasc.ts_score_vote_select(q_rot, W, index, sel, ws, n=n, K=K)
            ws = qasc.alloc_workspace(qasc.kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, n, n_cap, K))
            qasc.kv4_sparse_attn_paged(q_rot, kv, table, sel, out, ws, n=n, lse=lse)
        qasc.qasc_device_error()
        # the cache that the oracle keeps
        pos = 0
        sides = [[], []]
        for mm, kk, vv in log:
            p = np.tile(np.arange(pos, pos + mm), B)
            sides[0].append(okv4.values(*okv4.quantise(round_bf16(osv.rotate(kk, p, f.numpy(), False)))).reshape(B, mm, Hkv, 128))
            sides[1].append(okv4.values(*okv4.quantise(vv)).reshape(B, mm, Hkv, 128))
            pos += mm
        caches = [[np.concatenate(s, axis=1)[b].transpose(1, 0, 2) for b in range(B)] for s in sides]
        vmax = max(np.abs(x).max() for x in caches[1])
        if m > 1:
            tokens = [0, m - 1, m, 2 * m - 1]
            ref = osv.window_attention(f64(q_rot), *caches, [0, m, 2 * m], [n] * B, 4, n_cap, tokens=tokens)
            check_rows(out, lse, ref, n, vmax, rows=tokens, p=p_error([m] * B, Hq // Hkv))
        else:
            S = sel.cpu().numpy()
            want, _ = ots.sparse_attention(f64(q_rot), np.stack(caches[0]), np.stack(caches[1]), S, n, 4, 256)

            class Held:
                values = staticmethod(lambda side: caches[side])
            Held.Hkv = Hkv
            ref = sparse_ref(f64(q_rot), Held, [[S[b].tolist()] * Hkv for b in range(B)], n, 4, 256)
            assert np.abs(ref[0] - want).max() < 1e-9
            check_rows(out, lse, ref, n, vmax)
