"""Packed-batch serving calls as plain fp64 NumPy: position rotation and
append, causal attention over sink and local tokens, attention over a shared
prefix.

Test infrastructure only (see the package docstring).

A batch packs the new tokens of B sequences: sequence b has tokens
cu_q[b] .. cu_q[b + 1] - 1 and lens[b] cached tokens, its new ones the last, so
that its new token i stands at position lens[b] - (cu_q[b + 1] - cu_q[b]) + i.

Shapes: q [T, Hq, d]; k, v [T, Hkv, d]; caches are lists over sequences of
[Hkv, n, d] arrays (a pool is turned into them by paged.logical_rows or by the
test).  Query head h reads KV head h // (Hq // Hkv).
"""

import numpy as np


def positions(cu_q, lens, T):
    """(sequence, position) of every packed token; sequence -1 for tokens that
    no sequence holds."""
    seq = np.full(T, -1, dtype=np.int64)
    pos = np.zeros(T, dtype=np.int64)
    for b, n in enumerate(lens):
        lo, hi = int(cu_q[b]), int(cu_q[b + 1])
        for t in range(lo, hi):
            seq[t] = b
            pos[t] = n - (hi - lo) + (t - lo)
    return seq, pos


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, d] rotated: pair i of the first 2 len(inv_freq) values of a
    head turns by the angle pos[t] * inv_freq[i]; pairs are (i, i + half), or
    (2i, 2i + 1) when interleaved."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(pos, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        xa, xb = x[:, :, a].copy(), x[:, :, b].copy()
        x[:, :, a] = xa * c - xb * s
        x[:, :, b] = xb * c + xa * s
    return x


def attended(p, sink, local):
    """Positions that a query at p attends to, ascending."""
    return np.array([j for j in range(p + 1) if j < sink or j > p - local], dtype=np.int64)


def attend(q, K, V):
    """One query row [d] over keys K [m, d] and values V [m, d]: (output, lse,
    bound of |output| under sign changes, largest sum |q_e K_e| / sqrt(d));
    (0, -inf, 0, 0) when m = 0."""
    d = q.shape[0]
    if K.shape[0] == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    z = K @ q / np.sqrt(d)
    m = z.max()
    w = np.exp(z - m)
    total = w.sum()
    w /= total
    return w @ V, m + np.log(total), w @ np.abs(V), float((np.abs(K) @ np.abs(q)).max() / np.sqrt(d))


def window_attention(q, K, V, cu_q, lens, sink, local, tokens=None):
    """Causal attention over the first `sink` and the newest `local` tokens up
    to each query's position.  K, V: lists of [Hkv, >= lens[b], d].  Returns
    out [T, Hq, d], lse [T, Hq] and, for error bounds, A = sum_j p_j |V_j| and
    the largest sum |q_e K_e| / sqrt(d) of every row.  tokens: compute these
    packed tokens only (the others stay as rows without any key)."""
    return _attention(q, K, V, cu_q, lens, sink, local, None, None, tokens)


def prefix_attention(q, Kp, Vp, K, V, cu_q, lens, tokens=None):
    """Attention over a prefix [Hkv, n0, d] and causally over each sequence's
    own tokens (lists as in window_attention)."""
    return _attention(q, K, V, cu_q, lens, 0, 1 << 40, Kp, Vp, tokens)


def _attention(q, K, V, cu_q, lens, sink, local, Kp, Vp, tokens):
    q = np.asarray(q, dtype=np.float64)
    T, Hq, d = q.shape
    Hkv = K[0].shape[0]
    out, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    A, zabs = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    seq, pos = positions(cu_q, lens, T)
    for t in range(T) if tokens is None else tokens:
        if seq[t] < 0:
            continue
        j = attended(int(pos[t]), sink, local) if sink > 0 else np.arange(max(0, pos[t] - local + 1), pos[t] + 1)
        for h in range(Hq):
            g = h // (Hq // Hkv)
            Kt, Vt = K[seq[t]][g][j], V[seq[t]][g][j]
            if Kp is not None:
                Kt, Vt = np.concatenate([Kp[g], Kt]), np.concatenate([Vp[g], Vt])
            out[t, h], lse[t, h], A[t, h], zabs[t, h] = attend(q[t, h], Kt, Vt)
    return out, lse, A, zabs
