"""What fixes the packed-batch oracle other than itself: hand-worked rotations,
the library attention with explicit masks, and the decode step's attention
over sink and local tokens."""

import numpy as np
import pytest
import torch

from oracle import serving as osv
from oracle import tokenselect as ots


def test_positions_by_hand():
    seq, pos = osv.positions([0, 2, 2, 5], [7, 4, 3], 6)
    assert seq.tolist() == [0, 0, 2, 2, 2, -1]
    assert pos.tolist()[:5] == [5, 6, 0, 1, 2]


def test_quarter_turns():
    x = np.arange(8, dtype=np.float64).reshape(1, 1, 8)
    f = [np.pi / 2, 0.0]
    y = osv.rotate(x, [1], f, False)[0, 0]                    # pairs (0, 2), (1, 3)
    assert np.allclose(y, [-2, 1, 0, 3, 4, 5, 6, 7])
    y = osv.rotate(x, [1], f, True)[0, 0]                     # pairs (0, 1), (2, 3)
    assert np.allclose(y, [-1, 0, 2, 3, 4, 5, 6, 7])
    assert np.allclose(osv.rotate(x, [-1], f, True)[0, 0], [1, 0, 2, 3, 4, 5, 6, 7])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_makes_scores_relative(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))
    f = 0.3 ** np.arange(8)
    dot = [float((osv.rotate(q, [p], f, interleaved) * osv.rotate(k, [p - 5], f, interleaved)).sum())
           for p in (5, 11, 400)]
    assert np.allclose(dot, dot[0], rtol=1e-10)


def test_window_equals_masked_library_attention():
    rng = np.random.default_rng(2)
    Hq, Hkv, d, n, m = 4, 2, 8, 23, 9
    q = rng.normal(size=(m, Hq, d))
    K, V = rng.normal(size=(Hkv, n, d)), rng.normal(size=(Hkv, n, d))
    for sink, local in ((0, 1), (0, 6), (3, 5), (4, 40)):
        out, lse, _, _ = osv.window_attention(q, [K], [V], [0, m], [n], sink, local)
        i, j = np.arange(n - m, n)[:, None], np.arange(n)[None]
        mask = (j <= i) & ((j < sink) | (j > i - local))
        tt = lambda x: torch.from_numpy(np.ascontiguousarray(x))
        ref = torch.nn.functional.scaled_dot_product_attention(
            tt(q.transpose(1, 0, 2)), tt(np.repeat(K, 2, axis=0)), tt(np.repeat(V, 2, axis=0)), attn_mask=tt(mask))
        assert np.allclose(out, ref.numpy().transpose(1, 0, 2), atol=1e-12)
        z = np.einsum("thd,hjd->htj", q, np.repeat(K, 2, axis=0)) / np.sqrt(d)
        assert np.allclose(lse, np.log(np.where(mask, np.exp(z), 0).sum(-1)).T)


def test_single_token_equals_decode_step_without_selection():
    rng = np.random.default_rng(3)
    B, Hq, Hkv, d, n, sink, local = 2, 4, 2, 16, 60, 4, 10
    q, K, V = rng.normal(size=(B, Hq, d)), rng.normal(size=(B, Hkv, n, d)), rng.normal(size=(B, Hkv, n, d))
    want, want_lse = ots.sparse_attention(q, K, V, np.zeros((B, 0), dtype=np.int64), n, sink, local)
    out, lse, _, _ = osv.window_attention(q, list(K), list(V), [0, 1, 2], [n, n], sink, local)
    assert np.allclose(out, want, atol=1e-12) and np.allclose(lse, want_lse, atol=1e-12)


def test_prefix_equals_concatenated_caches():
    rng = np.random.default_rng(4)
    Hq, Hkv, d, n0 = 4, 2, 8, 13
    Kp, Vp = rng.normal(size=(Hkv, n0, d)), rng.normal(size=(Hkv, n0, d))
    lens, cu = [5, 0, 2], [0, 3, 4, 6]
    K, V = [rng.normal(size=(Hkv, n, d)) for n in lens], [rng.normal(size=(Hkv, n, d)) for n in lens]
    q = rng.normal(size=(6, Hq, d))
    out, lse, _, _ = osv.prefix_attention(q, Kp, Vp, K, V, cu, lens)
    full = [np.concatenate([Kp, x], axis=1) for x in K], [np.concatenate([Vp, x], axis=1) for x in V]
    want, want_lse, _, _ = osv.window_attention(q, *full, cu, [n0 + n for n in lens], 0, 1 << 30)
    rows = [0, 1, 2, 4, 5]     # sequence 1 attends to the prefix alone; its token stands in front of its cache
    assert np.allclose(out[rows], want[rows]) and np.allclose(lse[rows], want_lse[rows])
    alone = osv.attend(q[3, 1], Kp[0], Vp[0])
    assert np.allclose(out[3, 1], alone[0]) and np.allclose(lse[3, 1], alone[1])


def test_no_visible_token_gives_zero():
    K = [np.ones((1, 2, 4))]
    out, lse, _, _ = osv.window_attention(np.ones((3, 1, 4)), K, K, [0, 3], [2], 1, 1)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and np.all(np.isfinite(lse[1:]))
