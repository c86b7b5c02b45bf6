"""The failure path every kernel shares, exercised on the GPU without a
fault: a bounded wait on a barrier that nothing arrives on gives up, the
kernel records a timeout and returns, qasc_device_error() reports it once,
and the context keeps working."""

import time

import pytest
import torch

import synth
from oracle import tokenselect as ots

pytestmark = pytest.mark.gpu

qasc = pytest.importorskip("query_aware_sparse_compressed_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qasc._lib.load()


def test_bounded_wait_times_out_and_is_reported_once():
    qasc.qasc_device_error()                       # start from a clear error word
    t0 = time.perf_counter()
    qasc.qasc_selftest_bounded_wait(20000)         # 20 ms
    with pytest.raises(qasc.QascError) as e:
        qasc.qasc_device_error()
    elapsed = time.perf_counter() - t0
    assert e.value.status == 5                     # QASC_ERR_TIMEOUT
    assert 0.015 < elapsed < 5.0
    qasc.qasc_device_error()                       # reported once, then cleared


def test_context_usable_after_a_timeout():
    qasc.qasc_selftest_bounded_wait(1000)
    with pytest.raises(qasc.QascError):
        qasc.qasc_device_error()
    cfg = synth.DECODE_CONFIGS["tiny"]
    x = {k: v.cuda() for k, v in synth.decode_layer(cfg, 0).items()}
    n, sink, local = cfg.n, cfg.sink, cfg.local
    K = ots.budget_tokens(n, cfg.budget_permille, sink, local)
    index = torch.zeros((cfg.B, cfg.Hkv, x["K"].shape[2], 32), dtype=torch.bfloat16, device="cuda")
    qasc.ts_index_append(x["K"], x["W"], index, 0, n, Hq=cfg.Hq, n=n)
    sel = torch.empty((cfg.B, K), dtype=torch.int32, device="cuda")
    ws = qasc.alloc_workspace(qasc.ts_select_workspace_bytes(cfg.B, cfg.Hq, cfg.Hkv, n, x["K"].shape[2], K, sink,
                                                             local))
    qasc.ts_score_vote_select(x["q"], x["W"], index, sel, ws, n=n, K=K, sink=sink, local=local)
    qasc.qasc_device_error()
    s = sel.cpu()
    assert s.shape == (cfg.B, K) and bool((s[:, 1:] > s[:, :-1]).all())


# The attention kernel's roles, with a tile that never comes: whichever it is,
# the call returns with the error status and leaves nothing behind for the next
# one.  The schedules: shares and a merge (2 x 471 places over 152 blocks: three
# tiles of K and of V to each); whole items of two query tiles; of one, joined; in
# twos.
@pytest.mark.parametrize("Hq,Hkv,ql,lens,local", [
    (8, 2, [1], [60000], 1 << 30),
    (64, 8, [2048], [2100], 300),
    (16, 2, [300] * 6, [500] * 6, 90),
    (8, 8, [1] * 60, [700] * 60, 700),
])
def test_attention_returns_where_a_tile_never_comes(Hq, Hkv, ql, lens, local):
    B, T, n_cap = len(ql), sum(ql), max(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    q, K, V = rand(T, Hq, 128), rand(B, Hkv, n_cap, 128), rand(B, Hkv, n_cap, 128)
    cu = torch.tensor([sum(ql[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = qasc.alloc_workspace(qasc.kv_window_attn_workspace_bytes(T, B, Hq, Hkv, n_cap))
    want, out = torch.empty_like(q), torch.empty_like(q)
    kw = dict(local=local, cu_q=None if T == B else cu)
    qasc.kv_window_attn(q, K, V, ln, want, ws, **kw)
    qasc.qasc_device_error()
    for stall in (0, 1, 2, 3, 1 << 30):
        out.zero_()
        t0 = time.perf_counter()
        qasc.qasc_selftest_attn_wait(5000, stall, q, K, V, ln, out, ws, **kw)
        if stall < 1 << 30:
            with pytest.raises(qasc.QascError) as e:
                qasc.qasc_device_error()
            assert e.value.status == 5
            assert time.perf_counter() - t0 < 20.0
        else:
            qasc.qasc_device_error()
            assert torch.equal(out, want)
        out.zero_()
        qasc.kv_window_attn(q, K, V, ln, out, ws, **kw)
        qasc.qasc_device_error()
        assert torch.equal(out, want), "the call behind one without tile %d" % stall
