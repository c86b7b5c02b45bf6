"""Host-side checks of the 4-bit cache's calls (kv4_*): argument validation of the C
ABI and of the Python binding.  CPU only (no kernel is launched)."""

import ctypes

import pytest
import torch

import query_aware_sparse_compressed_gb300 as qasc
from query_aware_sparse_compressed_gb300 import _lib
from query_aware_sparse_compressed_gb300 import build as qbuild

FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced
MISALIGNED = ctypes.c_void_p(0x10008)
bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return _lib.load()


class Call:
    """The arguments of one call of each kind, valid unless changed."""

    def __init__(self):
        self.s = _lib.qasc_shape(3, 8, 2, 128, 32, 0, 512, 512)
        self.c = _lib.qasc_paged_cache(FAKE.value, 64, 8, 40)
        self.b = _lib.qasc_batch(FAKE.value, FAKE.value, 10)
        self.r = _lib.qasc_rope(FAKE.value, None, 128, 0)
        self.p = _lib.qasc_ts_params(100, 4, 256, 1)
        self.kv = _lib.qasc_kv4(FAKE.value, FAKE.value, FAKE.value, FAKE.value, 1.0, 0.5)
        self.q = self.k = self.v = self.K_out = self.V_out = self.out = self.ws = self.sel = FAKE
        self.q_out = ctypes.c_void_p(0x20000)
        self.lse, self.sel_len, self.ws_bytes = None, None, 1 << 40
        self.qs, self.ks, self.vs = 12 * 128, 12 * 128, 12 * 128
        self.kt, self.kh, self.vt, self.vh = 256, 128, 256, 128
        self.sink, self.local, self.max_q = 4, 256, 5

    def append(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv4_rope_append_paged if paged else lib.kv4_rope_append
        return fn(ctypes.byref(self.s), *cache, ctypes.byref(self.b), ctypes.byref(self.r), self.q, self.qs, self.k,
                  self.ks, self.v, self.vs, self.q_out, ctypes.byref(self.kv) if self.kv else None, None)

    def read(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv4_read_paged if paged else lib.kv4_read
        return fn(ctypes.byref(self.s), *cache, ctypes.byref(self.b), ctypes.byref(self.kv) if self.kv else None,
                  self.K_out, self.kt, self.kh, self.V_out, self.vt, self.vh, None)

    def window(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv4_window_attn_paged if paged else lib.kv4_window_attn
        return fn(ctypes.byref(self.s), *cache, ctypes.byref(self.b), self.max_q, self.sink, self.local, self.q,
                  ctypes.byref(self.kv) if self.kv else None, self.out, self.lse, self.ws, self.ws_bytes, None)

    def sparse(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv4_sparse_attn_paged if paged else lib.kv4_sparse_attn
        return fn(ctypes.byref(self.s), ctypes.byref(self.p), *cache, self.q,
                  ctypes.byref(self.kv) if self.kv else None, self.sel, self.sel_len, 0, self.out, self.lse, self.ws,
                  self.ws_bytes, None)


ALL = [lambda c, lib, i=i, paged=paged: getattr(c, i)(lib, paged) for i in ("append", "read", "window", "sparse")
       for paged in (True, False)]
BATCHED = ALL[:6]


@pytest.mark.parametrize("mutate,code", [
    (lambda c: setattr(c.s, "d", 64), 2),
    (lambda c: setattr(c.s, "Hkv", 3), 1),
    (lambda c: setattr(c.s, "n_cap", 500), 1),          # n > n_cap
    (lambda c: setattr(c, "kv", None), 1),
    (lambda c: setattr(c.kv, "K", None), 1),
    (lambda c: setattr(c.kv, "K", 0x10008), 1),
    (lambda c: setattr(c.kv, "K_sf", None), 1),
    (lambda c: setattr(c.kv, "K_sf", 0x10008), 1),
    (lambda c: setattr(c.kv, "V", 0x10001), 1),
    (lambda c: setattr(c.kv, "V_sf", None), 1),
    (lambda c: setattr(c.kv, "k_scale", 0.0), 1),
    (lambda c: setattr(c.kv, "k_scale", -1.0), 1),
    (lambda c: setattr(c.kv, "k_scale", 3.0), 1),
    (lambda c: setattr(c.kv, "k_scale", 2.0 ** 33), 1),
    (lambda c: setattr(c.kv, "v_scale", 2.0 ** -33), 1),
    (lambda c: setattr(c.kv, "v_scale", float("nan")), 1),
    (lambda c: setattr(c.kv, "v_scale", float("inf")), 1),
])
def test_every_call_rejects_a_bad_cache(lib, mutate, code):
    for call in ALL:
        c = Call()
        mutate(c)
        assert call(c, lib) == code, lib.qasc_last_error()
        assert lib.qasc_last_error()


@pytest.mark.parametrize("mutate,code", [
    (lambda c: setattr(c.b, "tokens", -1), 1),
    (lambda c: setattr(c.b, "tokens", 2 ** 31 // 8), 1),
    (lambda c: setattr(c.b, "lens", None), 1),
    (lambda c: setattr(c.b, "lens", 0x10002), 1),
    (lambda c: setattr(c.b, "cu_q", 0x10002), 1),
    (lambda c: setattr(c.b, "cu_q", None), 1),          # 10 tokens of 3 sequences
])
def test_batched_calls_reject_a_bad_batch(lib, mutate, code):
    for call in BATCHED:
        c = Call()
        mutate(c)
        assert call(c, lib) == code, lib.qasc_last_error()


@pytest.mark.parametrize("mutate", [
    lambda c: setattr(c.r, "rot_dim", 129),
    lambda c: setattr(c.r, "rot_dim", 144),
    lambda c: setattr(c.r, "rot_dim", -16),
    lambda c: setattr(c.r, "inv_freq", None),
    lambda c: setattr(c.r, "positions", 0x10002),
    lambda c: setattr(c, "qs", 12 * 128 + 4),
    lambda c: setattr(c, "ks", -8),
    lambda c: setattr(c, "vs", 2 ** 33),
    lambda c: setattr(c, "q", MISALIGNED),
    lambda c: setattr(c, "k", None),
    lambda c: setattr(c, "v", MISALIGNED),
    lambda c: setattr(c, "q_out", None),
    lambda c: setattr(c, "q_out", FAKE),                # in place, and q is not dense
    lambda c: setattr(c.c, "page_tokens", 96),
])
def test_append_rejects_bad_arguments(lib, mutate):
    c = Call()
    mutate(c)
    assert c.append(lib) == 1, lib.qasc_last_error()


@pytest.mark.parametrize("mutate", [
    lambda c: setattr(c, "K_out", None),
    lambda c: setattr(c, "V_out", MISALIGNED),
    lambda c: setattr(c, "kt", 132),
    lambda c: setattr(c, "kh", -8),
    lambda c: setattr(c, "vt", 2 ** 32),
    lambda c: setattr(c, "vh", 129),
])
def test_read_rejects_bad_arguments(lib, mutate):
    for paged in (True, False):
        c = Call()
        mutate(c)
        assert c.read(lib, paged) == 1, lib.qasc_last_error()


ATTENTION = [
    (lambda c: setattr(c, "q", None), 1),
    (lambda c: setattr(c, "out", None), 1),
    (lambda c: setattr(c, "out", MISALIGNED), 1),
    (lambda c: setattr(c, "lse", ctypes.c_void_p(0x10002)), 1),
    (lambda c: setattr(c, "ws", None), 3),
    (lambda c: setattr(c, "ws_bytes", 16), 3),
    (lambda c: setattr(c, "ws", ctypes.c_void_p(0x10010)), 1),
    (lambda c: (setattr(c.s, "B", 2049), setattr(c.s, "n", 64), setattr(c.s, "n_cap", 64), setattr(c.p, "K", 0),
                setattr(c.c, "pages_per_seq", 1)), 2),
]


@pytest.mark.parametrize("mutate,code", ATTENTION + [
    (lambda c: setattr(c, "sink", -1), 1),
    (lambda c: setattr(c, "local", 0), 1),
    (lambda c: setattr(c, "max_q", -1), 1),
    (lambda c: setattr(c, "max_q", 11), 1),             # of 10 tokens
])
def test_window_rejects_bad_arguments(lib, mutate, code):
    for paged in (True, False):
        c = Call()
        mutate(c)
        assert c.window(lib, paged) == code, lib.qasc_last_error()


@pytest.mark.parametrize("mutate,code", ATTENTION + [
    (lambda c: setattr(c.p, "K", 253), 1),              # more than the candidates
    (lambda c: setattr(c.p, "sink", -1), 1),
    (lambda c: setattr(c, "sel", None), 1),
    (lambda c: setattr(c, "sel", ctypes.c_void_p(0x10002)), 1),
    (lambda c: setattr(c, "sel_len", ctypes.c_void_p(0x10002)), 1),
])
def test_sparse_rejects_bad_arguments(lib, mutate, code):
    for paged in (True, False):
        c = Call()
        mutate(c)
        assert c.sparse(lib, paged) == code, lib.qasc_last_error()


def test_sizes_follow_the_calls_rules():
    ok = dict(T=10, B=3, Hq=8, Hkv=2, n_cap=512, local=256, sink=4, max_q=5)
    assert qasc.kv4_window_attn_workspace_bytes(**ok) > 0
    for bad in (dict(local=0), dict(sink=-1), dict(max_q=11), dict(T=-1), dict(Hkv=3), dict(B=2049), dict(n_cap=0)):
        with pytest.raises(qasc.QascError):
            qasc.kv4_window_attn_workspace_bytes(**{**ok, **bad})
    assert qasc.kv4_sparse_attn_workspace_bytes(3, 8, 2, 512, 512, 100) > 0
    for bad in (dict(K=253), dict(n=513), dict(sink=-1)):
        with pytest.raises(qasc.QascError):
            qasc.kv4_sparse_attn_workspace_bytes(**{**dict(B=3, Hq=8, Hkv=2, n=512, n_cap=512, K=100), **bad})


SHAPES = [   # B, Hq, Hkv, n_cap, local
    (2, 8, 8, 8192, 256), (16, 32, 8, 131072, 4096), (1, 64, 8, 32768, 32768), (64, 64, 8, 131072, 131072),
    (7, 8, 2, 5000, 1000), (3, 8, 1, 300, 1), (2048, 64, 8, 131071, 131071), (1, 8, 8, (1 << 24) - 1, 1 << 24),
]


@pytest.mark.parametrize("B,Hq,Hkv,n_cap,local", SHAPES)
def test_window_size_does_not_fall_with_a_larger_call(lib, B, Hq, Hkv, n_cap, local):
    steps = [1, 2, 16, 17, 18, 33, 53, 64, 65, 96, 100, 103, 128, 129, 130, 200, 257, 1000, 1941, 4181, 6502, 6602, 20000, 32768]

    def size(T, m, b=B):
        return qasc.kv4_window_attn_workspace_bytes(T, b, Hq, Hkv, n_cap, local=local, max_q=m)
    least = size(1, 1)
    below = {}
    for T in steps:
        for m in [m for m in steps if m <= T]:
            got = size(T, m)
            assert got >= least and got >= max((below[k] for k in below if k[0] <= T and k[1] <= m), default=0)
            assert got >= size(T, m, max(1, B // 2)) and got <= (5 << 30)
            below[T, m] = got
    assert len(set(below.values())) > 1 or local == 1


def test_window_sizes_of_calls_that_do_and_do_not_copy():
    """Where the rule for a copy goes back and forth: T, max_q of a call and of a smaller one."""
    for (B, Hq, Hkv, n_cap, local), (T, m), (T1, m1) in (
            ((2, 8, 8, 8192, 256), (6502, 4181), (6502, 1941)), ((2, 8, 8, 8192, 256), (6602, 6602), (6502, 1941)),
            ((16, 32, 8, 131072, 4096), (103, 53), (96, 53))):
        big, small = (qasc.kv4_window_attn_workspace_bytes(t, B, Hq, Hkv, n_cap, local=local, max_q=q) for t, q in ((T, m), (T1, m1)))
        assert big >= small > 50e6


@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_sparse_sink_and_local_of_any_number(monkeypatch, far):
    """More tokens than 32 bits hold mean all of them, as in the window calls; negative ones are refused."""
    assert qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, 512, 512, 0, sink=far) > 0
    assert qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, 512, 512, 0, local=far) > 0
    kv = qasc.alloc_kv4(1, 2, 64, device="cpu")
    q, ws = torch.zeros((1, 8, 128), dtype=bf), torch.zeros(1024, dtype=u8)
    passed = []
    monkeypatch.setattr(qasc, "_run", lambda fn, dev, stream, shape, cache, params, *rest: passed.append(params))
    for kw in (dict(sink=far, local=far), dict(sink=-far, local=4), dict(sink=4, local=-far)):
        qasc.kv4_sparse_attn(q, kv, None, q, ws, n=10, **kw)
    got = [_lib.qasc_ts_params.from_buffer_copy(p) for p in passed]
    assert (got[0].sink, got[0].local) == (2 ** 31 - 1, 2 ** 31 - 1) and got[1].sink < 0 and got[2].local < 0
    for bad in (dict(sink=-far), dict(local=-far)):
        with pytest.raises(qasc.QascError):
            qasc.kv4_sparse_attn_workspace_bytes(1, 8, 2, 512, 512, 0, **bad)


def test_no_tokens_is_no_call(lib):
    c = Call()
    c.b.tokens, c.max_q = 0, 0
    c.q = c.k = c.v = c.out = c.K_out = c.V_out = c.ws = None
    for call in BATCHED:
        assert call(c, lib) == 0, lib.qasc_last_error()


def test_binding_checks_the_cache():
    kv = qasc.alloc_kv4(3, 2, 64, device="cpu")
    assert kv.K.shape == (3, 2, 64, 64) and kv.V_sf.shape == (3, 2, 64, 8) and kv.K_sf.dtype is torch.float8_e4m3fn
    lens = torch.ones(3, dtype=i32)
    k = torch.zeros((3, 2, 128), dtype=bf)
    q = torch.zeros((3, 8, 128), dtype=bf)
    ws = torch.zeros(1024, dtype=u8)
    table = torch.zeros((3, 1), dtype=i32)
    for call in (lambda kv: qasc.kv4_rope_append(q, k, k, q, kv, lens, None), lambda kv: qasc.kv4_read(kv, lens, k, k),
                 lambda kv: qasc.kv4_window_attn(q, kv, lens, q, ws, local=4),
                 lambda kv: qasc.kv4_sparse_attn(q, kv, None, q, ws, n=10),
                 lambda kv: qasc.kv4_read_paged(kv, table, lens, k, k)):
        with pytest.raises(ValueError, match="CUDA"):
            call(kv)                                     # all is well but the device
        with pytest.raises(TypeError):
            call(tuple(kv))
        for bad in (dict(K=kv.K[..., :32]), dict(K=kv.K[0]), dict(V=kv.V[:, :1]), dict(K_sf=kv.K_sf.view(u8)),
                    dict(K=kv.K.float()), dict(V_sf=kv.K_sf[:, :, ::2]), dict(K=None), dict(V=3)):
            with pytest.raises((ValueError, TypeError)):
                call(qasc.KV4(**{**dict(zip(("K", "K_sf", "V", "V_sf"), kv)), **bad}))
    with pytest.raises(AttributeError):
        kv.K = kv.V
    with pytest.raises(ValueError, match="block_table"):
        qasc.kv4_read_paged(kv, torch.zeros((2, 1), dtype=i32), lens, k, k)


def test_binding_refuses_outputs_whose_rows_overlap():
    kv = qasc.alloc_kv4(1, 2, 64, device="cpu")
    lens = torch.tensor([5], dtype=i32)
    cu = torch.tensor([0, 5], dtype=i32)
    good = torch.zeros((1, 2, 64, 128), dtype=bf)[0].transpose(0, 1)[:5]
    flat = torch.zeros(1 << 16, dtype=bf)
    for bad in (flat.as_strided((5, 2, 128), (64, 8192, 1)), flat.as_strided((5, 2, 128), (128, 256, 1)),
                flat.as_strided((5, 2, 128), (0, 128, 1)), flat.as_strided((5, 2, 128), (512, 256, 2))):
        for pair in ((bad, good), (good, bad)):
            with pytest.raises(ValueError, match="overlap|contiguous"):
                qasc.kv4_read(kv, lens, *pair, cu_q=cu)
    with pytest.raises(ValueError, match="CUDA"):
        qasc.kv4_read(kv, lens, good, good, cu_q=cu)
