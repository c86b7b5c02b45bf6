"""Host-side checks of the packed-batch calls (kv_rope_append*,
kv_window_attn*, kv_prefix_attn_paged): argument validation of the C ABI and
of the Python binding.  CPU only (no kernel is launched)."""

import ctypes

import pytest
import torch

import query_aware_sparse_compressed_gb300 as qasc
from query_aware_sparse_compressed_gb300 import _lib
from query_aware_sparse_compressed_gb300 import build as qbuild

FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced
MISALIGNED = ctypes.c_void_p(0x10008)
bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
NO_DEVICE = not torch.cuda.is_available()


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
        self.q = self.k = self.v = self.q_out = self.K = self.V = self.out = self.ws = self.table0 = FAKE
        self.lse, self.ws_bytes = None, 1 << 40
        self.qs, self.ks, self.vs = 12 * 128, 12 * 128, 12 * 128
        self.sink, self.local, self.n_prefix = 4, 256, 100

    def append(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv_rope_append_paged if paged else lib.kv_rope_append
        return fn(ctypes.byref(self.s), *cache, ctypes.byref(self.b), ctypes.byref(self.r), self.q, self.qs, self.k,
                  self.ks, self.v, self.vs, self.q_out, self.K, self.V, None)

    def window(self, lib, paged=True):
        cache = (ctypes.byref(self.c),) if paged else ()
        fn = lib.kv_window_attn_paged if paged else lib.kv_window_attn
        return fn(ctypes.byref(self.s), *cache, ctypes.byref(self.b), self.sink, self.local, self.q, self.K, self.V,
                  self.out, self.lse, self.ws, self.ws_bytes, None)

    def prefix(self, lib):
        return lib.kv_prefix_attn_paged(ctypes.byref(self.s), ctypes.byref(self.c), self.table0, self.n_prefix,
                                        ctypes.byref(self.b), self.q, self.K, self.V, self.out, self.lse, self.ws,
                                        self.ws_bytes, None)


BATCH_RULES = [
    (lambda c: setattr(c.s, "d", 64), 2),
    (lambda c: setattr(c.s, "Hkv", 3), 1),
    (lambda c: setattr(c.s, "n_cap", 500), 1),          # n > n_cap
    (lambda c: setattr(c.b, "tokens", -1), 1),
    (lambda c: setattr(c.b, "tokens", 2 ** 31 // 8), 1),
    (lambda c: setattr(c.b, "tokens", 2 ** 62), 1),
    (lambda c: setattr(c.b, "lens", None), 1),
    (lambda c: setattr(c.b, "lens", 0x10002), 1),
    (lambda c: setattr(c.b, "cu_q", 0x10002), 1),
    (lambda c: setattr(c.b, "cu_q", None), 1),          # 10 tokens of 3 sequences
    (lambda c: setattr(c, "q", MISALIGNED), 1),
    (lambda c: setattr(c, "K", None), 1),
    (lambda c: setattr(c, "K", MISALIGNED), 1),
    (lambda c: setattr(c, "V", None), 1),
]


@pytest.mark.parametrize("mutate,code", BATCH_RULES)
def test_every_call_rejects_a_bad_batch(lib, mutate, code):
    for call in (lambda c: c.append(lib), lambda c: c.append(lib, False), lambda c: c.window(lib),
                 lambda c: c.window(lib, False), lambda c: c.prefix(lib)):
        c = Call()
        mutate(c)
        assert call(c) == code, lib.qasc_last_error()
        assert lib.qasc_last_error()


@pytest.mark.parametrize("mutate", [
    lambda c: setattr(c.r, "rot_dim", 129),
    lambda c: setattr(c.r, "rot_dim", 144),
    lambda c: setattr(c.r, "rot_dim", 8),
    lambda c: setattr(c.r, "rot_dim", -16),
    lambda c: setattr(c.r, "inv_freq", None),
    lambda c: setattr(c.r, "inv_freq", 0x10002),
    lambda c: setattr(c.r, "positions", 0x10002),
    lambda c: setattr(c, "qs", 12 * 128 + 4),
    lambda c: setattr(c, "ks", -8),
    lambda c: setattr(c, "vs", 2 ** 33),
    lambda c: setattr(c, "k", None),
    lambda c: setattr(c, "v", MISALIGNED),
    lambda c: setattr(c, "q_out", None),
    lambda c: setattr(c.c, "page_tokens", 96),
])
def test_append_rejects_bad_arguments(lib, mutate):
    c = Call()
    c.q_out = ctypes.c_void_p(0x20000)
    mutate(c)
    assert c.append(lib) == 1, lib.qasc_last_error()


def test_append_in_place_needs_dense_queries(lib):
    c = Call()
    assert c.append(lib) == 1 and b"dense" in lib.qasc_last_error()


@pytest.mark.parametrize("mutate,code", [
    (lambda c: setattr(c, "sink", -1), 1),
    (lambda c: setattr(c, "local", 0), 1),
    (lambda c: setattr(c, "q", None), 1),
    (lambda c: setattr(c, "out", None), 1),
    (lambda c: setattr(c, "out", MISALIGNED), 1),
    (lambda c: setattr(c, "lse", ctypes.c_void_p(0x10002)), 1),
    (lambda c: setattr(c, "ws", None), 3),
    (lambda c: setattr(c, "ws_bytes", 16), 3),
    (lambda c: setattr(c, "ws", ctypes.c_void_p(0x10010)), 1),
    (lambda c: (setattr(c.s, "B", 2049), setattr(c.s, "n", 64), setattr(c.s, "n_cap", 64),
                setattr(c.c, "pages_per_seq", 1)), 2),
])
def test_window_rejects_bad_arguments(lib, mutate, code):
    for paged in (True, False):
        c = Call()
        mutate(c)
        assert c.window(lib, paged) == code, lib.qasc_last_error()


@pytest.mark.parametrize("mutate,code", [
    (lambda c: setattr(c, "n_prefix", -1), 1),
    (lambda c: setattr(c, "n_prefix", 1 << 24), 1),
    (lambda c: setattr(c, "table0", None), 1),
    (lambda c: setattr(c, "table0", ctypes.c_void_p(0x10002)), 1),
    (lambda c: setattr(c, "ws_bytes", 16), 3),
    (lambda c: setattr(c.c, "num_pages", 0), 1),
])
def test_prefix_rejects_bad_arguments(lib, mutate, code):
    c = Call()
    mutate(c)
    assert c.prefix(lib) == code, lib.qasc_last_error()


def test_null_structures_are_rejected(lib):
    c = Call()
    assert lib.kv_window_attn(ctypes.byref(c.s), None, 4, 256, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 40, None) == 1
    assert lib.kv_rope_append(ctypes.byref(c.s), ctypes.byref(c.b), None, None, 0, FAKE, 256, FAKE, 256, None, FAKE,
                              FAKE, None) == 1
    assert lib.kv_prefix_attn_paged(ctypes.byref(c.s), None, FAKE, 10, ctypes.byref(c.b), FAKE, FAKE, FAKE, FAKE,
                                    None, FAKE, 1 << 40, None) == 1


def test_an_empty_batch_is_a_no_op(lib):
    c = Call()
    c.b.tokens = 0
    c.q = c.k = c.v = c.q_out = c.out = c.ws = None
    assert c.append(lib) == 0 and c.window(lib) == 0 and c.prefix(lib) == 0


@pytest.mark.skipif(not NO_DEVICE, reason="fake pointers must not reach a kernel")
def test_valid_calls_stop_at_the_missing_device(lib):
    c = Call()
    c.q_out = ctypes.c_void_p(0x20000)
    assert c.append(lib) == 4 and c.append(lib, False) == 4
    c.q = None                                   # keys and values only
    assert c.append(lib) == 4
    c = Call()
    assert c.window(lib) == 4 and c.window(lib, False) == 4 and c.prefix(lib) == 4
    c.n_prefix, c.table0 = 0, None
    assert c.prefix(lib) == 4
    c.r.rot_dim, c.r.inv_freq, c.q_out = 0, None, ctypes.c_void_p(0x20000)
    assert c.append(lib) == 4


def test_workspace_queries(lib):
    c = Call()
    for fn in (lib.kv_window_attn_workspace_bytes, lib.kv_prefix_attn_workspace_bytes):
        assert fn(ctypes.byref(c.s), 10) >= 256
        assert fn(ctypes.byref(c.s), -1) == 0 and lib.qasc_last_error()
        assert fn(None, 10) == 0 and lib.qasc_last_error()
        assert fn(ctypes.byref(c.s), 0) > 0
    big = _lib.qasc_shape(2049, 1, 1, 128, 32, 0, 64, 64)
    assert lib.kv_window_attn_workspace_bytes(ctypes.byref(big), 2049) == 0
    with pytest.raises(qasc.QascError):
        qasc.kv_window_attn_workspace_bytes(-1, 1, 8, 2, 512)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (32, 8), (8, 2), (24, 3), (64, 64), (1, 1), (8, 1)])
def test_workspace_does_not_fall_with_tokens_or_sequences(lib, Hq, Hkv):
    # an engine allocates for its largest batch and calls with smaller ones
    names = "kv_window_attn_workspace_bytes", "kv_prefix_attn_workspace_bytes"
    tokens = sorted({max(0, t + d) for t in [int(1.2 ** i) for i in range(80)] + [2 ** i for i in range(22)]
                     for d in (-1, 0, 1)})
    sized = {}
    for B in (1, 2, 7, 300, 2048 if Hkv < 64 else 1000):
        s = _lib.qasc_shape(B, Hq, Hkv, 128, 32, 0, 64, 64)
        for name in names:
            sizes = [getattr(lib, name)(ctypes.byref(s), t) for t in tokens]
            assert all(x > 0 for x in sizes) and sizes == sorted(sizes)
            assert all(x >= y for x, y in zip(sizes, sized.get(name, sizes)))
            sized[name] = sizes
        assert all(x >= y for x, y in zip(sized[names[1]], sized[names[0]]))


def test_selftest_of_the_attention_rejects_bad_limits(lib):
    c = Call()
    call = lambda limit, stall: lib.qasc_selftest_attn_wait(limit, stall, ctypes.byref(c.s), ctypes.byref(c.b), 4, 256,
                                                            FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 40, None)
    assert call(0, 0) == 1 and call(-5, 0) == 1 and call(2000001, 0) == 1 and call(1000, -1) == 1
    c.s.n_cap = 0
    assert call(1000, 0) == 1


def t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    # V pool of another page count
    lambda: qasc.kv_window_attn_paged(t(4, 8, 128), t(9, 2, 64, 128), t(8, 2, 64, 128), t(4, 3, dtype=i32),
                                      t(4, dtype=i32), t(4, 8, 128), t(256, dtype=u8), local=10),
    # block_table of another batch
    lambda: qasc.kv_window_attn_paged(t(4, 8, 128), t(9, 2, 64, 128), t(9, 2, 64, 128), t(3, 3, dtype=i32),
                                      t(4, dtype=i32), t(4, 8, 128), t(256, dtype=u8), local=10),
    # head dimension
    lambda: qasc.kv_window_attn(t(4, 8, 64), t(4, 2, 64, 128), t(4, 2, 64, 128), t(4, dtype=i32), t(4, 8, 128),
                                t(256, dtype=u8), local=10),
    # k not [T, Hkv, d]
    lambda: qasc.kv_rope_append(None, t(4, 2, 64), t(4, 2, 128), None, t(4, 2, 64, 128), t(4, 2, 64, 128),
                                t(4, dtype=i32), None),
    # a block table of one dimension, or none
    lambda: qasc.kv_window_attn_paged(t(4, 8, 128), t(9, 2, 64, 128), t(9, 2, 64, 128), t(4, dtype=i32),
                                      t(4, dtype=i32), t(4, 8, 128), t(256, dtype=u8), local=10),
    # cu_q of another batch
    lambda: qasc.kv_window_attn(t(4, 8, 128), t(2, 2, 64, 128), t(2, 2, 64, 128), t(2, dtype=i32), t(4, 8, 128),
                                t(256, dtype=u8), local=10, cu_q=t(4, dtype=i32)),
    # prefix pages
    lambda: qasc.kv_prefix_attn_paged(t(4, 8, 128), t(9, 2, 64, 128), t(9, 2, 64, 128), t(1, dtype=i32),
                                      t(4, 3, dtype=i32), t(4, dtype=i32), t(4, 8, 128), t(256, dtype=u8),
                                      n_prefix=65),
    # positions of another batch
    lambda: qasc.kv_rope_append(None, t(4, 2, 128), t(4, 2, 128), None, t(4, 2, 64, 128), t(4, 2, 64, 128),
                                t(4, dtype=i32), None, positions=t(3, dtype=i32)),
])
def test_wrong_extents_are_rejected_before_the_library(call):
    with pytest.raises(ValueError, match="must have shape|must be a CUDA tensor"):
        call()


def test_tensors_on_the_host_are_rejected(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qasc.kv_window_attn(t(4, 8, 128), t(4, 2, 64, 128), t(4, 2, 64, 128), t(4, dtype=i32), t(4, 8, 128),
                            t(256, dtype=u8), local=10)
    with pytest.raises(ValueError, match="must have shape"):
        qasc._heads(t(3, 2, 128), "k", 4, 2, -1)
    with pytest.raises(ValueError, match="contiguous within a token"):
        qasc._heads(t(4, 128, 2).transpose(1, 2), "k", 4, 2, -1)
    with pytest.raises(ValueError, match="must have shape"):
        qasc._at(t(4, 8, 128), "out", bf, (4, 8, 64), -1)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        qasc._at(t(4, 8, 128), "out", bf, (4, 8, 128), 0)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        qasc._at([1, 2], "out", bf, (2,), 0)


@pytest.mark.parametrize("given,sent", [(0, 0), (4, 4), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                        (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1), (-3, -3), (-2 ** 40, -1)])
def test_sink_and_local_beyond_32_bits_keep_their_meaning(lib, monkeypatch, given, sent):
    # the library takes 32 bits, to which ctypes cuts without a word: 2^32 + 5 would be 5
    calls = []
    monkeypatch.setattr(qasc, "_run", lambda fn, dev, stream, shape, cache, *args: calls.append(args))
    args = (t(2, 8, 128), t(2, 2, 64, 128), t(2, 2, 64, 128), t(2, dtype=i32), t(2, 8, 128), t(256, dtype=u8))
    qasc.kv_window_attn(*args, local=given, sink=given)
    args = (t(2, 8, 128), t(9, 2, 64, 128), t(9, 2, 64, 128), t(2, 3, dtype=i32), t(2, dtype=i32), t(2, 8, 128),
            t(256, dtype=u8))
    qasc.kv_window_attn_paged(*args, local=given, sink=given)
    for sink, local in (c[1:3] for c in calls):
        assert sink == local == sent and ctypes.c_int32(sink).value == sink
    assert len(calls) == 2


def test_packed_descriptors_equal_the_structures():
    big = 1 << 40
    assert _lib.pack_shape(3, 8, 2, 128, 32, 0, big, big + 1) == bytes(_lib.qasc_shape(3, 8, 2, 128, 32, 0, big, big + 1))
    assert _lib.pack_cache(big, 64, 8, big) == bytes(_lib.qasc_paged_cache(big, 64, 8, big))
    assert _lib.pack_batch(0, big, 10) == bytes(_lib.qasc_batch(None, big, 10))
    assert _lib.pack_rope(big, 0, 128, 1) == bytes(_lib.qasc_rope(big, None, 128, 1))
