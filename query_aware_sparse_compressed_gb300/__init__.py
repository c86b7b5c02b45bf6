"""Query-aware sparse KV selection and attention on GB300 (sm_103a).

Thin Python binding over the C ABI of libqasc (include/qasc.h): every call
checks and marshals torch tensors (device memory) into pointers and sizes and
enqueues the library's CUDA kernels on the current (or given) stream.  No step
of the computation runs in Python or PyTorch; if the library is missing the
calls raise.

Entry points keep the C names:
  ts_index_append, ts_select_workspace_bytes, ts_score_vote_select,
  ts_attn_workspace_bytes, ts_sparse_attn, ts_sparse_attn_noalloc,
  ts_head_select_workspace_bytes, ts_score_select_per_head,
  ts_sparse_attn_per_head, ts_expand_capacity, ts_expand_workspace_bytes,
  ts_expand_neighbors, ts_sparse_attn_ex, ts_index_append_paged,
  ts_score_vote_select_paged, ts_score_select_per_head_paged,
  ts_sparse_attn_paged, ts_ring_flush,
  kv_rope_append, kv_rope_append_paged,
  kv_window_attn_workspace_bytes, kv_window_attn, kv_window_attn_paged,
  kv_prefix_attn_workspace_bytes, kv_prefix_attn_paged,
  KV4, alloc_kv4, kv4_rope_append, kv4_rope_append_paged, kv4_read,
  kv4_read_paged, kv4_window_attn_workspace_bytes, kv4_window_attn,
  kv4_window_attn_paged, kv4_sparse_attn_workspace_bytes, kv4_sparse_attn,
  kv4_sparse_attn_paged,
  ts_dense_attn_workspace_bytes, ts_dense_attn, snapkv_workspace_bytes,
  snapkv_compress, qasc_status_string, qasc_last_error, qasc_last_cuda_error, qasc_device_error,
  qasc_selftest_bounded_wait, qasc_selftest_attn_wait, qasc_version.
"""

import ctypes

import torch

from . import _lib

D = 128
D_IDX = 32


class QascError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__("%s: %s" % (_lib.STATUS_NAMES.get(status, str(status)), message))


def _L():
    return _lib.load()


def _check(status):
    if status != _lib.QASC_OK:
        msg = _L().qasc_last_error()
        raise QascError(status, msg.decode() if msg else "")


def _sized(nbytes):
    """A size query's answer; 0 with a message means the library rejected
    the arguments (the same checks as the call being sized)."""
    if nbytes == 0:
        msg = _L().qasc_last_error()
        if msg:
            raise QascError(_lib.QASC_ERR_INVALID_ARG, msg.decode())
    return int(nbytes)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t, name, dtype):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.device.index != torch.cuda.current_device():
        # The library launches on the current device; another GPU's memory
        # would be dereferenced by its kernels.
        raise ValueError("%s is on %s but the current device is cuda:%d" % (name, t.device,
                                                                             torch.cuda.current_device()))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _dims(t, name, dims):
    """Raise unless tensor t (None passes) has these dimensions (None = any).
    The library sees only pointers, so every extent is checked here."""
    if t is None:
        return
    got = tuple(t.shape)
    if len(got) != len(dims) or any(d is not None and g != d for g, d in zip(got, dims)):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple("*" if d is None else d for d in dims), got))


def make_shape(B, Hq, Hkv, n, n_cap):
    return _lib.qasc_shape(B, Hq, Hkv, D, D_IDX, 0, n, n_cap)


def ts_params(K, sink=4, local=256, vmin=1):
    return _lib.qasc_ts_params(K, sink, local, vmin)


def snap_params(c, window=32, pool_k=3):
    return _lib.qasc_snap_params(c, window, pool_k, 0)


def budget_tokens(n, budget_permille, sink=4, local=256):
    """K = min(floor(budget * n), |C|) with the floor taken in integers."""
    c1 = max(n - local, sink)
    return min((budget_permille * n) // 1000, c1 - sink)


def alloc_workspace(nbytes, device=None):
    """Caller-owned workspace (uint8) of at least nbytes, 256-byte aligned."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ TokenSelect
def ts_index_append(K, W, index, start, count, *, Hq=None, n=None, stream=None):
    """index[b, g, start:start+count] = RNE_bf16(K[b, g, rows] @ W[g])."""
    _dims(K, "K", (None, None, None, D))
    B, Hkv, n_cap, _ = K.shape
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(index, "index", (B, Hkv, n_cap, D_IDX))
    shape = make_shape(B, Hq or Hkv, Hkv, n or n_cap, n_cap)
    _check(_L().ts_index_append(ctypes.byref(shape), _ptr(K, "K", torch.bfloat16), _ptr(W, "W", torch.bfloat16),
                                _ptr(index, "index", torch.bfloat16), int(start), int(count), _stream(stream)))


def ts_select_workspace_bytes(B, Hq, Hkv, n, n_cap, K, sink=4, local=256, vmin=1):
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(K, sink, local, vmin)
    return _sized(_L().ts_select_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def ts_score_vote_select(q, W, index, sel, workspace, *, n, K, sink=4, local=256, vmin=1, stream=None):
    """sel[b, :K] = the selected candidate tokens of sequence b, ascending."""
    _dims(q, "q", (None, None, D))
    B, Hq, _ = q.shape
    _dims(index, "index", (B, None, None, D_IDX))
    _, Hkv, n_cap, _ = index.shape
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(sel, "sel", (B, K))
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(K, sink, local, vmin)
    _check(_L().ts_score_vote_select(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                                     _ptr(W, "W", torch.bfloat16), _ptr(index, "index", torch.bfloat16),
                                     _ptr(sel, "sel", torch.int32), _ptr(workspace, "workspace", torch.uint8),
                                     workspace.numel(), _stream(stream)))


def _attn_dims(q, K, V, out, lse):
    _dims(q, "q", (None, None, D))
    B, Hq, _ = q.shape
    _dims(K, "K", (B, None, None, D))
    _, Hkv, n_cap, _ = K.shape
    _dims(V, "V", (B, Hkv, n_cap, D))
    _dims(out, "out", (B, Hq, D))
    _dims(lse, "lse", (B, Hq))
    return B, Hq, Hkv, n_cap


def ts_attn_workspace_bytes(B, Hq, Hkv, n, n_cap, K, sink=4, local=256):
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(K, sink, local, 1)
    return _sized(_L().ts_attn_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def ts_sparse_attn(q, K, V, sel, out, workspace, *, n, sink=4, local=256, lse=None, stream=None):
    """out[b, h] = attention of q[b, h] over sink + sel[b] + local tokens."""
    B, Hq, Hkv, n_cap = _attn_dims(q, K, V, out, lse)
    _dims(sel, "sel", (B, None))
    Ksel = sel.shape[1] if sel is not None else 0
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(Ksel, sink, local, 1)
    _check(_L().ts_sparse_attn(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                               _ptr(K, "K", torch.bfloat16), _ptr(V, "V", torch.bfloat16),
                               _ptr(sel, "sel", torch.int32) if Ksel else None,
                               _ptr(out, "out", torch.float32), _ptr(lse, "lse", torch.float32),
                               _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def ts_head_select_workspace_bytes(B, Hq, Hkv, n, n_cap, K, sink=4, local=256):
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(K, sink, local, 1)
    return _sized(_L().ts_head_select_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def ts_score_select_per_head(q, W, index, sel, workspace, *, n, K, sink=4, local=256, stream=None):
    """sel[b, g, :K] = the candidates with the K largest group-summed scores
    of KV head g, ascending (selection without voting)."""
    _dims(q, "q", (None, None, D))
    B, Hq, _ = q.shape
    _dims(index, "index", (B, None, None, D_IDX))
    _, Hkv, n_cap, _ = index.shape
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(sel, "sel", (B, Hkv, K))
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(K, sink, local, 1)
    _check(_L().ts_score_select_per_head(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                                         _ptr(W, "W", torch.bfloat16), _ptr(index, "index", torch.bfloat16),
                                         _ptr(sel, "sel", torch.int32), _ptr(workspace, "workspace", torch.uint8),
                                         workspace.numel(), _stream(stream)))


def ts_sparse_attn_per_head(q, K, V, sel, out, workspace, *, n, sink=4, local=256, lse=None, stream=None):
    """out[b, h] = attention of q[b, h] over sink + sel[b, g(h)] + local tokens."""
    B, Hq, Hkv, n_cap = _attn_dims(q, K, V, out, lse)
    _dims(sel, "sel", (B, Hkv, None))
    Ksel = sel.shape[2] if sel is not None else 0
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(Ksel, sink, local, 1)
    _check(_L().ts_sparse_attn_per_head(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                                        _ptr(K, "K", torch.bfloat16), _ptr(V, "V", torch.bfloat16),
                                        _ptr(sel, "sel", torch.int32) if Ksel else None,
                                        _ptr(out, "out", torch.float32), _ptr(lse, "lse", torch.float32),
                                        _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                        _stream(stream)))


def ts_expand_capacity(n, K, radius, sink=4, local=256, n_cap=None, B=1, Hq=1, Hkv=1):
    shape = make_shape(B, Hq, Hkv, n, n_cap or n)
    params = ts_params(K, sink, local, 1)
    return _sized(_L().ts_expand_capacity(ctypes.byref(shape), ctypes.byref(params), radius))


def ts_expand_workspace_bytes(n, K, rows, sink=4, local=256):
    shape = make_shape(1, 1, 1, n, n)
    params = ts_params(K, sink, local, 1)
    return _sized(_L().ts_expand_workspace_bytes(ctypes.byref(shape), ctypes.byref(params), rows))


def ts_expand_neighbors(sel, radius, sel_out, lengths, workspace, *, n, sink=4, local=256, stream=None):
    """sel_out[r, :lengths[r]] = ascending union of [j - radius, j + radius]
    over j in sel[r], within the candidates; sel is [rows, K] (or [B, Hkv, K],
    flattened to rows)."""
    lead = tuple(sel_out.shape[:-1])
    if tuple(sel.shape[:-1]) != lead or tuple(lengths.shape) != lead:
        raise ValueError("sel %s, sel_out %s and lengths %s must share their leading dimensions"
                         % (tuple(sel.shape), tuple(sel_out.shape), tuple(lengths.shape)))
    rows = sel_out.numel() // sel_out.shape[-1]
    K = sel.shape[-1]
    shape = make_shape(1, 1, 1, n, n)
    params = ts_params(K, sink, local, 1)
    _check(_L().ts_expand_neighbors(ctypes.byref(shape), ctypes.byref(params), rows,
                                    _ptr(sel, "sel", torch.int32) if K else None, radius,
                                    _ptr(sel_out, "sel_out", torch.int32), sel_out.shape[-1],
                                    _ptr(lengths, "lengths", torch.int32),
                                    _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                    _stream(stream)))


def ts_sparse_attn_ex(q, K, V, sel, out, workspace, *, n, sink=4, local=256, lengths=None, per_kv_head=False,
                      lse=None, stream=None):
    """Attention over sink + sel[b] (or sel[b, g(h)] when per_kv_head) + local,
    using only the first lengths[...] entries of each list when given."""
    B, Hq, Hkv, n_cap = _attn_dims(q, K, V, out, lse)
    _dims(sel, "sel", (B, Hkv, None) if per_kv_head else (B, None))
    _dims(lengths, "lengths", (B, Hkv) if per_kv_head else (B,))
    Ksel = sel.shape[-1] if sel is not None else 0
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(Ksel, sink, local, 1)
    _check(_L().ts_sparse_attn_ex(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                                  _ptr(K, "K", torch.bfloat16), _ptr(V, "V", torch.bfloat16),
                                  _ptr(sel, "sel", torch.int32) if Ksel else None,
                                  _ptr(lengths, "lengths", torch.int32), 1 if per_kv_head else 0,
                                  _ptr(out, "out", torch.float32), _ptr(lse, "lse", torch.float32),
                                  _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def paged_cache(block_table, page_tokens, num_pages):
    """Descriptor of a paged pool: block_table [B, pages_per_seq] int32 on
    the device maps each sequence's logical pages of page_tokens tokens to
    pool pages ([num_pages, Hkv, page_tokens, width] pools)."""
    bt = _ptr(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, pages_per_seq]")
    return _lib.qasc_paged_cache(bt.value, int(page_tokens), int(block_table.shape[1]), int(num_pages))


def _pool_geometry(pool, block_table, width=D):
    _dims(pool, "pool", (None, None, None, width))
    _dims(block_table, "block_table", (None, None))
    num_pages, Hkv, P, _ = pool.shape
    B, pps = block_table.shape
    return B, Hkv, P, num_pages, pps * P


def ts_index_append_paged(K_pool, W, index_pool, block_table, start, count, *, Hq=None, n=None, stream=None):
    """Index rows of tokens [start, start + count) of every sequence, in the
    pool page that holds each token."""
    B, Hkv, P, num_pages, n_cap = _pool_geometry(K_pool, block_table)
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(index_pool, "index_pool", (num_pages, Hkv, P, D_IDX))
    shape = make_shape(B, Hq or Hkv, Hkv, n or n_cap, n_cap)
    cache = paged_cache(block_table, P, num_pages)
    _check(_L().ts_index_append_paged(ctypes.byref(shape), ctypes.byref(cache), _ptr(K_pool, "K_pool", torch.bfloat16),
                                      _ptr(W, "W", torch.bfloat16), _ptr(index_pool, "index_pool", torch.bfloat16),
                                      int(start), int(count), _stream(stream)))


def ts_score_vote_select_paged(q, W, index_pool, block_table, sel, workspace, *, n, K, sink=4, local=256, vmin=1,
                               stream=None):
    """ts_score_vote_select over a paged index pool (workspace:
    ts_select_workspace_bytes with n_cap = pages_per_seq * page_tokens)."""
    B, Hkv, P, num_pages, n_cap = _pool_geometry(index_pool, block_table, D_IDX)
    _dims(q, "q", (B, None, D))
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(sel, "sel", (B, K))
    shape = make_shape(B, q.shape[1], Hkv, n, n_cap)
    params = ts_params(K, sink, local, vmin)
    cache = paged_cache(block_table, P, num_pages)
    _check(_L().ts_score_vote_select_paged(ctypes.byref(shape), ctypes.byref(params), ctypes.byref(cache),
                                           _ptr(q, "q", torch.bfloat16), _ptr(W, "W", torch.bfloat16),
                                           _ptr(index_pool, "index_pool", torch.bfloat16),
                                           _ptr(sel, "sel", torch.int32), _ptr(workspace, "workspace", torch.uint8),
                                           workspace.numel(), _stream(stream)))


def ts_score_select_per_head_paged(q, W, index_pool, block_table, sel, workspace, *, n, K, sink=4, local=256,
                                   stream=None):
    """ts_score_select_per_head over a paged index pool (workspace:
    ts_head_select_workspace_bytes with n_cap = pages_per_seq * page_tokens)."""
    B, Hkv, P, num_pages, n_cap = _pool_geometry(index_pool, block_table, D_IDX)
    _dims(q, "q", (B, None, D))
    _dims(W, "W", (Hkv, D, D_IDX))
    _dims(sel, "sel", (B, Hkv, K))
    shape = make_shape(B, q.shape[1], Hkv, n, n_cap)
    params = ts_params(K, sink, local, 1)
    cache = paged_cache(block_table, P, num_pages)
    _check(_L().ts_score_select_per_head_paged(ctypes.byref(shape), ctypes.byref(params), ctypes.byref(cache),
                                               _ptr(q, "q", torch.bfloat16), _ptr(W, "W", torch.bfloat16),
                                               _ptr(index_pool, "index_pool", torch.bfloat16),
                                               _ptr(sel, "sel", torch.int32),
                                               _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
                                               _stream(stream)))


def _ring(ring, B, Hkv):
    if ring is None:
        return None
    rk, rv = ring
    if rk.shape != rv.shape or rk.dim() != 4 or tuple(rk.shape[:2]) != (B, Hkv) or rk.shape[3] != D:
        raise ValueError("ring K and V must both be [B=%d, Hkv=%d, R, %d]" % (B, Hkv, D))
    return _lib.qasc_local_ring(_ptr(rk, "ring K", torch.bfloat16).value, _ptr(rv, "ring V", torch.bfloat16).value,
                                int(rk.shape[2]))


def ts_sparse_attn_paged(q, K_pool, V_pool, block_table, sel, out, workspace, *, n, sink=4, local=256, ring=None,
                         lengths=None, per_kv_head=False, lse=None, stream=None):
    """ts_sparse_attn_ex over a paged pool; ring = (ring_K, ring_V), each
    [B, Hkv, R, d] with token t at slot t mod R, supplies the local tokens."""
    B, Hkv, P, num_pages, n_cap = _pool_geometry(K_pool, block_table)
    _dims(V_pool, "V_pool", (num_pages, Hkv, P, D))
    _dims(q, "q", (B, None, D))
    Hq = q.shape[1]
    _dims(out, "out", (B, Hq, D))
    _dims(lse, "lse", (B, Hq))
    _dims(sel, "sel", (B, Hkv, None) if per_kv_head else (B, None))
    _dims(lengths, "lengths", (B, Hkv) if per_kv_head else (B,))
    Ksel = sel.shape[-1] if sel is not None else 0
    shape = make_shape(B, q.shape[1], Hkv, n, n_cap)
    params = ts_params(Ksel, sink, local, 1)
    cache = paged_cache(block_table, P, num_pages)
    rg = _ring(ring, B, Hkv)
    _check(_L().ts_sparse_attn_paged(ctypes.byref(shape), ctypes.byref(params), ctypes.byref(cache),
                                     ctypes.byref(rg) if rg is not None else None, _ptr(q, "q", torch.bfloat16),
                                     _ptr(K_pool, "K_pool", torch.bfloat16), _ptr(V_pool, "V_pool", torch.bfloat16),
                                     _ptr(sel, "sel", torch.int32) if Ksel else None,
                                     _ptr(lengths, "lengths", torch.int32), 1 if per_kv_head else 0,
                                     _ptr(out, "out", torch.float32), _ptr(lse, "lse", torch.float32),
                                     _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream)))


def ts_ring_flush(ring, W, K_pool, V_pool, index_pool, block_table, start, count, *, n=None, stream=None):
    """Tokens [start, start + count) of every sequence from the ring into
    their pages (K and V rows copied, index rows written)."""
    B, Hkv, P, num_pages, n_cap = _pool_geometry(K_pool, block_table)
    _dims(V_pool, "V_pool", (num_pages, Hkv, P, D))
    _dims(index_pool, "index_pool", (num_pages, Hkv, P, D_IDX))
    _dims(W, "W", (Hkv, D, D_IDX))
    shape = make_shape(B, Hkv, Hkv, n or n_cap, n_cap)
    cache = paged_cache(block_table, P, num_pages)
    rg = _ring(ring, B, Hkv)
    _check(_L().ts_ring_flush(ctypes.byref(shape), ctypes.byref(cache), ctypes.byref(rg) if rg is not None else None,
                              _ptr(W, "W", torch.bfloat16), _ptr(K_pool, "K_pool", torch.bfloat16),
                              _ptr(V_pool, "V_pool", torch.bfloat16), _ptr(index_pool, "index_pool", torch.bfloat16),
                              int(start), int(count), _stream(stream)))


def ts_sparse_attn_noalloc(q, K, V, sel, out, *, n, sink=4, local=256, lse=None, stream=None):
    """ts_sparse_attn without a workspace, for callers that cannot allocate
    device memory: the split-K scratch is a fixed 16 MiB area inside the
    library, shared by all calls (serialise calls that could overlap)."""
    B, Hq, Hkv, n_cap = _attn_dims(q, K, V, out, lse)
    _dims(sel, "sel", (B, None))
    Ksel = sel.shape[1] if sel is not None else 0
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = ts_params(Ksel, sink, local, 1)
    _check(_L().ts_sparse_attn_noalloc(ctypes.byref(shape), ctypes.byref(params), _ptr(q, "q", torch.bfloat16),
                                       _ptr(K, "K", torch.bfloat16), _ptr(V, "V", torch.bfloat16),
                                       _ptr(sel, "sel", torch.int32) if Ksel else None,
                                       _ptr(out, "out", torch.float32), _ptr(lse, "lse", torch.float32),
                                       _stream(stream)))


def ts_dense_attn_workspace_bytes(B, Hq, Hkv, n, n_cap):
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    return _sized(_L().ts_dense_attn_workspace_bytes(ctypes.byref(shape)))


def ts_dense_attn(q, K, V, out, workspace, *, n, lse=None, stream=None):
    """out[b, h] = attention of q[b, h] over all n cached tokens (the baseline)."""
    B, Hq, Hkv, n_cap = _attn_dims(q, K, V, out, lse)
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    _check(_L().ts_dense_attn(ctypes.byref(shape), _ptr(q, "q", torch.bfloat16), _ptr(K, "K", torch.bfloat16),
                              _ptr(V, "V", torch.bfloat16), _ptr(out, "out", torch.float32),
                              _ptr(lse, "lse", torch.float32), _ptr(workspace, "workspace", torch.uint8),
                              workspace.numel(), _stream(stream)))


# ------------------------------------------------------- packed batches
# These calls sit in an engine's per-layer loop, where the host's time per call
# counts: one test per tensor against the call's device, and the device against
# the current one at the end.
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_Tensor = torch.Tensor
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
# of a process that holds a CUDA tensor, so that CUDA is up (0.06 us; torch.cuda.current_device 0.3)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _at(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this dtype and shape on device index
    dev (the checks of _dims and _ptr)."""
    if (isinstance(t, _Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    _dims(t, name, tuple(shape))
    _on_device(t.get_device(), name)
    return _ptr(t, name, dtype).value


def _on_device(dev, name):
    """Raise unless dev is the current CUDA device, where the library launches."""
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    current = _current_device()
    if dev != current:
        raise ValueError("%s is on cuda:%d but the current device is cuda:%d" % (name, dev, current))


def _heads(t, name, T, H, dev):
    """A [T, H, d] tensor whose tokens may lie apart (a part of a fused
    projection): its address and the values between tokens."""
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != (T, H, D):
        _dims(t, name, (T, H, D))
    st = t.stride()
    if T > 0 and (st[2] != 1 or (st[1] != D and H > 1)):
        raise ValueError("%s must be contiguous within a token, got strides %s" % (name, st))
    if t.dtype is not _BF16 or t.get_device() != dev:
        _on_device(t.get_device(), name)
        _ptr(t[:0], name, _BF16)     # raises
    return t.data_ptr(), st[0] if T > 1 else H * D


def _batch(cu_q, lens, T, dev):
    """The packed batch and B; cu_q [B + 1] (None: one token per sequence)."""
    if not isinstance(lens, _Tensor) or lens.dim() != 1:
        raise ValueError("kv_lens must be a [B] tensor")
    B = lens.shape[0]
    return _lib.pack_batch(0 if cu_q is None else _at(cu_q, "cu_q", _I32, (B + 1,), dev),
                           _at(lens, "kv_lens", _I32, (B,), dev), T), B


def _cache(K, V, block_table, B, Hkv, dev):
    """K and V [B, Hkv, n_cap, d], or pools [num_pages, Hkv, P, d] under
    block_table [B, pages_per_seq]: (descriptor or None, n_cap, Hkv, addresses
    of K and V)."""
    shape = K.shape
    if len(shape) != 4 or shape[3] != D or (Hkv is not None and shape[1] != Hkv):
        _dims(K, "K", (None if block_table is not None else B, Hkv, None, D))
    if block_table is None:
        if shape[0] != B:
            _dims(K, "K", (B, Hkv, None, D))
        cache, n_cap = None, shape[2]
    else:
        table = block_table.shape
        if len(table) != 2 or table[0] != B:
            _dims(block_table, "block_table", (B, None))
        n_cap = table[1] * shape[2]
        cache = _lib.pack_cache(_at(block_table, "block_table", _I32, table, dev), shape[2], table[1], shape[0])
    return cache, n_cap, shape[1], _at(K, "K", _BF16, shape, dev), _at(V, "V", _BF16, shape, dev)


def _table(block_table):
    if not isinstance(block_table, _Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must have shape (B, pages_per_seq)")


def _run(fn, dev, stream, shape, cache, *args):
    """One call of the library: shape and cache descriptors (packed), then args and the stream."""
    _on_device(dev, "the call's first tensor")
    if stream is None:
        s = _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    else:
        s = _stream(stream)
    if cache is None:
        status = fn(shape, *args, s)
    else:
        status = fn(shape, cache, *args, s)
    if status != _lib.QASC_OK:
        _check(status)


def _new_rows(q, k, v, q_out, T, Hkv, inv_freq, positions, interleaved, dev):
    """An append's queries, keys and values: Hq, the library's arguments for them,
    and the rotation's descriptor."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    Hq, qp, qs, op = Hkv, None, 0, None
    if q is not None:
        if not isinstance(q, _Tensor) or q.dim() != 3:
            raise ValueError("q must be a [T, Hq, %d] tensor" % D)
        Hq = q.shape[1]
        qp, qs = _heads(q, "q", T, Hq, dev)
        op = _at(q_out, "q_out", _BF16, (T, Hq, D), dev)
    kp, ks = _heads(k, "k", T, Hkv, dev)
    vp, vs = _heads(v, "v", T, Hkv, dev)
    rot, fp = 0, 0
    if inv_freq is not None:
        _dims(inv_freq, "inv_freq", (None,))
        rot, fp = 2 * inv_freq.shape[0], _at(inv_freq, "inv_freq", _F32, inv_freq.shape, dev)
    pp = 0 if positions is None else _at(positions, "positions", _I32, (T,), dev)
    return Hq, (qp, qs, kp, ks, vp, vs, op), _lib.pack_rope(fp, pp, rot, 1 if interleaved else 0)


def _rope_append(name, q, k, v, q_out, K, V, block_table, kv_lens, inv_freq, cu_q, positions, interleaved, stream):
    if not isinstance(k, _Tensor) or k.dim() != 3:
        raise ValueError("k must be a [T, Hkv, %d] tensor" % D)
    dev = k.get_device()
    T, Hkv, _ = k.shape
    batch, B = _batch(cu_q, kv_lens, T, dev)
    cache, n_cap, Hkv, Kp, Vp = _cache(K, V, block_table, B, Hkv, dev)
    Hq, rows, rope = _new_rows(q, k, v, q_out, T, Hkv, inv_freq, positions, interleaved, dev)
    _run(getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hq, Hkv, D, D_IDX, 0, n_cap, n_cap), cache, batch, rope,
         *rows, Kp, Vp)


def kv_rope_append(q, k, v, q_out, K, V, kv_lens, inv_freq, *, cu_q=None, positions=None, interleaved=False,
                   stream=None):
    """New tokens' keys (rotated) and values into K, V [B, Hkv, n_cap, d], and
    their rotated queries into q_out.  q [T, Hq, d] (None: keys and values
    only), k, v [T, Hkv, d] may be parts of one fused projection; sequence b
    has tokens cu_q[b] .. cu_q[b + 1] (None: one each), the last of its
    kv_lens[b] cached ones; inv_freq [rot_dim / 2] (None: no rotation) turns
    by the cache position, or by positions [T]."""
    _rope_append("kv_rope_append", q, k, v, q_out, K, V, None, kv_lens, inv_freq, cu_q, positions, interleaved,
                 stream)


def kv_rope_append_paged(q, k, v, q_out, K_pool, V_pool, block_table, kv_lens, inv_freq, *, cu_q=None,
                         positions=None, interleaved=False, stream=None):
    """kv_rope_append into a paged pool [num_pages, Hkv, P, d]."""
    _table(block_table)
    _rope_append("kv_rope_append_paged", q, k, v, q_out, K_pool, V_pool, block_table, kv_lens, inv_freq, cu_q,
                 positions, interleaved, stream)


def _attn(name, q, K, V, block_table, kv_lens, out, workspace, cu_q, lse, stream, front, behind, fn=None):
    """front: the library's arguments before the batch, behind: those after it;
    fn: called in place of the library's `name`."""
    if not isinstance(q, _Tensor) or q.dim() != 3:
        raise ValueError("q must have shape (T, Hq, %d)" % D)
    dev = q.get_device()
    shape = q.shape
    T, Hq, d = shape
    if d != D:
        _dims(q, "q", (T, Hq, D))
    batch, B = _batch(cu_q, kv_lens, T, dev)
    cache, n_cap, Hkv, Kp, Vp = _cache(K, V, block_table, B, None, dev)
    qp = _at(q, "q", _BF16, shape, dev)
    op = _at(out, "out", _BF16, shape, dev)
    lp = None if lse is None else _at(lse, "lse", _F32, (T, Hq), dev)
    ws_bytes = workspace.numel()
    wp = _at(workspace, "workspace", _U8, (ws_bytes,), dev)
    _run(fn or getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hq, Hkv, D, D_IDX, 0, n_cap, n_cap), cache, *front,
         batch, *behind, qp, Kp, Vp, op, lp, wp, ws_bytes)


def _tokens32(n):
    """A number of tokens in the library's 32 bits, to which ctypes cuts without
    an error: a cache holds fewer than 2^24, so that any more mean the same."""
    return n if -0x80000000 <= n < 0x80000000 else (0x7fffffff if n > 0 else -1)


def kv_window_attn_workspace_bytes(T, B, Hq, Hkv, n_cap):
    return _sized(_L().kv_window_attn_workspace_bytes(ctypes.byref(make_shape(B, Hq, Hkv, n_cap, n_cap)), T))


def kv_window_attn(q, K, V, kv_lens, out, workspace, *, local, sink=4, cu_q=None, lse=None, stream=None):
    """out[t, h] = causal attention of the new token t over the first `sink`
    and the newest `local` cached tokens of its sequence up to its own
    position; q, out [T, Hq, d] bf16, K, V [B, Hkv, n_cap, d], the batch as
    for kv_rope_append."""
    _attn("kv_window_attn", q, K, V, None, kv_lens, out, workspace, cu_q, lse, stream, (),
          (_tokens32(sink), _tokens32(local)))


def kv_window_attn_paged(q, K_pool, V_pool, block_table, kv_lens, out, workspace, *, local, sink=4, cu_q=None,
                         lse=None, stream=None):
    """kv_window_attn over a paged pool [num_pages, Hkv, P, d]."""
    _table(block_table)
    _attn("kv_window_attn_paged", q, K_pool, V_pool, block_table, kv_lens, out, workspace, cu_q, lse, stream, (),
          (_tokens32(sink), _tokens32(local)))


def kv_prefix_attn_workspace_bytes(T, B, Hq, Hkv, n_cap):
    return _sized(_L().kv_prefix_attn_workspace_bytes(ctypes.byref(make_shape(B, Hq, Hkv, n_cap, n_cap)), T))


def kv_prefix_attn_paged(q, K_pool, V_pool, prefix_table, block_table, kv_lens, out, workspace, *, n_prefix,
                         cu_q=None, lse=None, stream=None):
    """Causal attention of sequences that share their first n_prefix tokens
    (the pool pages prefix_table [ceil(n_prefix / P)]), a long one read once for
    all of them; block_table and kv_lens describe each sequence's own tokens behind
    the prefix."""
    _table(block_table)
    pt = None
    if n_prefix > 0:
        pt = _at(prefix_table, "prefix_table", _I32, (-(-n_prefix // K_pool.shape[2]),), block_table.get_device())
    _attn("kv_prefix_attn_paged", q, K_pool, V_pool, block_table, kv_lens, out, workspace, cu_q, lse, stream,
          (pt, n_prefix), ())


# ---------------------------------------------------------- the 4-bit cache
class KV4:
    """A 4-bit cache: codes K, V [B, Hkv, n_cap, 64] uint8 and scales K_sf, V_sf
    [B, Hkv, n_cap, 8] float8_e4m3fn, or pools [num_pages, Hkv, P, ..] of them;
    value i of a row = factor * scale[i // 16] * code[i], the codes 4-bit floats,
    k_scale and v_scale the factors of keys and values (powers of two).  A handle
    that a program keeps with its cache: its tensors are checked once, at the first
    call, and do not change."""
    __slots__ = ("K", "K_sf", "V", "V_sf", "k_scale", "v_scale", "_checked")

    def __init__(self, K, K_sf, V, V_sf, k_scale=1.0, v_scale=1.0):
        for name, value in zip(KV4.__slots__, (K, K_sf, V, V_sf, float(k_scale), float(v_scale), None)):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("a KV4 does not change; make another of its tensors")

    def __iter__(self):
        return iter((self.K, self.K_sf, self.V, self.V_sf, self.k_scale, self.v_scale))


_E4M3 = torch.float8_e4m3fn


def alloc_kv4(rows, Hkv, tokens, device=None, k_scale=1.0, v_scale=1.0):
    """A cache of zeros: rows = B and tokens = n_cap, or the pages of a pool and
    their tokens."""
    codes, scales = (torch.zeros((2, rows, Hkv, tokens, w), dtype=torch.uint8, device=device or "cuda")
                     for w in (D // 2, D // 16))
    return KV4(codes[0], scales[0].view(_E4M3), codes[1], scales[1].view(_E4M3), k_scale, v_scale)


def _check4(kv):
    """Checks a KV4's tensors: (device index, shape of K, addresses, descriptor)."""
    if not isinstance(kv.K, _Tensor) or kv.K.dim() != 4 or kv.K.shape[3] != D // 2:
        raise ValueError("kv.K must be a [B or num_pages, Hkv, tokens, %d] tensor" % (D // 2))
    dev, shape = kv.K.get_device(), kv.K.shape
    scales = shape[:3] + (D // 16,)
    where = (_at(kv.K, "kv.K", _U8, shape, dev), _at(kv.K_sf, "kv.K_sf", _E4M3, scales, dev),
             _at(kv.V, "kv.V", _U8, shape, dev), _at(kv.V_sf, "kv.V_sf", _E4M3, scales, dev))
    checked = dev, tuple(shape), where, _lib.pack_kv4(*where, kv.k_scale, kv.v_scale)
    object.__setattr__(kv, "_checked", checked)
    return checked


def _cache4(kv, block_table, B, Hkv, dev):
    """A KV4 [B, Hkv, n_cap, ..], or of pools under block_table [B, pages_per_seq]:
    (descriptor of the pool or None, n_cap, Hkv, descriptor of the cache)."""
    if type(kv) is not KV4:
        raise TypeError("kv must be a KV4")
    checked = kv._checked
    if checked is None or checked[2] != (kv.K.data_ptr(), kv.K_sf.data_ptr(), kv.V.data_ptr(), kv.V_sf.data_ptr()):
        checked = _check4(kv)
    rows, heads, tokens, _ = shape = checked[1]
    if checked[0] != dev or (Hkv is not None and heads != Hkv) or (block_table is None and rows != B):
        _dims(kv.K, "kv.K", (B if block_table is None else None, Hkv, None, D // 2))
        raise ValueError("kv is on cuda:%d, the call's other tensors on %s" % (checked[0], "cuda:%d" % dev if dev >= 0 else "the CPU"))
    if block_table is None:
        return None, tokens, heads, checked[3]
    table = block_table.shape
    if len(table) != 2 or table[0] != B:
        _dims(block_table, "block_table", (B, None))
    cache = _lib.pack_cache(_at(block_table, "block_table", _I32, table, dev), tokens, table[1], rows)
    return cache, table[1] * tokens, heads, checked[3]


def _rope_append4(name, q, k, v, q_out, kv, block_table, kv_lens, inv_freq, cu_q, positions, interleaved, stream):
    if not isinstance(k, _Tensor) or k.dim() != 3:
        raise ValueError("k must be a [T, Hkv, %d] tensor" % D)
    dev = k.get_device()
    T, Hkv, _ = k.shape
    batch, B = _batch(cu_q, kv_lens, T, dev)
    cache, n_cap, Hkv, kvp = _cache4(kv, block_table, B, Hkv, dev)
    Hq, rows, rope = _new_rows(q, k, v, q_out, T, Hkv, inv_freq, positions, interleaved, dev)
    _run(getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hq, Hkv, D, D_IDX, 0, n_cap, n_cap), cache, batch, rope,
         *rows, kvp)


def kv4_rope_append(q, k, v, q_out, kv, kv_lens, inv_freq, *, cu_q=None, positions=None, interleaved=False, stream=None):
    """kv_rope_append into a 4-bit cache kv (KV4): new tokens' keys (rotated) and
    values quantised, their rotated queries into q_out."""
    _rope_append4("kv4_rope_append", q, k, v, q_out, kv, None, kv_lens, inv_freq, cu_q, positions, interleaved, stream)


def kv4_rope_append_paged(q, k, v, q_out, kv_pool, block_table, kv_lens, inv_freq, *, cu_q=None, positions=None,
                          interleaved=False, stream=None):
    """kv4_rope_append into pools (a KV4 of [num_pages, Hkv, P, ..])."""
    _table(block_table)
    _rope_append4("kv4_rope_append_paged", q, k, v, q_out, kv_pool, block_table, kv_lens, inv_freq, cu_q, positions,
                  interleaved, stream)


def _strided_rows(t, name, T, Hkv, dev):
    """A [T, Hkv, d] output whose tokens and heads may lie apart: its address and the
    values between tokens and between heads."""
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != (T, Hkv, D):
        _dims(t, name, (T, Hkv, D))
    st = t.stride()
    if T > 0 and st[2] != 1:
        raise ValueError("%s must be contiguous within a head, got strides %s" % (name, st))
    # rows that share memory would be written by several threads
    a, b = sorted(((st[0], T), (st[1], Hkv)))
    if (a[1] > 1 and a[0] < D) or (b[1] > 1 and b[0] < D + (a[1] - 1) * a[0]):
        raise ValueError("%s: rows overlap, got strides %s" % (name, st))
    if t.dtype is not _BF16 or t.get_device() != dev:
        _on_device(t.get_device(), name)
        _ptr(t[:0], name, _BF16)     # raises
    return t.data_ptr(), st[0] if T > 1 else Hkv * D, st[1] if Hkv > 1 else D


def _read4(name, kv, block_table, kv_lens, K_out, V_out, cu_q, stream):
    if not isinstance(K_out, _Tensor) or K_out.dim() != 3:
        raise ValueError("K_out must be a [T, Hkv, %d] tensor" % D)
    dev = K_out.get_device()
    T = K_out.shape[0]
    batch, B = _batch(cu_q, kv_lens, T, dev)
    cache, n_cap, Hkv, kvp = _cache4(kv, block_table, B, None, dev)
    _run(getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hkv, Hkv, D, D_IDX, 0, n_cap, n_cap), cache, batch, kvp,
         *_strided_rows(K_out, "K_out", T, Hkv, dev), *_strided_rows(V_out, "V_out", T, Hkv, dev))


def kv4_read(kv, kv_lens, K_out, V_out, *, cu_q=None, stream=None):
    """The newest tokens of a 4-bit cache back in bf16: K_out, V_out [T, Hkv, d],
    packed as new tokens are (cu_q; whole sequences with the sums of kv_lens).
    Their tokens and heads may lie apart (e.g. cache[0].transpose(0, 1))."""
    _read4("kv4_read", kv, None, kv_lens, K_out, V_out, cu_q, stream)


def kv4_read_paged(kv_pool, block_table, kv_lens, K_out, V_out, *, cu_q=None, stream=None):
    """kv4_read from pools (a KV4 of [num_pages, Hkv, P, ..])."""
    _table(block_table)
    _read4("kv4_read_paged", kv_pool, block_table, kv_lens, K_out, V_out, cu_q, stream)


def kv4_window_attn_workspace_bytes(T, B, Hq, Hkv, n_cap, *, local, sink=4, max_q=None):
    """Bytes with which every call of up to T tokens, max_q of a sequence (None: T), takes
    its fastest form; calls accept less, down to the size for max_q = 1."""
    return _sized(_L().kv4_window_attn_workspace_bytes(ctypes.byref(make_shape(B, Hq, Hkv, n_cap, n_cap)), T,
                                                       T if max_q is None else max_q, _tokens32(sink), _tokens32(local)))


def _queries(q):
    if not isinstance(q, _Tensor) or q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must have shape (T, Hq, %d)" % D)
    return q.shape[0], q.shape[1], q.get_device()


def _outputs(q, out, lse, workspace, dev):
    """Addresses of the queries, and the arguments that end every attention call."""
    ws_bytes = workspace.numel()
    return _at(q, "q", _BF16, q.shape, dev), (
        _at(out, "out", _BF16, q.shape, dev), None if lse is None else _at(lse, "lse", _F32, q.shape[:2], dev),
        _at(workspace, "workspace", _U8, (ws_bytes,), dev), ws_bytes)


def _window4(name, q, kv, block_table, kv_lens, out, workspace, local, sink, cu_q, max_q, lse, stream):
    T, Hq, dev = _queries(q)
    batch, B = _batch(cu_q, kv_lens, T, dev)
    cache, n_cap, Hkv, kvp = _cache4(kv, block_table, B, None, dev)
    qp, outputs = _outputs(q, out, lse, workspace, dev)
    _run(getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hq, Hkv, D, D_IDX, 0, n_cap, n_cap), cache, batch,
         T if max_q is None else max_q, _tokens32(sink), _tokens32(local), qp, kvp, *outputs)


def kv4_window_attn(q, kv, kv_lens, out, workspace, *, local, sink=4, cu_q=None, max_q=None, lse=None, stream=None):
    """kv_window_attn over a 4-bit cache kv (KV4); max_q: the most new tokens of any
    sequence where the caller knows it (None: T)."""
    _window4("kv4_window_attn", q, kv, None, kv_lens, out, workspace, local, sink, cu_q, max_q, lse, stream)


def kv4_window_attn_paged(q, kv_pool, block_table, kv_lens, out, workspace, *, local, sink=4, cu_q=None, max_q=None,
                          lse=None, stream=None):
    """kv4_window_attn over pools (a KV4 of [num_pages, Hkv, P, ..])."""
    _table(block_table)
    _window4("kv4_window_attn_paged", q, kv_pool, block_table, kv_lens, out, workspace, local, sink, cu_q, max_q, lse,
             stream)


def kv4_sparse_attn_workspace_bytes(B, Hq, Hkv, n, n_cap, K, sink=4, local=256):
    shape, params = make_shape(B, Hq, Hkv, n, n_cap), ts_params(K, _tokens32(sink), _tokens32(local), 1)
    return _sized(_L().kv4_sparse_attn_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def _sparse4(name, q, kv, block_table, sel, out, workspace, n, sink, local, lengths, per_kv_head, lse, stream):
    B, Hq, dev = _queries(q)
    cache, n_cap, Hkv, kvp = _cache4(kv, block_table, B, None, dev)
    qp, outputs = _outputs(q, out, lse, workspace, dev)
    lists = (B, Hkv) if per_kv_head else (B,)
    K = sel.shape[-1] if sel is not None else 0
    sp = _at(sel, "sel", _I32, lists + (K,), dev) if K else None
    up = None if lengths is None else _at(lengths, "lengths", _I32, lists, dev)
    params = _lib.pack_params(K, _tokens32(sink), _tokens32(local), 1)
    _run(getattr(_L(), name), dev, stream, _lib.pack_shape(B, Hq, Hkv, D, D_IDX, 0, n, n_cap), None,
         *((params,) if cache is None else (params, cache)), qp, kvp, sp, up, 1 if per_kv_head else 0, *outputs)


def kv4_sparse_attn(q, kv, sel, out, workspace, *, n, sink=4, local=256, lengths=None, per_kv_head=False, lse=None,
                    stream=None):
    """out[b, h] = attention over the sink, listed and local tokens of a 4-bit cache kv
    (KV4) of n tokens: sel [B, K] or (per_kv_head) [B, Hkv, K] with lengths [B] or
    [B, Hkv], as for ts_sparse_attn_ex; q, out [B, Hq, d] bf16."""
    _sparse4("kv4_sparse_attn", q, kv, None, sel, out, workspace, n, sink, local, lengths, per_kv_head, lse, stream)


def kv4_sparse_attn_paged(q, kv_pool, block_table, sel, out, workspace, *, n, sink=4, local=256, lengths=None,
                          per_kv_head=False, lse=None, stream=None):
    """kv4_sparse_attn over pools (a KV4 of [num_pages, Hkv, P, ..])."""
    _table(block_table)
    _sparse4("kv4_sparse_attn_paged", q, kv_pool, block_table, sel, out, workspace, n, sink, local, lengths,
             per_kv_head, lse, stream)


# ------------------------------------------------------------------ SnapKV
def snapkv_workspace_bytes(B, Hq, Hkv, n, n_cap, c, window=32, pool_k=3):
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = snap_params(c, window, pool_k)
    return _sized(_L().snapkv_workspace_bytes(ctypes.byref(shape), ctypes.byref(params)))


def snapkv_compress(q_obs, K, V, idx, K_out, V_out, workspace, *, n, c, pool_k=3, stream=None):
    """Keep min(c, n) entries per KV head chosen by observation-window attention."""
    _dims(q_obs, "q_obs", (None, None, None, D))
    B, Hq, w, _ = q_obs.shape
    _dims(K, "K", (B, None, None, D))
    _, Hkv, n_cap, _ = K.shape
    _dims(V, "V", (B, Hkv, n_cap, D))
    c_out = min(c, n)
    _dims(idx, "idx", (B, Hkv, c_out))
    _dims(K_out, "K_out", (B, Hkv, c_out, D))
    _dims(V_out, "V_out", (B, Hkv, c_out, D))
    shape = make_shape(B, Hq, Hkv, n, n_cap)
    params = snap_params(c, w, pool_k)
    _check(_L().snapkv_compress(ctypes.byref(shape), ctypes.byref(params), _ptr(q_obs, "q_obs", torch.bfloat16),
                                _ptr(K, "K", torch.bfloat16), _ptr(V, "V", torch.bfloat16),
                                _ptr(idx, "idx", torch.int32), _ptr(K_out, "K_out", torch.bfloat16),
                                _ptr(V_out, "V_out", torch.bfloat16), _ptr(workspace, "workspace", torch.uint8),
                                workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------ status
def qasc_status_string(status):
    return _L().qasc_status_string(int(status)).decode()


def qasc_last_error():
    return _L().qasc_last_error().decode()


def qasc_last_cuda_error():
    return _L().qasc_last_cuda_error().decode()


def qasc_device_error(stream=None):
    _check(_L().qasc_device_error(_stream(stream)))


def qasc_selftest_bounded_wait(limit_us, stream=None):
    """Run one kernel whose bounded wait cannot complete; it gives up after
    limit_us and records a timeout for the next qasc_device_error()."""
    _check(_L().qasc_selftest_bounded_wait(int(limit_us), _stream(stream)))


def qasc_selftest_attn_wait(limit_us, stall, q, K, V, kv_lens, out, workspace, *, local, sink=4, cu_q=None, lse=None,
                            stream=None):
    """kv_window_attn in which no block gets its K and V tiles from the stall-th
    on, with waits that give up after limit_us: the next qasc_device_error()
    reports the timeout and out and lse are undefined."""
    call = _L().qasc_selftest_attn_wait
    _attn("qasc_selftest_attn_wait", q, K, V, None, kv_lens, out, workspace, cu_q, lse, stream, (),
          (_tokens32(sink), _tokens32(local)), fn=lambda *args: call(int(limit_us), int(stall), *args))


def qasc_version():
    return int(_L().qasc_version())
