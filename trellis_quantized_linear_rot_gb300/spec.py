"""The operators between the decode-row projections when several rows of a
pass belong to one sequence (include/tf_spec.h): a tree of drafted tokens is
written into a paged cache, attends to it, is verified against the target's
probabilities, and the accepted path is kept. A tree of one node is ordinary
decoding.

    tf_kv_write(k_new, v_new, k_cache, v_cache, page_table, lengths)
    out, lse = tf_tree_attention(q, k_cache, v_cache, page_table, lengths, parents)
    counts, path, tokens, logprobs = tf_verify_draft(logits, drafted, parents, u_sample)
    lengths = tf_kv_keep(k_cache, v_cache, page_table, lengths, path, counts)

Like the projections, the calls are asynchronous on the current stream (or
`stream=`), refuse bad arguments before launching anything, and leave what
only the device can see (an index outside its array) to tf_device_error.

A call of one token runs for a few microseconds on the GPU, less than a
careless binding takes on the host, so the functions here look each
attribute up once, take the stream's handle without making a stream object,
and pack tf_kv_cache into bytes.
"""

import ctypes
import struct

TF_MAX_NODES = 128

_VP, _I, _L, _D, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t


class KVCache(ctypes.Structure):
    """tf_kv_cache of tf_spec.h."""
    _fields_ = [("k", _VP), ("v", _VP), ("stride_layer", _L), ("stride_page", _L), ("stride_token", _L),
                ("stride_head", _L), ("page_table", _VP), ("lengths", _VP), ("stride_table", _L),
                ("dtype", ctypes.c_int32), ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("table_width", ctypes.c_int32)]


_pack_cache = struct.Struct("@9q8i").pack   # the fields of KVCache, in order

# A cache is passed as a pointer: ctypes.byref of a KVCache, or its bytes.
SIGNATURES = {
    "tf_kv_write": (_I, [_VP, _VP, _VP, _L, _L, _L, _I, _VP]),
    "tf_tree_attention": (_I, [_VP, _VP, _L, _L, _L, _VP, _L, _VP, _VP, _I, _I, _D, _VP, _SZ, _VP]),
    "tf_tree_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "tf_verify_draft": (_I, [_VP, _I, _L, _L, _VP, _L, _L, _VP, _VP, _L, _VP, _VP, _D, _I, _I, _I, _VP, _VP, _VP, _VP,
                             _VP, _SZ, _VP]),
    "tf_verify_draft_workspace_bytes": (_SZ, [_I, _I]),
    "tf_kv_keep": (_I, [_VP, _VP, _VP, _I, _VP, _VP]),
}

_workspaces = {}
_tf = torch = _lib = _codes = _raw_stream = None


def _load():
    """The package, torch and the library, looked up on the first call (the
    package imports this module, and torch only where it is used)."""
    global _tf, torch, _lib, _codes, _raw_stream
    import torch as _torch
    import trellis_quantized_linear_rot_gb300 as tf
    lib = tf.lib()
    _tf, torch = tf, _torch
    _codes = {_torch.float16: tf.TF_F16, _torch.float32: tf.TF_F32, _torch.bfloat16: tf.TF_BF16}
    _raw_stream = _torch._C._cuda_getCurrentRawStream
    _lib = lib
    return lib


def _check(status, what):
    if status:
        raise _tf.TFError(status, what)


def _strides(t):
    """Strides, 0 for a dimension of one element (its stride means nothing)."""
    st = t.stride()
    if 1 in t.shape:
        st = tuple([0 if n == 1 else s for n, s in zip(t.shape, st)])
    return st


def _handle(stream, device):
    return stream.cuda_stream if stream is not None else _raw_stream(device.index or 0)


def _empty(stream, shape, dtype, device):
    """A new tensor whose memory belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _int32(t, name, shape):
    if t.dtype != torch.int32:
        raise TypeError("%s must be int32" % name)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous and of shape %s" % (name, tuple(shape)))


def _parents(parents, batch, nodes):
    """Row stride of parents: [batch, nodes], or one [nodes] for all sequences."""
    if parents.dtype != torch.int32:
        raise TypeError("parents must be int32")
    shape = parents.shape
    if (shape != (batch, nodes) and shape != (nodes,)) or (nodes > 1 and parents.stride(-1) != 1):
        raise ValueError("parents must be of shape %s or %s, rows contiguous" % ((batch, nodes), (nodes,)))
    return 0 if len(shape) == 1 or batch == 1 else parents.stride(0)


def _cache(k, v, page_table, lengths, layers=False):
    """(packed tf_kv_cache, batch); k's shape and the other tensors are checked."""
    shape, st = k.shape, k.stride()
    dims = len(shape)
    if dims != 4 and not (layers and dims == 5):
        raise ValueError("a cache is [%spages, page_size, kv_heads, head_dim]" % ("layers, " if layers else ""))
    same = v.stride() == st
    if 1 in shape:
        st = _strides(k)
        same = _strides(v) == st
    if not same or v.shape != shape or v.dtype != k.dtype or st[-1] != 1:
        raise ValueError("k_cache and v_cache must share shape, strides and dtype, the last dimension contiguous")
    int32 = torch.int32
    if page_table.dtype != int32 or lengths.dtype != int32:
        raise TypeError("page_table and lengths must be int32")
    table, rows, batch = page_table.shape, page_table.stride(), lengths.shape
    if len(batch) != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be [batch], contiguous")
    batch = batch[0]
    if len(table) != 2 or table[0] != batch or (rows[1] != 1 and table[1] > 1):
        raise ValueError("page_table must be [batch, table_width], rows contiguous")
    code = _codes.get(k.dtype, -1)
    if dims == 5:
        packed = _pack_cache(k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], st[3], page_table.data_ptr(),
                             lengths.data_ptr(), rows[0], code, shape[0], shape[1], shape[2], shape[3], shape[4],
                             batch, table[1])
    else:
        packed = _pack_cache(k.data_ptr(), v.data_ptr(), 0, st[0], st[1], st[2], page_table.data_ptr(),
                             lengths.data_ptr(), rows[0], code, 1, shape[0], shape[1], shape[2], shape[3], batch,
                             table[1])
    return packed, batch


def _captured(stream):
    """Whether the stream the call runs on is being captured, which is not
    always what the current one is."""
    if stream is None:
        return torch._C._cuda_isCurrentStreamCapturing()
    with torch.cuda.stream(stream):
        return torch._C._cuda_isCurrentStreamCapturing()


def _workspace(name, nbytes, device, handle, stream):
    """The workspace the binding keeps for the stream. While the stream is
    captured into a graph each call gets its own (its zeroing is captured
    too): a kept one may be dropped for a larger one, and the graph would go
    on using its memory."""
    ws = _workspaces.get((name, device.index, handle))
    if ws is not None and ws[1] >= nbytes and not _captured(stream):
        return ws
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device):
        t = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device)
        ws = (t.data_ptr(), nbytes, t)
        if not torch.cuda.is_current_stream_capturing():
            _workspaces[name, device.index, handle] = ws
    return ws


def _given(workspace):
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def forget_workspaces():
    """Drops the workspaces kept by the binding (after an aborted kernel they
    are made anew, zeroed)."""
    _workspaces.clear()


def tf_kv_write(k_new, v_new, k_cache, v_cache, page_table, lengths, stream=None):
    """Writes the tree's keys and values (k_new, v_new: [batch, nodes, kv_heads,
    head_dim], any strides with the last dimension contiguous) into slots
    lengths[b] + i of the cache [pages, page_size, kv_heads, head_dim]."""
    lib = _lib or _load()
    c, batch = _cache(k_cache, v_cache, page_table, lengths)
    shape = k_new.shape
    st = _strides(k_new)
    if v_new.shape != shape or _strides(v_new) != st or st[-1] != 1:
        raise ValueError("k_new and v_new must share shape and strides, the last dimension contiguous")
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype:
        raise TypeError("k_new and v_new must have the cache's dtype")
    if len(shape) != 4 or shape[0] != batch or shape[2:] != k_cache.shape[2:]:
        raise ValueError("k_new must be [batch, nodes, kv_heads, head_dim]")
    _check(lib.tf_kv_write(c, k_new.data_ptr(), v_new.data_ptr(), st[0], st[1], st[2], shape[1],
                           _handle(stream, k_cache.device)), "tf_kv_write")


def tf_tree_attention_workspace(batch, nodes, heads, kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for tf_tree_attention calls of up to these sizes."""
    need = (_lib or _load()).tf_tree_attention_workspace_bytes
    n = need(batch, nodes, heads, kv_heads, head_dim)
    if n:   # fewer kv heads have more rows each, and need more
        n = need(batch, nodes, heads, 1, head_dim)
    return torch.zeros(max(n, 1), dtype=torch.uint8, device=device)


def tf_tree_attention(q, k_cache, v_cache, page_table, lengths, parents, scale=None, out=None, lse=None,
                      workspace=None, stream=None):
    """Attention of the tree's nodes over the cache (see tf_tree_attention).

    q: [batch, nodes, heads, head_dim] (last dimension contiguous); caches
    [pages, page_size, kv_heads, head_dim]; page_table [batch, width], lengths
    [batch], parents [batch, nodes] or [nodes], all int32. scale defaults to
    1/sqrt(head_dim). Returns (out, lse): out like q, contiguous; lse fp32
    [batch, nodes, heads].
    """
    lib = _lib or _load()
    cache, batch = _cache(k_cache, v_cache, page_table, lengths)
    shape, dtype, device = q.shape, q.dtype, q.device
    if dtype != k_cache.dtype:
        raise TypeError("q must have the cache's dtype")
    st = _strides(q)
    if len(shape) != 4 or shape[0] != batch or shape[3] != k_cache.shape[3] or st[3] != 1:
        raise ValueError("q must be [batch, nodes, heads, head_dim], the last dimension contiguous")
    b, n, h, d = shape
    ps = _parents(parents, b, n)
    if out is None:
        out = _empty(stream, shape, dtype, device)
    elif out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and dtype")
    if lse is None:
        lse = _empty(stream, (b, n, h), torch.float32, device)
    elif lse.shape != (b, n, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [batch, nodes, heads]")
    handle = _handle(stream, device)
    if workspace is not None:
        ws = _given(workspace)
    else:
        ws = _workspace("attention", lib.tf_tree_attention_workspace_bytes(b, n, h, k_cache.shape[2], d), device,
                        handle, stream)
    _check(lib.tf_tree_attention(cache, q.data_ptr(), st[0], st[1], st[2], parents.data_ptr(), ps, out.data_ptr(),
                                 lse.data_ptr(), n, h, d ** -0.5 if scale is None else scale, ws[0], ws[1], handle),
           "tf_tree_attention")
    return out, lse


def tf_verify_draft_workspace(batch, nodes, device="cuda"):
    """A zeroed workspace for tf_verify_draft calls of up to these sizes."""
    n = (_lib or _load()).tf_verify_draft_workspace_bytes(batch, nodes)
    return torch.zeros(max(n, 1), dtype=torch.uint8, device=device)


def tf_verify_draft(logits, tokens, parents, u_sample, temperature=1.0, draft_logits=None, u_accept=None,
                    workspace=None, stream=None):
    """Which drafted tokens the target accepts (see tf_verify_draft).

    logits, draft_logits: [batch, nodes, vocab] fp32, fp16 or bf16 (last
    dimension contiguous); tokens int32 [batch, nodes]; parents [batch, nodes]
    or [nodes]; u_sample, u_accept fp32 [batch, nodes] (u_sample may be None
    at temperature 0, u_accept without draft_logits). Returns (counts, path,
    out_tokens, logprobs).
    """
    lib = _lib or _load()
    shape, dtype = logits.shape, logits.dtype
    st = _strides(logits)
    if len(shape) != 3 or (shape[2] > 1 and st[2] != 1):
        raise ValueError("logits must be [batch, nodes, vocab], the last dimension contiguous")
    b, n, v = shape
    rows = torch.Size((b, n))
    _int32(tokens, "tokens", rows)
    ps = _parents(parents, b, n)
    draft, ds = None, st
    if draft_logits is not None:
        ds = _strides(draft_logits)
        if draft_logits.shape != shape or draft_logits.dtype != dtype or (v > 1 and ds[2] != 1):
            raise ValueError("draft_logits must be like logits, the last dimension contiguous")
        draft = draft_logits.data_ptr()
    us = ua = None
    if u_sample is not None:
        if u_sample.dtype != torch.float32 or u_sample.shape != rows or not u_sample.is_contiguous():
            raise ValueError("u_sample must be contiguous fp32 [batch, nodes]")
        us = u_sample.data_ptr()
    if u_accept is not None:
        if u_accept.dtype != torch.float32 or u_accept.shape != rows or not u_accept.is_contiguous():
            raise ValueError("u_accept must be contiguous fp32 [batch, nodes]")
        ua = u_accept.data_ptr()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("unsupported dtype %s" % dtype)
    device = logits.device
    counts = _empty(stream, (b,), torch.int32, device)
    path = _empty(stream, rows, torch.int32, device)
    out = _empty(stream, rows, torch.int32, device)
    logprobs = _empty(stream, rows, torch.float32, device)
    handle = _handle(stream, device)
    if workspace is not None:
        ws = _given(workspace)
    else:
        ws = _workspace("verify", lib.tf_verify_draft_workspace_bytes(b, n), device, handle, stream)
    _check(lib.tf_verify_draft(logits.data_ptr(), code, st[0], st[1], draft, ds[0], ds[1], tokens.data_ptr(),
                               parents.data_ptr(), ps, ua, us, temperature, b, n, v, counts.data_ptr(),
                               path.data_ptr(), out.data_ptr(), logprobs.data_ptr(), ws[0], ws[1], handle),
           "tf_verify_draft")
    return counts, path, out, logprobs


def tf_kv_keep(k_cache, v_cache, page_table, lengths, path, counts, new_lengths=None, stream=None):
    """Moves the accepted path's cache rows together, in every layer (caches
    [pages, page_size, kv_heads, head_dim], or with a leading layers
    dimension). Returns the new lengths."""
    lib = _lib or _load()
    c, batch = _cache(k_cache, v_cache, page_table, lengths, layers=True)
    shape = path.shape
    if len(shape) != 2 or shape[0] != batch or not path.is_contiguous():
        raise ValueError("path must be [batch, nodes], contiguous")
    if path.dtype != torch.int32:
        raise TypeError("path must be int32")
    _int32(counts, "counts", lengths.shape)
    if new_lengths is None:
        new_lengths = _empty(stream, lengths.shape, torch.int32, lengths.device)
    else:
        _int32(new_lengths, "new_lengths", lengths.shape)
    _check(lib.tf_kv_keep(c, path.data_ptr(), counts.data_ptr(), shape[1], new_lengths.data_ptr(),
                          _handle(stream, k_cache.device)), "tf_kv_keep")
    return new_lengths
