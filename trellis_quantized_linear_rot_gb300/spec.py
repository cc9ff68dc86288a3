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
"""

import ctypes

TF_MAX_NODES = 128

_VP, _I, _L, _D, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t


class KVCache(ctypes.Structure):
    """tf_kv_cache of tf_spec.h."""
    _fields_ = [("k", _VP), ("v", _VP), ("stride_layer", _L), ("stride_page", _L), ("stride_token", _L),
                ("stride_head", _L), ("page_table", _VP), ("lengths", _VP), ("stride_table", _L),
                ("dtype", ctypes.c_int32), ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("table_width", ctypes.c_int32)]


_C = ctypes.POINTER(KVCache)
SIGNATURES = {
    "tf_kv_write": (_I, [_C, _VP, _VP, _L, _L, _L, _I, _VP]),
    "tf_tree_attention": (_I, [_C, _VP, _L, _L, _L, _VP, _L, _VP, _VP, _I, _I, _D, _VP, _SZ, _VP]),
    "tf_tree_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "tf_verify_draft": (_I, [_VP, _I, _L, _L, _VP, _L, _L, _VP, _VP, _L, _VP, _VP, _D, _I, _I, _I, _VP, _VP, _VP, _VP,
                             _VP, _SZ, _VP]),
    "tf_verify_draft_workspace_bytes": (_SZ, [_I, _I]),
    "tf_kv_keep": (_I, [_C, _VP, _VP, _I, _VP, _VP]),
}

_workspaces = {}


def _bind():
    """The package's own helpers (imported late: the package imports this module)."""
    import trellis_quantized_linear_rot_gb300 as tf
    return tf


def _strides(t):
    """Strides, 0 for a dimension of one element (its stride means nothing)."""
    return tuple(0 if n == 1 else st for n, st in zip(t.shape, t.stride()))


def _int32(t, name, shape):
    import torch
    if t.dtype != torch.int32:
        raise TypeError("%s must be int32" % name)
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous and of shape %s" % (name, shape))


def _parents(parents, batch, nodes):
    """Row stride of parents: [batch, nodes], or one [nodes] for all sequences."""
    import torch
    if parents.dtype != torch.int32:
        raise TypeError("parents must be int32")
    if tuple(parents.shape) not in ((nodes,), (batch, nodes)) or (nodes > 1 and parents.stride(-1) != 1):
        raise ValueError("parents must be of shape %s or %s, rows contiguous" % ((batch, nodes), (nodes,)))
    return 0 if parents.dim() == 1 or batch == 1 else parents.stride(0)


def _cache(tf, k, v, page_table, lengths, layers=False):
    import torch
    if k.dim() != 4 and not (layers and k.dim() == 5):
        raise ValueError("a cache is [%spages, page_size, kv_heads, head_dim]" % ("layers, " if layers else ""))
    st = _strides(k)
    if k.shape != v.shape or st != _strides(v) or k.dtype != v.dtype or st[-1] != 1:
        raise ValueError("k_cache and v_cache must share shape, strides and dtype, the last dimension contiguous")
    if page_table.dtype != torch.int32 or lengths.dtype != torch.int32:
        raise TypeError("page_table and lengths must be int32")
    batch = lengths.shape[0]
    if page_table.dim() != 2 or page_table.shape[0] != batch or page_table.stride(1) != 1 and page_table.shape[1] > 1:
        raise ValueError("page_table must be [batch, table_width], rows contiguous")
    if lengths.dim() != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be [batch], contiguous")
    return KVCache(k.data_ptr(), v.data_ptr(), st[0] if k.dim() == 5 else 0, st[-4], st[-3], st[-2],
                   page_table.data_ptr(), lengths.data_ptr(), page_table.stride(0), tf._dtype_code(k.dtype),
                   k.shape[0] if k.dim() == 5 else 1, k.shape[-4], k.shape[-3], k.shape[-2], k.shape[-1], batch,
                   page_table.shape[1])


def _workspace(given, name, nbytes, device, stream):
    """The caller's workspace, or one the binding keeps for the stream. While a
    graph is being captured each call gets its own (its zeroing is captured
    too), since a kept one could outlive the graph's memory."""
    import torch
    if given is not None:
        return given
    if torch.cuda.is_current_stream_capturing():
        with torch.cuda.stream(stream):
            return torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device)
    key = (name, device.index, stream.cuda_stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.stream(stream):
            ws = _workspaces[key] = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device)
    return ws


def forget_workspaces():
    """Drops the workspaces kept by the binding (after an aborted kernel they
    are made anew, zeroed)."""
    _workspaces.clear()


def tf_kv_write(k_new, v_new, k_cache, v_cache, page_table, lengths, stream=None):
    """Writes the tree's keys and values (k_new, v_new: [batch, nodes, kv_heads,
    head_dim], any strides with the last dimension contiguous) into slots
    lengths[b] + i of the cache [pages, page_size, kv_heads, head_dim]."""
    tf = _bind()
    c = _cache(tf, k_cache, v_cache, page_table, lengths)
    st = _strides(k_new)
    if k_new.shape != v_new.shape or st != _strides(v_new) or st[-1] != 1:
        raise ValueError("k_new and v_new must share shape and strides, the last dimension contiguous")
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype:
        raise TypeError("k_new and v_new must have the cache's dtype")
    if k_new.dim() != 4 or k_new.shape[0] != c.batch or tuple(k_new.shape[2:]) != tuple(k_cache.shape[2:]):
        raise ValueError("k_new must be [batch, nodes, kv_heads, head_dim]")
    tf._check(tf.lib().tf_kv_write(c, k_new.data_ptr(), v_new.data_ptr(), st[0], st[1], st[2], k_new.shape[1],
                                   tf._stream(stream)), "tf_kv_write")


def tf_tree_attention_workspace(batch, nodes, heads, kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for tf_tree_attention calls of up to these sizes."""
    import torch
    n = _bind().lib().tf_tree_attention_workspace_bytes(batch, nodes, heads, kv_heads, head_dim)
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
    import torch
    tf = _bind()
    c = _cache(tf, k_cache, v_cache, page_table, lengths)
    if q.dtype != k_cache.dtype:
        raise TypeError("q must have the cache's dtype")
    if q.dim() != 4 or q.shape[0] != c.batch or q.shape[3] != c.head_dim or q.stride(-1) != 1:
        raise ValueError("q must be [batch, nodes, heads, head_dim], the last dimension contiguous")
    b, n, h, d = q.shape
    ps = _parents(parents, b, n)
    if stream is None:
        stream = torch.cuda.current_stream()
    if out is None:
        out = torch.empty((b, n, h, d), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((b, n, h), dtype=torch.float32, device=q.device)
    if tuple(out.shape) != (b, n, h, d) or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape and dtype")
    if tuple(lse.shape) != (b, n, h) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [batch, nodes, heads]")
    need = tf.lib().tf_tree_attention_workspace_bytes(b, n, h, c.kv_heads, d)
    ws = _workspace(workspace, "attention", need, q.device, stream)
    st = _strides(q)
    tf._check(tf.lib().tf_tree_attention(c, q.data_ptr(), st[0], st[1], st[2], parents.data_ptr(), ps, out.data_ptr(),
                                         lse.data_ptr(), n, h, d ** -0.5 if scale is None else scale, ws.data_ptr(),
                                         ws.numel() * ws.element_size(), stream.cuda_stream), "tf_tree_attention")
    return out, lse


def tf_verify_draft_workspace(batch, nodes, device="cuda"):
    """A zeroed workspace for tf_verify_draft calls of up to these sizes."""
    import torch
    n = _bind().lib().tf_verify_draft_workspace_bytes(batch, nodes)
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
    import torch
    tf = _bind()
    if logits.dim() != 3 or (logits.shape[2] > 1 and logits.stride(2) != 1):
        raise ValueError("logits must be [batch, nodes, vocab], the last dimension contiguous")
    b, n, v = logits.shape
    _int32(tokens, "tokens", (b, n))
    ps = _parents(parents, b, n)
    ds = (0, 0)
    if draft_logits is not None:
        if draft_logits.shape != logits.shape or draft_logits.dtype != logits.dtype or \
                (v > 1 and draft_logits.stride(2) != 1):
            raise ValueError("draft_logits must be like logits, the last dimension contiguous")
        ds = _strides(draft_logits)
    for t, name in ((u_sample, "u_sample"), (u_accept, "u_accept")):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (b, n) or not t.is_contiguous()):
            raise ValueError("%s must be contiguous fp32 [batch, nodes]" % name)
    if stream is None:
        stream = torch.cuda.current_stream()
    dev = logits.device
    counts = torch.empty((b,), dtype=torch.int32, device=dev)
    path = torch.empty((b, n), dtype=torch.int32, device=dev)
    out = torch.empty((b, n), dtype=torch.int32, device=dev)
    logprobs = torch.empty((b, n), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, "verify", tf.lib().tf_verify_draft_workspace_bytes(b, n), dev, stream)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = _strides(logits)
    tf._check(tf.lib().tf_verify_draft(logits.data_ptr(), tf._dtype_code(logits.dtype), st[0], st[1],
                                       ptr(draft_logits), ds[0], ds[1], tokens.data_ptr(), parents.data_ptr(), ps,
                                       ptr(u_accept), ptr(u_sample), temperature, b, n, v, counts.data_ptr(),
                                       path.data_ptr(), out.data_ptr(), logprobs.data_ptr(), ws.data_ptr(),
                                       ws.numel() * ws.element_size(), stream.cuda_stream), "tf_verify_draft")
    return counts, path, out, logprobs


def tf_kv_keep(k_cache, v_cache, page_table, lengths, path, counts, new_lengths=None, stream=None):
    """Moves the accepted path's cache rows together, in every layer (caches
    [pages, page_size, kv_heads, head_dim], or with a leading layers
    dimension). Returns the new lengths."""
    import torch
    tf = _bind()
    c = _cache(tf, k_cache, v_cache, page_table, lengths, layers=True)
    if path.dim() != 2:
        raise ValueError("path must be [batch, nodes]")
    _int32(path, "path", (c.batch, path.shape[1]))
    _int32(counts, "counts", (c.batch,))
    if new_lengths is None:
        new_lengths = torch.empty_like(lengths)
    _int32(new_lengths, "new_lengths", (c.batch,))
    tf._check(tf.lib().tf_kv_keep(c, path.data_ptr(), counts.data_ptr(), path.shape[1], new_lengths.data_ptr(),
                                  tf._stream(stream)), "tf_kv_keep")
    return new_lengths
