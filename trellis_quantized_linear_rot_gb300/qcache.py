"""The operators between the qkv projection and the attention when the paged
cache is held in 4 or 8 bits (include/tf_qcache.h): queries and keys are
normed for each head and rotated by their positions, keys and values are
quantised as they are written, read back, attended to, and the accepted path
of a drafted tree is kept.

    k_cache, v_cache, scales = tf_kvq_cache(pages, page_size, kv_heads, head_dim, bits=4)
    q, k = tf_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, hadamard=True)
    tf_kvq_write(k, v, k_cache, v_cache, scales, page_table, lengths)
    out, lse = tf_kvq_attention(q, k_cache, v_cache, scales, page_table, lengths, parents)
    lengths = tf_kvq_keep(k_cache, v_cache, scales, page_table, lengths, path, counts)
    k, v = tf_kvq_read(k_cache, v_cache, scales, page_table, lengths, slots=4096, head_dim=128)

Calls are asynchronous on the current stream (or `stream=`), refuse bad
arguments before launching anything, and leave what only the device can see
(an index outside its array) to tf_device_error. Like those of spec.py they
look each attribute up once: a call of one token runs for a few microseconds.
"""

import ctypes
import struct

from . import spec
from .spec import _check, _empty, _given, _handle, _int32, _parents, _strides, _workspace

_VP, _I, _L, _D, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t


class HeadRows(ctypes.Structure):
    """tf_head_rows of tf_qcache.h."""
    _fields_ = [("x", _VP), ("y", _VP), ("weight", _VP), ("x_seq", _L), ("x_node", _L), ("x_head", _L),
                ("y_seq", _L), ("y_node", _L), ("y_head", _L), ("heads", ctypes.c_int32)]


class KVQCache(ctypes.Structure):
    """tf_kvq_cache of tf_qcache.h."""
    _fields_ = [("k", _VP), ("v", _VP), ("scales", _VP), ("stride_layer", _L), ("stride_page", _L),
                ("stride_token", _L), ("stride_head", _L), ("scale_layer", _L), ("scale_page", _L),
                ("scale_token", _L), ("scale_head", _L), ("page_table", _VP), ("lengths", _VP), ("stride_table", _L),
                ("bits", ctypes.c_int32), ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("table_width", ctypes.c_int32)]


_pack_rows = struct.Struct("@9qi4x").pack      # the fields of HeadRows, in order
_pack_cache = struct.Struct("@14q8i").pack     # and of KVQCache

NO_NORM, INTERLEAVED, HADAMARD = 1, 2, 4

# Rows and caches are passed as pointers: ctypes.byref of a structure, or its bytes.
SIGNATURES = {
    "tf_qk_norm_rope": (_I, [_VP, _VP, _I, _I, _VP, _L, _VP, _I, _D, _I, _I, _I, _I, _VP]),
    "tf_kvq_write": (_I, [_VP, _VP, _L, _L, _L, _VP, _L, _L, _L, _I, _VP, _I, _VP]),
    "tf_kvq_read": (_I, [_VP, _VP, _VP, _VP, _I, _L, _L, _L, _I, _VP]),
    "tf_kvq_attention": (_I, [_VP, _VP, _I, _L, _L, _L, _VP, _L, _VP, _VP, _I, _I, _D, _VP, _SZ, _VP]),
    "tf_kvq_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "tf_kvq_keep": (_I, [_VP, _VP, _VP, _I, _VP, _VP]),
}

_lib = torch = _codes = None


def _load():
    """The library and torch, looked up on the first call."""
    global _lib, torch, _codes
    lib = spec._load()
    torch, _codes = spec.torch, spec._codes
    _lib = lib
    return lib


def tf_kvq_cache(pages, page_size, kv_heads, head_dim, bits=4, layers=None, device="cuda"):
    """An empty cache (k_cache, v_cache, scales) of the shapes that the calls
    here take, its rows of one head and page side by side in memory: codes
    [(layers,) pages, page_size, kv_heads, head_dim * bits / 8] uint8, factors
    [(layers,) pages, page_size, kv_heads, 2] bf16."""
    if bits not in (4, 8) or head_dim not in (64, 128, 256):
        raise ValueError("a cache has 4 or 8 bits and heads of 64, 128 or 256")
    _lib or _load()
    lead = (pages,) if layers is None else (layers, pages)
    shape = lead + (kv_heads, page_size)
    k, v = (torch.zeros(shape + (head_dim * bits // 8,), dtype=torch.uint8, device=device) for _ in range(2))
    scales = torch.zeros(shape + (2,), dtype=torch.bfloat16, device=device)
    return k.transpose(-3, -2), v.transpose(-3, -2), scales.transpose(-3, -2)


def _cache(k, v, scales, page_table, lengths, head_dim, layers=False):
    """(packed tf_kvq_cache, batch) for heads of head_dim (None: whatever fits)."""
    shape, st = k.shape, k.stride()
    dims = len(shape)
    if dims != 4 and not (layers and dims == 5):
        raise ValueError("a cache is [%spages, page_size, kv_heads, bytes]" % ("layers, " if layers else ""))
    same, sc = v.stride() == st, scales.stride()
    if 1 in shape:
        st = _strides(k)
        same, sc = _strides(v) == st, _strides(scales)
    if k.dtype != torch.uint8 or v.dtype != torch.uint8 or scales.dtype != torch.bfloat16:
        raise TypeError("codes must be uint8 and scales bfloat16")
    if not same or v.shape != shape or st[-1] != 1:
        raise ValueError("k_cache and v_cache must share shape and strides, the last dimension contiguous")
    if scales.shape[:-1] != shape[:-1] or scales.shape[-1] != 2 or sc[-1] != 1:
        raise ValueError("scales must be like the codes, with a last dimension of 2, contiguous")
    width = shape[-1]
    if head_dim is None:   # only rows as a whole count
        bits, head_dim = (4, 64) if width == 32 else (8, width)
    elif width * 2 == head_dim:
        bits = 4
    elif width == head_dim:
        bits = 8
    else:
        raise ValueError("a row of %d bytes does not hold a head of %d in 4 or 8 bits" % (width, head_dim))
    int32 = torch.int32
    if page_table.dtype != int32 or lengths.dtype != int32:
        raise TypeError("page_table and lengths must be int32")
    table, rows, batch = page_table.shape, page_table.stride(), lengths.shape
    if len(batch) != 1 or not lengths.is_contiguous():
        raise ValueError("lengths must be [batch], contiguous")
    batch = batch[0]
    if len(table) != 2 or table[0] != batch or (rows[1] != 1 and table[1] > 1):
        raise ValueError("page_table must be [batch, table_width], rows contiguous")
    i = dims - 4
    packed = _pack_cache(k.data_ptr(), v.data_ptr(), scales.data_ptr(), st[0] if i else 0, st[i], st[i + 1], st[i + 2],
                         sc[0] if i else 0, sc[i], sc[i + 1], sc[i + 2], page_table.data_ptr(), lengths.data_ptr(),
                         rows[0], bits, shape[0] if i else 1, shape[i], shape[i + 1], shape[i + 2], head_dim, batch,
                         table[1])
    return packed, batch


def _code(dtype, fp32=False):
    code = _codes.get(dtype, -1)
    if code < 0 or (dtype == torch.float32 and not fp32):
        raise TypeError("unsupported dtype %s" % dtype)
    return code


def _rows(x, y, weight, batch, nodes, head_dim, dtype, name):
    """Packed tf_head_rows."""
    shape, st = x.shape, _strides(x)
    if len(shape) != 4 or shape[0] != batch or shape[1] != nodes or shape[3] != head_dim or st[3] != 1:
        raise ValueError("%s must be [batch, nodes, heads, head_dim], the last dimension contiguous" % name)
    if x.dtype != dtype:
        raise TypeError("q and k must share their dtype")
    out = st if y is x else _strides(y)
    if y.shape != shape or y.dtype != dtype or out[3] != 1:
        raise ValueError("%s_out must be of %s's shape and dtype, the last dimension contiguous" % (name, name))
    if weight is not None and (weight.shape != (head_dim,) or (weight.stride(0) != 1)):
        raise ValueError("%s_weight must be [head_dim], contiguous" % name)
    return _pack_rows(x.data_ptr(), y.data_ptr(), 0 if weight is None else weight.data_ptr(), st[0], st[1], st[2],
                      out[0], out[1], out[2], shape[2])


def tf_qk_norm_rope(q, k, positions, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                    hadamard=False, q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head, then their rotation by position
    (see tf_qk_norm_rope in tf_qcache.h).

    q: [batch, nodes, heads, head_dim], k: [batch, nodes, kv_heads, head_dim]
    or None, fp16 or bf16 (last dimension contiguous: parts of a projection's
    rows); positions int32 [batch, nodes] or [nodes], negative for rows that
    are not there; inv_freq fp64 [rotary / 2] or None for no rotation; weights
    [head_dim] or None. eps None leaves the norm out. hadamard=True rotates
    q and k over the head as well, which leaves q.k as it is and makes keys fit
    4 bits better. q_out, k_out may be q and k. Returns (q_out, k_out).
    """
    lib = _lib or _load()
    shape, dtype, device = q.shape, q.dtype, q.device
    if len(shape) != 4:
        raise ValueError("q must be [batch, nodes, heads, head_dim], the last dimension contiguous")
    b, n, _, d = shape
    if q_out is None:
        q_out = _empty(stream, shape, dtype, device)
    packed = _rows(q, q_out, q_weight, b, n, d, dtype, "q")
    weight = q_weight
    packed_k = None
    if k is not None:
        if k_out is None:
            k_out = _empty(stream, k.shape, dtype, device)
        packed_k = _rows(k, k_out, k_weight, b, n, d, dtype, "k")
        if k_weight is not None:
            if weight is not None and weight.dtype != k_weight.dtype:
                raise TypeError("q_weight and k_weight must share their dtype")
            weight = k_weight
    if positions.dtype != torch.int32:
        raise TypeError("positions must be int32")
    ps = positions.shape
    if (ps != (b, n) and ps != (n,)) or (n > 1 and positions.stride(-1) != 1):
        raise ValueError("positions must be of shape %s or %s, rows contiguous" % ((b, n), (n,)))
    rotary, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64:
            raise TypeError("inv_freq must be float64")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be [rotary / 2], contiguous")
        rotary, freq = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    flags = (NO_NORM if eps is None else 0) | (INTERLEAVED if interleaved else 0) | (HADAMARD if hadamard else 0)
    _check(lib.tf_qk_norm_rope(packed, packed_k, _code(dtype), 0 if weight is None else _code(weight.dtype, True),
                               positions.data_ptr(), 0 if len(ps) == 1 or b == 1 else positions.stride(0), freq,
                               rotary, 0.0 if eps is None else eps, flags, b, n, d, _handle(stream, device)),
           "tf_qk_norm_rope")
    return q_out, k_out


def tf_kvq_write(k_new, v_new, k_cache, v_cache, scales, page_table, lengths, counts=None, stream=None):
    """Quantises keys and values (k_new, v_new: [batch, nodes, kv_heads,
    head_dim] fp16 or bf16, last dimension contiguous) into slots lengths[b] +
    i of the cache, i < counts[b] (int32 [batch]; None: all). nodes may be a
    tree's or a part of a prompt."""
    lib = _lib or _load()
    shape = k_new.shape
    if len(shape) != 4:
        raise ValueError("k_new must be [batch, nodes, kv_heads, head_dim]")
    c, batch = _cache(k_cache, v_cache, scales, page_table, lengths, shape[3])
    st, sv = _strides(k_new), _strides(v_new)
    if v_new.shape != shape or st[3] != 1 or sv[3] != 1:
        raise ValueError("k_new and v_new must share their shape, the last dimension contiguous")
    if v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new must share their dtype")
    if shape[0] != batch or shape[2] != k_cache.shape[2]:
        raise ValueError("k_new must be [batch, nodes, kv_heads, head_dim]")
    at = None
    if counts is not None:
        _int32(counts, "counts", lengths.shape)
        at = counts.data_ptr()
    _check(lib.tf_kvq_write(c, k_new.data_ptr(), st[0], st[1], st[2], v_new.data_ptr(), sv[0], sv[1], sv[2],
                            _code(k_new.dtype), at, shape[1], _handle(stream, k_cache.device)), "tf_kvq_write")


def tf_kvq_read(k_cache, v_cache, scales, page_table, lengths, starts=None, slots=None, head_dim=None, dtype=None,
                k_out=None, v_out=None, stream=None):
    """The values of slots starts[b] + i (int32 [batch]; None: 0) below
    lengths[b], into k_out, v_out [batch, slots, kv_heads, head_dim] fp16 or
    bf16 (last dimension contiguous); rows of other slots are left as they
    were. Without outputs given, slots and head_dim say their shape, dtype
    (fp16) their type, and rows of other slots are 0. Returns (k_out, v_out)."""
    lib = _lib or _load()
    if k_out is None or v_out is None:
        if k_out is not None or v_out is not None or slots is None or head_dim is None:
            raise ValueError("give k_out and v_out, or slots and head_dim")
        shape = (lengths.shape[0], slots, k_cache.shape[2], head_dim)
        device = k_cache.device
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device):
            k_out, v_out = (torch.zeros(shape, dtype=dtype or torch.float16, device=device) for _ in range(2))
    shape = k_out.shape
    if len(shape) != 4:
        raise ValueError("k_out must be [batch, slots, kv_heads, head_dim]")
    c, batch = _cache(k_cache, v_cache, scales, page_table, lengths, shape[3])
    st = _strides(k_out)
    if v_out.shape != shape or _strides(v_out) != st or st[3] != 1:
        raise ValueError("k_out and v_out must share shape and strides, the last dimension contiguous")
    if v_out.dtype != k_out.dtype:
        raise TypeError("k_out and v_out must share their dtype")
    if shape[0] != batch or shape[2] != k_cache.shape[2]:
        raise ValueError("k_out must be [batch, slots, kv_heads, head_dim]")
    at = None
    if starts is not None:
        _int32(starts, "starts", lengths.shape)
        at = starts.data_ptr()
    _check(lib.tf_kvq_read(c, at, k_out.data_ptr(), v_out.data_ptr(), _code(k_out.dtype), st[0], st[1], st[2],
                           shape[1], _handle(stream, k_cache.device)), "tf_kvq_read")
    return k_out, v_out


def tf_kvq_attention_workspace(batch, nodes, heads, kv_heads, head_dim, device="cuda"):
    """A zeroed workspace for tf_kvq_attention calls of up to these sizes."""
    need = (_lib or _load()).tf_kvq_attention_workspace_bytes
    n = need(batch, nodes, heads, kv_heads, head_dim)
    if n:   # fewer kv heads have more rows each, and need more
        n = need(batch, nodes, heads, 1, head_dim)
    return torch.zeros(max(n, 1), dtype=torch.uint8, device=device)


def tf_kvq_attention(q, k_cache, v_cache, scales, page_table, lengths, parents, scale=None, out=None, lse=None,
                     workspace=None, stream=None):
    """Attention of the tree's nodes over a quantised cache (see
    tf_kvq_attention): tf_tree_attention with the codes and factors of
    tf_kvq_cache in the caches' place. q fp16 or bf16. Returns (out, lse)."""
    lib = _lib or _load()
    shape, dtype, device = q.shape, q.dtype, q.device
    st = _strides(q)
    if len(shape) != 4 or st[3] != 1:
        raise ValueError("q must be [batch, nodes, heads, head_dim], the last dimension contiguous")
    b, n, h, d = shape
    cache, batch = _cache(k_cache, v_cache, scales, page_table, lengths, d)
    if b != batch:
        raise ValueError("q must be [batch, nodes, heads, head_dim], the last dimension contiguous")
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
        ws = _workspace("kvq attention", lib.tf_kvq_attention_workspace_bytes(b, n, h, k_cache.shape[2], d), device,
                        handle, stream)
    _check(lib.tf_kvq_attention(cache, q.data_ptr(), _code(dtype), st[0], st[1], st[2], parents.data_ptr(), ps,
                                out.data_ptr(), lse.data_ptr(), n, h, d ** -0.5 if scale is None else scale, ws[0],
                                ws[1], handle), "tf_kvq_attention")
    return out, lse


def tf_kvq_keep(k_cache, v_cache, scales, page_table, lengths, path, counts, new_lengths=None, stream=None):
    """tf_kv_keep for a quantised cache (with or without a leading layers
    dimension). Returns the new lengths."""
    lib = _lib or _load()
    c, batch = _cache(k_cache, v_cache, scales, page_table, lengths, None, layers=True)
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
    _check(lib.tf_kvq_keep(c, path.data_ptr(), counts.data_ptr(), shape[1], new_lengths.data_ptr(),
                           _handle(stream, k_cache.device)), "tf_kvq_keep")
    return new_lengths
