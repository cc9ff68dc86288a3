"""Host-side checks of the entry points of tf_spec.h that need no GPU: each
refuses bad arguments with the documented status before it makes any CUDA
call, and empty batches touch nothing."""

import ctypes
import os

import pytest

import trellis_quantized_linear_rot_gb300 as tf
from trellis_quantized_linear_rot_gb300.spec import KVCache

P, MIS, NUL = 0x10000, 0x10008, None
S = None


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tf.library_path()):
        from trellis_quantized_linear_rot_gb300 import build
        build.build()
    return tf.lib()


def cache(**kw):
    f = dict(k=P, v=P, stride_layer=0, stride_page=16384, stride_token=1024, stride_head=128, page_table=P, lengths=P,
             stride_table=4, dtype=tf.TF_F16, layers=1, pages=8, page_size=16, kv_heads=8, head_dim=128, batch=2,
             table_width=4)
    f.update(kw)
    return KVCache(**f)


BAD_CACHES = [
    (dict(batch=-1), tf.TF_ERR_SHAPE), (dict(batch=65536), tf.TF_ERR_SHAPE), (dict(layers=0), tf.TF_ERR_SHAPE),
    (dict(pages=0), tf.TF_ERR_SHAPE), (dict(page_size=0), tf.TF_ERR_SHAPE), (dict(kv_heads=0), tf.TF_ERR_SHAPE),
    (dict(head_dim=0), tf.TF_ERR_SHAPE), (dict(head_dim=100), tf.TF_ERR_SHAPE), (dict(table_width=0), tf.TF_ERR_SHAPE),
    (dict(table_width=1 << 28), tf.TF_ERR_SHAPE), (dict(stride_page=-8), tf.TF_ERR_SHAPE),
    (dict(stride_table=-1), tf.TF_ERR_SHAPE), (dict(dtype=tf.TF_F32), tf.TF_ERR_DTYPE), (dict(dtype=5), tf.TF_ERR_DTYPE),
    (dict(k=NUL), tf.TF_ERR_NULL), (dict(v=NUL), tf.TF_ERR_NULL), (dict(page_table=NUL), tf.TF_ERR_NULL),
    (dict(lengths=NUL), tf.TF_ERR_NULL), (dict(k=MIS), tf.TF_ERR_ALIGN), (dict(v=MIS), tf.TF_ERR_ALIGN),
    (dict(stride_token=1028), tf.TF_ERR_ALIGN), (dict(stride_head=129), tf.TF_ERR_ALIGN),
    (dict(lengths=0x10002), tf.TF_ERR_ALIGN)]


def byref(c):
    return None if c is None else ctypes.byref(c)


def write(lib, c, k=P, v=P, st=(1024, 1024, 128), n=3):
    return lib.tf_kv_write(byref(c), k, v, *st, n, S)


def attend(lib, c, q=P, st=(40960, 5120, 128), par=P, sp=3, out=P, lse=P, n=3, h=40, scale=0.1, ws=P, nb=1 << 40):
    return lib.tf_tree_attention(byref(c), q, *st, par, sp, out, lse, n, h, scale, ws, nb, S)


def keep(lib, c, path=P, counts=P, n=3, new=0x20000):
    return lib.tf_kv_keep(byref(c), path, counts, n, new, S)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_operator_refuses_a_bad_cache(lib, bad, status):
    c = cache(**bad)
    for f in (write, attend, keep):
        assert f(lib, c) == status, f.__name__


def test_write_refusals(lib):
    assert write(lib, None) == tf.TF_ERR_NULL
    assert write(lib, cache(layers=2)) == tf.TF_ERR_SHAPE
    assert write(lib, cache(), n=-1) == tf.TF_ERR_SHAPE
    assert write(lib, cache(), n=129) == tf.TF_ERR_SHAPE
    assert write(lib, cache(), st=(-8, 1024, 128)) == tf.TF_ERR_SHAPE
    assert write(lib, cache(), k=NUL) == write(lib, cache(), v=NUL) == tf.TF_ERR_NULL
    assert write(lib, cache(), k=MIS) == write(lib, cache(), st=(1024, 1020, 128)) == tf.TF_ERR_ALIGN
    assert write(lib, cache(batch=0, k=NUL), k=NUL) == tf.TF_OK
    assert write(lib, cache(), n=0, k=NUL) == tf.TF_OK


def test_attention_refusals(lib):
    assert attend(lib, None) == tf.TF_ERR_NULL
    assert attend(lib, cache(layers=2)) == tf.TF_ERR_SHAPE
    for d in (8, 96, 512):
        assert attend(lib, cache(head_dim=d)) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), h=41) == attend(lib, cache(), h=0) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), n=129) == attend(lib, cache(), n=-1) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), st=(-8, 0, 0)) == attend(lib, cache(), sp=-1) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), scale=float("inf")) == attend(lib, cache(), scale=float("nan")) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(batch=65535), n=128, h=40) == tf.TF_ERR_SHAPE       # too many rows
    assert attend(lib, cache(batch=1000, table_width=1 << 20), n=1) == tf.TF_ERR_SHAPE   # too many tiles to number
    for k in ("q", "par", "out", "lse", "ws"):
        assert attend(lib, cache(), **{k: NUL}) == tf.TF_ERR_NULL, k
    for k in ("q", "out", "ws"):
        assert attend(lib, cache(), **{k: MIS}) == tf.TF_ERR_ALIGN, k
    assert attend(lib, cache(), st=(40960, 5121, 128)) == tf.TF_ERR_ALIGN
    assert attend(lib, cache(batch=0), q=NUL) == attend(lib, cache(), n=0, q=NUL) == tf.TF_OK
    f = lib.tf_tree_attention_workspace_bytes
    assert f(-1, 1, 8, 8, 64) == f(1, 129, 8, 8, 64) == f(1, 1, 9, 8, 64) == f(1, 1, 8, 8, 96) == 0


def test_attention_refuses_a_scale_that_fp32_cannot_hold(lib):
    for scale in (1e39, -1e39, 1e300, 3.4e38, -2.4e38):   # the last two times log2(e) = 1.44
        assert attend(lib, cache(), scale=scale) == tf.TF_ERR_SHAPE, scale
    for scale in (2.3e38, -2.3e38, 0.0, 1e-45, -1e-300):
        assert attend(lib, cache(), scale=scale) != tf.TF_ERR_SHAPE, scale


def test_keep_refusals(lib):
    assert keep(lib, None) == tf.TF_ERR_NULL
    assert keep(lib, cache(), n=0) == keep(lib, cache(), n=200) == tf.TF_ERR_SHAPE
    for k in ("path", "counts", "new"):
        assert keep(lib, cache(), **{k: NUL}) == tf.TF_ERR_NULL, k
        assert keep(lib, cache(), **{k: 0x20002}) == tf.TF_ERR_ALIGN, k
    assert keep(lib, cache(), new=P) == keep(lib, cache(), new=P + 4) == tf.TF_ERR_POINTER   # lengths themselves
    assert keep(lib, cache(batch=0), path=NUL) == tf.TF_OK


def test_keep_refuses_new_lengths_over_what_its_blocks_read(lib):
    """Every block of a sequence reads its length, count, path and pages, and
    one of them writes the new length."""
    c = cache(page_table=0x30000, lengths=0x40000)     # 2 sequences, 4 pages each
    call = lambda new: keep(lib, c, path=0x50000, counts=0x60000, new=new)  # noqa: E731
    for begin, size in ((0x30000, 2 * 4 * 4), (0x40000, 2 * 4), (0x50000, 2 * 3 * 4), (0x60000, 2 * 4)):
        for new in (begin - 4, begin, begin + size - 4):
            assert call(new) == tf.TF_ERR_POINTER, hex(new)
    wide = cache(page_table=0x30000, lengths=0x40000, stride_table=100)
    assert keep(lib, wide, path=0x50000, counts=0x60000, new=0x30000 + 103 * 4) == tf.TF_ERR_POINTER
    import torch
    if not torch.cuda.is_available():
        for begin, size in ((0x30000, 2 * 4 * 4), (0x40000, 2 * 4), (0x50000, 2 * 3 * 4), (0x60000, 2 * 4)):
            for new in (begin - 8, begin + size):
                assert call(new) == tf.TF_ERR_CUDA, hex(new)   # past the checks


def test_verify_refusals(lib):
    def v(logits=P, dt=tf.TF_F32, st=(400, 100), draft=P, dst=(400, 100), tok=P, par=P, sp=4, ua=P, us=P, t=1.0, b=2,
          n=4, vocab=100, counts=P, path=P, out=P, lp=P, ws=P, nb=1 << 40):
        return lib.tf_verify_draft(logits, dt, *st, draft, *dst, tok, par, sp, ua, us, t, b, n, vocab, counts, path,
                                   out, lp, ws, nb, S)
    for bad in (dict(b=-1), dict(b=65536), dict(n=0), dict(n=129), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                dict(st=(-1, 0)), dict(dst=(0, -1)), dict(sp=-1), dict(t=-0.5), dict(t=float("nan")),
                dict(t=float("inf")), dict(t=1e-39)):
        assert v(**bad) == tf.TF_ERR_SHAPE, bad
    assert v(dt=3) == tf.TF_ERR_DTYPE
    for k in ("logits", "tok", "par", "ua", "us", "counts", "path", "out", "lp", "ws"):
        assert v(**{k: NUL}) == tf.TF_ERR_NULL, k
    for k in ("logits", "draft", "tok", "par", "ua", "us", "counts", "path", "out", "lp"):
        assert v(**{k: 0x10002}) == tf.TF_ERR_ALIGN, k
    assert v(ws=MIS) == tf.TF_ERR_ALIGN
    assert v(b=0, logits=NUL) == tf.TF_OK
    f = lib.tf_verify_draft_workspace_bytes
    assert f(-1, 4) == f(1, 0) == f(1, 129) == 0


def test_verify_refuses_a_temperature_whose_reciprocal_fp32_cannot_hold(lib):
    def v(t):
        return lib.tf_verify_draft(P, tf.TF_F32, 400, 100, None, 0, 0, P, P, 4, None, P, t, 2, 4, 100, P, P, P, P, P,
                                   1 << 40, S)
    for t in (1e-39, 1e-300, 1e46, 1e300):     # infinite, or 0, which makes an infinite logit a NaN
        assert v(t) == tf.TF_ERR_SHAPE, t
    for t in (0.0, 3e-39, 1.0, 1e38, 1e44):
        assert v(t) != tf.TF_ERR_SHAPE, t


def test_without_gpu_valid_calls_fail_cleanly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (write, attend, keep):
        assert f(lib, cache()) in (tf.TF_ERR_CUDA, tf.TF_ERR_POINTER)


def test_status_text(lib):
    assert lib.tf_status_string(tf.TF_ERR_INDEX).decode() not in ("", "unknown status")
    assert ctypes.sizeof(KVCache) == 104


def test_the_bindings_bytes_are_the_structure():
    from trellis_quantized_linear_rot_gb300 import spec
    values = [0x1000, 0x2000, 3, 4, 5, 6, 0x7000, 0x8000, 9, 10, 11, 12, 13, 14, 15, 16, 17]
    assert spec._pack_cache(*values) == bytes(KVCache(*values))
