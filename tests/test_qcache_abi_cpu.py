"""Host-side checks of the entry points of tf_qcache.h that need no GPU: each
refuses bad arguments with the documented status before it makes any CUDA
call, and empty batches touch nothing. The binding refuses bad tensors."""

import ctypes
import os

import numpy as np
import pytest

import qcache_oracle as qo
import trellis_quantized_linear_rot_gb300 as tf
from trellis_quantized_linear_rot_gb300 import qcache
from trellis_quantized_linear_rot_gb300.qcache import HeadRows, KVQCache

P, MIS, NUL = 0x10000, 0x10008, None
S = None


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tf.library_path()):
        from trellis_quantized_linear_rot_gb300 import build
        build.build()
    return tf.lib()


def cache(**kw):
    f = dict(k=P, v=P, scales=P, stride_layer=0, stride_page=8192, stride_token=512, stride_head=64, scale_layer=0,
             scale_page=256, scale_token=16, scale_head=2, page_table=P, lengths=P, stride_table=4, bits=4, layers=1,
             pages=8, page_size=16, kv_heads=8, head_dim=128, batch=2, table_width=4)
    f.update(kw)
    return KVQCache(**f)


BAD_CACHES = [
    (dict(batch=-1), tf.TF_ERR_SHAPE), (dict(batch=65536), tf.TF_ERR_SHAPE), (dict(layers=0), tf.TF_ERR_SHAPE),
    (dict(pages=0), tf.TF_ERR_SHAPE), (dict(page_size=0), tf.TF_ERR_SHAPE), (dict(kv_heads=0), tf.TF_ERR_SHAPE),
    (dict(head_dim=0), tf.TF_ERR_SHAPE), (dict(head_dim=96), tf.TF_ERR_SHAPE), (dict(head_dim=512), tf.TF_ERR_SHAPE),
    (dict(table_width=0), tf.TF_ERR_SHAPE), (dict(table_width=1 << 28), tf.TF_ERR_SHAPE),
    (dict(stride_page=-16), tf.TF_ERR_SHAPE), (dict(scale_token=-2), tf.TF_ERR_SHAPE), (dict(stride_table=-1), tf.TF_ERR_SHAPE),
    (dict(bits=3), tf.TF_ERR_BITS), (dict(bits=16), tf.TF_ERR_BITS), (dict(k=NUL), tf.TF_ERR_NULL),
    (dict(v=NUL), tf.TF_ERR_NULL), (dict(scales=NUL), tf.TF_ERR_NULL), (dict(page_table=NUL), tf.TF_ERR_NULL),
    (dict(lengths=NUL), tf.TF_ERR_NULL), (dict(k=MIS), tf.TF_ERR_ALIGN), (dict(v=MIS), tf.TF_ERR_ALIGN),
    (dict(scales=0x10002), tf.TF_ERR_ALIGN), (dict(stride_token=520), tf.TF_ERR_ALIGN), (dict(stride_head=72), tf.TF_ERR_ALIGN),
    (dict(scale_head=3), tf.TF_ERR_ALIGN), (dict(lengths=0x10002), tf.TF_ERR_ALIGN)]


def byref(c):
    return None if c is None else ctypes.byref(c)


def write(lib, c, k=P, v=P, dt=tf.TF_F16, st=(1024, 1024, 128), sv=(2048, 2048, 128), counts=P,
          n=3):
    return lib.tf_kvq_write(byref(c), k, *st, v, *sv, dt, counts, n, S)


def read(lib, c, starts=P, k=P, v=P, dt=tf.TF_BF16, st=(1024, 1024, 128), n=3):
    return lib.tf_kvq_read(byref(c), starts, k, v, dt, *st, n, S)


def attend(lib, c, q=P, dt=tf.TF_F16, st=(40960, 5120, 128), par=P, sp=3, out=P, lse=P, n=3, h=40, scale=0.1, ws=P,
           nb=1 << 40):
    return lib.tf_kvq_attention(byref(c), q, dt, *st, par, sp, out, lse, n, h, scale, ws, nb, S)


def keep(lib, c, path=P, counts=P, n=3, new=0x20000):
    return lib.tf_kvq_keep(byref(c), path, counts, n, new, S)


def rows(**kw):
    f = dict(x=P, y=P, weight=P, x_seq=4096, x_node=1024, x_head=128, y_seq=4096, y_node=1024, y_head=128, heads=8)
    f.update(kw)
    return HeadRows(**f)


def norm(lib, q, k, dt=tf.TF_F16, wdt=tf.TF_F16, pos=P, sp=4, freq=P, rotary=128, eps=1e-6, flags=0, b=2, n=4, d=128):
    return lib.tf_qk_norm_rope(byref(q), byref(k), dt, wdt, pos, sp, freq, rotary, eps, flags, b, n, d, S)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_operator_refuses_a_bad_cache(lib, bad, status):
    c = cache(**bad)
    for f in (write, read, attend, keep):
        assert f(lib, c) == status, f.__name__


def test_norm_refusals(lib):
    assert norm(lib, None, rows()) == tf.TF_ERR_NULL
    for bad in (dict(heads=0), dict(heads=65536), dict(x_seq=-8), dict(y_node=-8)):
        assert norm(lib, rows(**bad), rows()) == norm(lib, rows(), rows(**bad)) == tf.TF_ERR_SHAPE, bad
    for bad in (dict(b=-1), dict(n=-1), dict(d=96), dict(d=512), dict(rotary=-16), dict(rotary=24), dict(rotary=144),
                dict(sp=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(flags=8),
                dict(flags=-1), dict(b=1 << 16, n=1 << 16)):
        assert norm(lib, rows(), rows(), **bad) == tf.TF_ERR_SHAPE, bad
    assert norm(lib, rows(), rows(), dt=tf.TF_F32) == norm(lib, rows(), rows(), wdt=5) == tf.TF_ERR_DTYPE
    for k in ("x", "y"):
        assert norm(lib, rows(**{k: NUL}), rows()) == norm(lib, rows(), rows(**{k: NUL})) == tf.TF_ERR_NULL, k
        assert norm(lib, rows(**{k: MIS}), rows()) == norm(lib, rows(), rows(**{k: MIS})) == tf.TF_ERR_ALIGN, k
    assert norm(lib, rows(), rows(), pos=NUL) == norm(lib, rows(), rows(), freq=NUL) == tf.TF_ERR_NULL
    assert norm(lib, rows(), rows(), pos=0x10002) == norm(lib, rows(), rows(), freq=0x10004) == tf.TF_ERR_ALIGN
    assert norm(lib, rows(weight=0x10001), rows()) == norm(lib, rows(weight=0x10002), rows(), wdt=tf.TF_F32) == tf.TF_ERR_ALIGN
    assert norm(lib, rows(x_head=132), rows()) == norm(lib, rows(), rows(y_seq=4100)) == tf.TF_ERR_ALIGN
    assert norm(lib, rows(x=NUL), rows(), b=0) == norm(lib, rows(x=NUL), None, n=0) == tf.TF_OK


def test_write_and_read_refusals(lib):
    for f in (write, read):
        assert f(lib, None) == tf.TF_ERR_NULL
        assert f(lib, cache(layers=2)) == f(lib, cache(), n=-1) == f(lib, cache(), st=(-8, 1024, 128)) == tf.TF_ERR_SHAPE
        assert f(lib, cache(batch=60000), n=1 << 20) == tf.TF_ERR_SHAPE
        assert f(lib, cache(), dt=tf.TF_F32) == f(lib, cache(), dt=7) == tf.TF_ERR_DTYPE
        assert f(lib, cache(), k=NUL) == f(lib, cache(), v=NUL) == tf.TF_ERR_NULL
        assert f(lib, cache(), k=MIS) == f(lib, cache(), v=MIS) == f(lib, cache(), st=(1024, 1020, 128)) == tf.TF_ERR_ALIGN
        assert f(lib, cache(batch=0, k=NUL), k=NUL) == f(lib, cache(), n=0, k=NUL) == tf.TF_OK
    assert write(lib, cache(), sv=(8, -8, 0)) == tf.TF_ERR_SHAPE and write(lib, cache(), sv=(8, 4, 0)) == tf.TF_ERR_ALIGN
    assert write(lib, cache(), counts=0x10002) == read(lib, cache(), starts=0x10002) == tf.TF_ERR_ALIGN


def test_attention_refusals(lib):
    assert attend(lib, None) == tf.TF_ERR_NULL
    assert attend(lib, cache(layers=2)) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), h=41) == attend(lib, cache(), h=0) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), n=129) == attend(lib, cache(), n=-1) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), st=(-8, 0, 0)) == attend(lib, cache(), sp=-1) == tf.TF_ERR_SHAPE
    for scale in (float("inf"), float("nan"), 1e39, -2.4e38):
        assert attend(lib, cache(), scale=scale) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(batch=65535), n=128, h=40) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(batch=1000, table_width=1 << 20), n=1) == tf.TF_ERR_SHAPE
    assert attend(lib, cache(), dt=tf.TF_F32) == tf.TF_ERR_DTYPE
    for k in ("q", "par", "out", "lse", "ws"):
        assert attend(lib, cache(), **{k: NUL}) == tf.TF_ERR_NULL, k
    for k in ("q", "out", "ws"):
        assert attend(lib, cache(), **{k: MIS}) == tf.TF_ERR_ALIGN, k
    assert attend(lib, cache(), st=(40960, 5121, 128)) == tf.TF_ERR_ALIGN
    assert attend(lib, cache(batch=0), q=NUL) == attend(lib, cache(), n=0, q=NUL) == tf.TF_OK
    f = lib.tf_kvq_attention_workspace_bytes
    assert f(-1, 1, 8, 8, 64) == f(1, 129, 8, 8, 64) == f(1, 1, 9, 8, 64) == f(1, 1, 8, 8, 96) == 0


def test_keep_refusals(lib):
    assert keep(lib, None) == tf.TF_ERR_NULL
    assert keep(lib, cache(), n=0) == keep(lib, cache(), n=200) == tf.TF_ERR_SHAPE
    for k in ("path", "counts", "new"):
        assert keep(lib, cache(), **{k: NUL}) == tf.TF_ERR_NULL, k
        assert keep(lib, cache(), **{k: 0x20002}) == tf.TF_ERR_ALIGN, k
    c = cache(page_table=0x30000, lengths=0x40000)     # 2 sequences, 4 pages each
    for begin, size in ((0x30000, 2 * 4 * 4), (0x40000, 2 * 4), (0x50000, 2 * 3 * 4), (0x60000, 2 * 4)):
        for new in (begin - 4, begin, begin + size - 4):
            assert keep(lib, c, path=0x50000, counts=0x60000, new=new) == tf.TF_ERR_POINTER, hex(new)
    assert keep(lib, cache(batch=0), path=NUL) == tf.TF_OK


def test_without_gpu_valid_calls_fail_cleanly(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (write, read, attend, keep):
        assert f(lib, cache()) in (tf.TF_ERR_CUDA, tf.TF_ERR_POINTER)
    assert norm(lib, rows(), rows()) in (tf.TF_ERR_CUDA, tf.TF_ERR_POINTER)
    assert norm(lib, rows(), None, freq=NUL, rotary=0) in (tf.TF_ERR_CUDA, tf.TF_ERR_POINTER)


def test_the_bindings_bytes_are_the_structures():
    values = list(range(0x1000, 0x1000 + 22))
    assert qcache._pack_cache(*values) == bytes(KVQCache(*values)) and ctypes.sizeof(KVQCache) == 144
    assert qcache._pack_rows(*values[:10]) == bytes(HeadRows(*values[:10])) and ctypes.sizeof(HeadRows) == 80


def test_the_binding_refuses_tensors_that_do_not_fit():
    import torch
    k, v, s = tf.tf_kvq_cache(6, 16, 2, 128, bits=4, device="cpu")
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    new = torch.zeros((2, 3, 2, 128), dtype=torch.float16)
    ok = dict(k_new=new, v_new=new, k_cache=k, v_cache=v, scales=s, page_table=table, lengths=lens)

    def call(**kw):
        return tf.tf_kvq_write(**{**ok, **kw})

    for kw in (dict(k_new=new.float(), v_new=new.float()), dict(v_new=new.bfloat16()), dict(scales=s.half()),
               dict(k_cache=k.to(torch.int32), v_cache=v.to(torch.int32)), dict(lengths=lens.long()),
               dict(counts=lens.long())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(k_new=new[..., :64], v_new=new[..., :64], k_cache=k[..., :24], v_cache=v[..., :24]),
               dict(k_new=new[:1], v_new=new[:1]), dict(v_new=new[:, :2]), dict(scales=s[:4]), dict(scales=s[..., :1]),
               dict(v_cache=v.contiguous()), dict(k_cache=k[0], v_cache=v[0]), dict(page_table=table[:1]),
               dict(counts=torch.zeros(3, dtype=torch.int32)), dict(k_new=new[0], v_new=new[0])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(), dict(slots=4), dict(k_out=new)):
        with pytest.raises(ValueError):
            tf.tf_kvq_read(k, v, s, table, lens, **kw)
    for kw in (dict(bits=3), dict(head_dim=96)):
        with pytest.raises(ValueError):
            tf.tf_kvq_cache(2, 16, 1, **{"head_dim": 128, **kw}, device="cpu")
    pos, freq = torch.zeros((2, 3), dtype=torch.int32), torch.ones(64, dtype=torch.float64)
    for kw in (dict(positions=pos.long()), dict(inv_freq=freq.float()), dict(k=new.bfloat16()),
               dict(q_weight=torch.ones(128).half(), k_weight=torch.ones(128))):
        with pytest.raises(TypeError):
            tf.tf_qk_norm_rope(**{**dict(q=new, k=new, positions=pos, inv_freq=freq, q_out=new, k_out=new), **kw})
    for kw in (dict(positions=pos[:1]), dict(inv_freq=freq[::2]), dict(k=new[:, :2]), dict(q_out=new[:1]),
               dict(q_weight=torch.ones(64)), dict(q=new[0])):
        with pytest.raises(ValueError):
            tf.tf_qk_norm_rope(**{**dict(q=new, k=new, positions=pos, inv_freq=freq, q_out=new, k_out=new), **kw})


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_pins(bits):
    """The oracle itself, on rows worked out by hand."""
    most = 7 if bits == 4 else 127
    x = np.zeros((5, 64))
    x[0, :4] = [most, -most, 0.5, 1.5]          # s = 1: ties go to even
    x[1, 0], x[1, 1] = np.inf, 3.0
    x[2, 5] = np.nan
    x[4, :2] = [most * 2.0, 1.0]                # s = 2: 0.5 is a tie
    c, s = qo.quantise(x, bits)
    assert c[0, :4].tolist() == [most, -most, 0, 2] and s[0] == 1
    assert np.isnan(s[1]) and np.isnan(s[2]) and not c[1:3].any()
    assert s[3] == 0 and not c[3].any() and s[4] == 2 and c[4, 1] == 0
    assert np.array_equal(qo.unpack(qo.pack(c, bits), bits), c)
    assert qo.to_bf16(np.float32(1.00390625)) == 1.0 and qo.to_bf16(np.float32(1.01171875)) == np.float32(1.015625)


def test_a_quotient_is_no_tie_by_less_than_the_kernel_can_tell():
    """x of 11 bits, s of 8: x / s below 128 is exactly halfway between whole
    numbers or at least 2^-12 away from it, and x times 1 / s (fp32, off by a
    unit in its last place either way), rounded to a multiple of 2^-13, rounds
    to the same whole number as the quotient does: over all mantissas, in the
    order of the kernel's steps."""
    f = np.float32
    big = f(1536.0)
    mant_x = np.arange(1024, 2048, dtype=np.int64)
    for mant_s in range(128, 256):
        for e in range(-11, 8):
            q = mant_x * 2.0 ** e / mant_s
            use = q < 127.5
            if not use.any():
                continue
            x, s = (mant_x * 2.0 ** e)[use], float(mant_s)
            off = np.abs(q[use] - np.floor(q[use]) - 0.5)
            assert np.all((off == 0) | (off >= 2.0 ** -12))
            inv = f(1) / f(s)
            for r in (inv, np.nextafter(inv, f(0)), np.nextafter(inv, f(1))):
                t = (x.astype(f) * r + big) - big
                assert np.array_equal(np.rint(t), np.rint(x / s)), (mant_s, e)


def test_a_factor_is_its_quotient_in_every_bit():
    """top * RN(1 / m), corrected once by fma(-m, q, top), is RN(top / m) for
    every mantissa of a 16-bit number (fma by exact arithmetic in fp64: the
    products have at most 35 bits)."""
    f = np.float32
    top = np.arange(1024, 2048, dtype=np.float64)
    for m in (7.0, 127.0):
        inv = f(1) / f(m)
        q = (top.astype(f) * inv).astype(f)
        rest = (top - m * q.astype(np.float64)).astype(f)
        got = (rest.astype(np.float64) * np.float64(inv) + q.astype(np.float64)).astype(f)
        assert np.array_equal(got, (top / m).astype(f))
        assert np.array_equal(got, (top.astype(f) / f(m)))
