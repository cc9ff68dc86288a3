"""Head norms with positions and the quantised cache on the GPU, against the
plain 64-bit forms of qcache_oracle.py: types, widths, head layouts, lengths
from nothing to long, odd pages and strides, trees with absent nodes, what is
masked holding NaN, offsets past 32 bits, streams and graphs."""

import numpy as np
import pytest

import qcache_oracle as qo
import spec_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tf.lib()
    yield
    tf.tf_device_error()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


def tree(kind, n, rng):
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    par = [-1] + [int(rng.integers(max(0, j - 6), j)) for j in range(1, n)]
    if kind == "padded":
        for j in range(n - max(1, n // 3), n):
            par[j] = -2
    if kind == "holes":
        for j in range(2, n, 3):
            par[j] = -5
    return par


def raised():
    with pytest.raises(tf.TFError) as e:
        tf.tf_device_error()
    assert e.value.status == tf.TF_ERR_INDEX


class Case:
    """A quantised paged cache of random rows with scattered pages. layout:
    "hnd" as tf_kvq_cache makes it, "nhd" heads inside a slot, "both" keys and
    values of a page in one tensor, rows padded."""

    def __init__(self, bits, dtype, lens, n, kh, group, d, page, seed=0, spare=2, layout="hnd", spoil=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bits, self.dtype, self.lens, self.n, self.kh, self.h, self.d = bits, dtype, lens, n, kh, kh * group, d
        self.page = page
        b = len(lens)
        per = max(1, -(-(max(max(lens), 0) + n) // page))
        pages = b * per + spare
        w = d * bits // 8
        lo = 1 if bits == 8 else 0
        if layout == "hnd":
            self.k, self.v, self.s = tf.tf_kvq_cache(pages, page, kh, d, bits)
        elif layout == "nhd":
            self.k, self.v = (torch.zeros((pages, page, kh, w), dtype=torch.uint8, device="cuda") for _ in range(2))
            self.s = torch.zeros((pages, page, kh, 2), dtype=torch.bfloat16, device="cuda")
        else:
            both = torch.zeros((pages, 2, page, kh, w + 16), dtype=torch.uint8, device="cuda")
            self.k, self.v = both[:, 0, :, :, :w], both[:, 1, :, :, :w]
            self.s = torch.zeros((pages, page, kh, 6), dtype=torch.bfloat16, device="cuda")[..., 2:4]
        for x in (self.k, self.v):
            c = torch.randint(lo, 256, x.shape, device="cuda", generator=g).to(torch.uint8)
            if bits == 4:    # a code of -8 is none that a write leaves
                c = torch.where((c & 15) == 0, c + 1, c)
                c = torch.where((c >> 4) == 0, c + 16, c)
            x.copy_(c)
        size = torch.randn(self.s.shape, device="cuda", generator=g).exp() / (4.0 if bits == 4 else 64.0)
        self.s.copy_(size)
        perm = torch.randperm(pages, device="cuda", generator=g)[: b * per]
        self.table = perm.to(torch.int32).view(b, per).contiguous()
        self.lengths = i32(lens)
        rows = torch.randn((b, n, (self.h + 2 * kh) * d), device="cuda", generator=g).to(DT[dtype])
        self.q = rows[:, :, : self.h * d].view(b, n, self.h, d)
        self.k_new = rows[:, :, self.h * d: (self.h + kh) * d].view(b, n, kh, d)
        self.v_new = rows[:, :, (self.h + kh) * d:].view(b, n, kh, d)
        if spoil:                 # every slot that no row may see: NaN rows
            self.s.view(torch.int16)[~self.used()] = 0x7FFF

    def used(self, extra=None):
        used = torch.zeros(self.k.shape[:2], dtype=torch.bool, device="cuda")
        for i, ln in enumerate(self.lens):
            if ln < 0:
                continue
            s = torch.arange(ln + (self.n if extra is None else extra), device="cuda")
            used[self.table[i].long()[s // self.page], s % self.page] = True
        return used

    def attend(self, parents, **kw):
        return tf.tf_kvq_attention(self.q, self.k, self.v, self.s, self.table, self.lengths, parents, **kw)

    def check(self, parents, scale=None, out=None, lse=None):
        b = len(self.lens)
        par = np.broadcast_to(np.asarray(parents, dtype=np.int64), (b, self.n))
        if out is None:
            out, lse = self.attend(i32(parents), scale=scale)
            tf.tf_device_error()
        scale = self.d ** -0.5 if scale is None else scale
        kk, vv = (qo.unpack(x.cpu().numpy(), self.bits) for x in (self.k, self.v))
        ss, qq, tb = f64(self.s), f64(self.q), self.table.cpu().numpy()
        got_o, got_l = f64(out), f64(lse)
        for i, ln in enumerate(self.lens):
            if ln < 0:
                assert np.all(got_o[i] == 0) and np.all(got_l[i] == -np.inf)
                continue
            total = ln + self.n
            pg, rw = so.slot_rows(tb[i], self.page, total)
            seen = np.ones((self.n, total), dtype=bool)
            seen[:, ln:] = so.seen_nodes(list(par[i]))
            seen[par[i] < -1] = False
            o, l, mag, err, top = qo.attend(qq[i], kk[pg, rw], ss[pg, rw, :, 0], vv[pg, rw], ss[pg, rw, :, 1], seen,
                                            scale, self.bits)
            tol_o, tol_l = qo.attend_bounds(o, l, mag, err, top, self.dtype, total, self.bits)
            assert np.array_equal(np.isneginf(got_l[i]), np.isneginf(l)), i
            fin = np.isfinite(l)
            off = np.abs(got_l[i][fin] - l[fin])
            assert np.all(off <= tol_l[fin]), (i, off.max())
            bad = ~(np.abs(got_o[i] - o) <= tol_o)
            assert not bad.any(), (i, np.argwhere(bad)[:4].tolist(), np.abs(got_o[i] - o).max(), bad.mean())
            assert np.all(got_o[i][~fin] == 0)
        return out, lse


# -------------------------------------------------------- norms and positions
def norm_check(dtype, b, n, h, kh, d, rotary, interleaved, hadamard, eps=1e-6, wdt="same", seed=0, far=1000, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = (scale * torch.randn((b, n, h + 2 * kh, d), device="cuda", generator=g)).to(DT[dtype])
    q, k = rows[:, :, :h], rows[:, :, h:h + kh]
    pos = torch.randint(0, far, (b, n), device="cuda", generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / max(rotary, 1))
    wt = None
    if wdt is not None:
        wt = (0.5 + torch.rand((2, d), device="cuda", generator=g)).to(DT[dtype] if wdt == "same" else wdt).unbind(0)
    got = tf.tf_qk_norm_rope(q, k, pos, freq if rotary else None, *(wt or (None, None)), eps=eps,
                             interleaved=interleaved, hadamard=hadamard)
    tf.tf_device_error()
    for x, y, w in zip((q, k), got, wt or (None, None)):
        assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
        fr = f64(freq)
        want, mag = qo.norm_rope(f64(x), 1.0 if w is None else f64(w), pos.cpu().numpy(), fr, eps, interleaved, hadamard)
        tol = qo.norm_rope_bound(want, mag, dtype, pos.cpu().numpy(), fr, d)
        off = np.abs(f64(y) - want)
        assert np.all(off <= tol), (np.argwhere(off > tol)[:4].tolist(), (off / tol).max())
    return q, k, pos, freq, wt, got


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 32), (128, 0), (256, 256), (256, 64),
                                      (256, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hadamard", [False, True])
def test_norm_rope_heads_and_rotations(dtype, d, rotary, interleaved, hadamard):
    norm_check(dtype, 2, 5, 6, 2, d, rotary, interleaved, hadamard, seed=d + rotary)


@pytest.mark.parametrize("b,n,h,kh", [(1, 1, 1, 1), (1, 1, 40, 8), (3, 1, 5, 1), (1, 700, 3, 1), (2, 333, 48, 8),
                                      (33, 7, 17, 17), (1, 1, 200, 3)])
def test_norm_rope_sizes(b, n, h, kh):
    norm_check("bf16", b, n, h, kh, 128, 128, False, True, seed=n)
    norm_check("fp16", b, n, h, kh, 64, 64, True, False, seed=n + 1)


@pytest.mark.parametrize("wdt", [None, torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("eps", [None, 0.0, 1e-6, 0.5])
def test_norm_rope_weights_and_eps(wdt, eps):
    for dtype in ("fp16", "bf16"):
        norm_check(dtype, 2, 3, 4, 2, 128, 128, False, False, eps=eps, wdt=wdt, seed=3)


@pytest.mark.parametrize("far", [131072, 2 ** 31 - 1])
def test_norm_rope_far_positions(far):
    norm_check("fp16", 4, 50, 2, 1, 128, 128, False, False, far=far, seed=9)


@pytest.mark.parametrize("scale", [1e-4, 300.0])
def test_norm_rope_small_and_large_rows(scale):
    norm_check("fp16", 2, 9, 3, 1, 128, 64, False, True, scale=scale, seed=10, eps=1e-12)
    norm_check("bf16", 2, 9, 3, 1, 128, 64, False, True, scale=scale, seed=10, eps=0.0)


@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("power", [70, 120, -45, -80, -120])
def test_norm_rope_rows_whose_squares_leave_fp32(power, hadamard):
    norm_check("bf16", 2, 9, 3, 1, 128, 128, False, hadamard, scale=2.0 ** power, seed=11, eps=0.0)
    if power > 0:
        norm_check("bf16", 2, 9, 3, 1, 128, 128, False, hadamard, scale=2.0 ** power, seed=12)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_rope_rows_of_all_sizes_beside_each_other(d):
    powers = torch.tensor([0, 70, -50, 3, 120, -110, -7, 100], device="cuda").repeat(20)[:150]
    norm_check("bf16", 2, 15, 3, 1, d, d, True, False, scale=torch.exp2(powers.float()).view(2, 15, 5, 1), seed=13, eps=0.0)


def test_norm_rope_in_place_strided_and_one_position_for_all():
    q, k, pos, freq, wt, want = norm_check("bf16", 3, 17, 6, 2, 128, 128, False, True, seed=4)
    rows = q._base.clone()
    q2, k2 = rows[:, :, :6], rows[:, :, 6:8]
    back = tf.tf_qk_norm_rope(q2, k2, pos, freq, *wt, hadamard=True, q_out=q2, k_out=k2)
    assert back[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(rows[:, :, 8:], q._base[:, :, 8:])                 # values are not touched
    same = pos[:1].expand(3, 17)
    a = tf.tf_qk_norm_rope(q, k, same.contiguous(), freq, *wt)
    c = tf.tf_qk_norm_rope(q, k, pos[0], freq, *wt)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    alone = tf.tf_qk_norm_rope(q, None, pos[0], freq, wt[0])
    assert torch.equal(alone[0], a[0]) and alone[1] is None
    head_first = q.transpose(1, 2).contiguous().transpose(1, 2)            # another order of heads and nodes
    out = torch.empty((3, 6, 17, 136), dtype=torch.bfloat16, device="cuda")[..., :128].transpose(1, 2)
    d = tf.tf_qk_norm_rope(head_first, None, pos[0], freq, wt[0], q_out=out)
    assert torch.equal(d[0], a[0])


def test_norm_rope_negative_positions_are_left_alone():
    q, k, pos, freq, wt, want = norm_check("fp16", 2, 40, 5, 1, 64, 64, False, False, seed=5)
    pos = pos.clone()
    gone = torch.rand(pos.shape, device="cuda") < 0.4
    pos[gone] = -1
    qo_, ko_ = torch.full_like(want[0], 7), torch.full_like(want[1], 7)
    tf.tf_qk_norm_rope(q, k, pos, freq, *wt, q_out=qo_, k_out=ko_)
    assert torch.equal(qo_[~gone], want[0][~gone]) and torch.equal(ko_[~gone], want[1][~gone])
    assert (qo_[gone] == 7).all() and (ko_[gone] == 7).all()


def test_norm_rope_products_stay_with_the_hadamard_rotation():
    q, k, pos, freq, wt, plain = norm_check("bf16", 1, 20, 2, 2, 128, 128, False, False, seed=6)
    turned = tf.tf_qk_norm_rope(q, k, pos, freq, *wt, hadamard=True)
    dot = lambda a, c: torch.einsum("bnhd,bmhd->bhnm", a.double(), c.double())  # noqa: E731
    x, y = dot(*plain), dot(*turned)
    # both sides of each product are rounded once (2^-8): off by 2^-7 of the product of the norms at most
    size = plain[0].double().norm(dim=-1).max() * plain[1].double().norm(dim=-1).max()
    assert ((x - y).abs() <= 2 * 2.0 ** -7 * size).all()


def test_norm_rope_not_finite_rows_stay_their_own():
    q, k, pos, freq, wt, want = norm_check("fp16", 1, 30, 4, 1, 128, 128, False, True, seed=7)
    q2 = q.clone()
    q2[0, 7, 2, 5], q2[0, 9, 0, 0] = float("nan"), float("inf")
    got = tf.tf_qk_norm_rope(q2, k, pos, freq, *wt, hadamard=True)[0]
    same = torch.ones((1, 30, 4), dtype=torch.bool, device="cuda")
    same[0, 7, 2] = same[0, 9, 0] = False
    assert torch.equal(got[same], want[0][same]) and not torch.isfinite(got[~same]).any()


# ------------------------------------------------------------ write and read
def special_rows(x, dtype):
    """Rows where quantising can go wrong, over the first rows of x."""
    flat = x.reshape(-1, x.shape[-1])
    big = torch.finfo(DT[dtype]).max
    tiny = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    d = flat.shape[1]
    ramp = torch.arange(d, device="cuda") - d // 2
    rows = [torch.zeros(d), torch.full((d,), big), torch.full((d,), -big), torch.full((d,), tiny), ramp / 2.0,
            7 * ((ramp % 15) - 7) / 7.0, (ramp % 29 - 14) / 2.0, (ramp % 509 - 254) / 2.0, ramp * tiny, ramp * 1e-5,
            torch.where(ramp == 3, 1000.0, 0.01), torch.where(ramp == 3, float("nan"), 1.0),
            torch.where(ramp == 0, float("inf"), 1.0), torch.where(ramp == 5, -float("inf"), 0.0)]
    for i, r in enumerate(rows):
        if i < len(flat):
            flat[i] = torch.as_tensor(r).to(flat)
    x.copy_(flat.view(x.shape))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,kh,d,page,layout", [(1, 8, 128, 16, "hnd"), (5, 3, 64, 7, "nhd"), (70, 2, 256, 32, "both"),
                                                (17, 1, 64, 1, "hnd"), (300, 2, 128, 24, "nhd")])
def test_write_is_the_definition_and_touches_nothing_else(bits, dtype, n, kh, d, page, layout):
    lens = [0, 45, -1, 31]
    c = Case(bits, dtype, lens, n, kh, 1, d, page, seed=n, layout=layout)
    special_rows(c.k_new, dtype)
    special_rows(c.v_new, dtype)
    for counts in (None, [n, max(0, n - 3), n, n // 2]):
        want = [x.cpu().numpy().copy() for x in (c.k, c.v)]
        want_s = f64(c.s)
        for i, ln in enumerate(lens):
            m = 0 if ln < 0 else n if counts is None else counts[i]
            s = ln + np.arange(m)
            pg, rw = c.table[i].cpu().numpy()[s // page], s % page
            for x, (w, new) in enumerate(zip(want, (c.k_new, c.v_new))):
                whole, factor = qo.quantise(f64(new[i, :m]), bits)
                w[pg, rw] = qo.pack(whole, bits)
                want_s[pg, rw, :, x] = factor
        tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, c.table, c.lengths, counts=None if counts is None else i32(counts))
        tf.tf_device_error()
        assert np.array_equal(c.k.cpu().numpy(), want[0]) and np.array_equal(c.v.cpu().numpy(), want[1])
        assert np.array_equal(f64(c.s), want_s, equal_nan=True)
        c.k_new, c.v_new = -c.v_new, c.k_new * 1   # contiguous rows the second time


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_factors_of_every_16_bit_number(bits, dtype):
    """A row for each finite magnitude that the type has as its largest, with
    parts of it in the others: ties, and what is next to them."""
    tops = torch.arange(0, 1 << 15, dtype=torch.int16, device="cuda").view(DT[dtype])
    tops = tops[torch.isfinite(tops)]
    n, most = len(tops), 7 if bits == 4 else 127
    share = torch.linspace(-1, 1, 64, device="cuda", dtype=torch.float64)
    share[:30] = (torch.arange(30, device="cuda") - 14.5) / most     # near ties
    share[0] = -1.0
    for parts in (share, share.clamp(-1, 1)):     # (the first go past the largest, some to infinity)
        x = (tops.double()[:, None] * parts).to(DT[dtype])
        x[:, 63] = tops
        k, v, s = tf.tf_kvq_cache(-(-n // 64), 64, 1, 64, bits)
        table = torch.arange(k.shape[0], device="cuda", dtype=torch.int32)[None]
        rows = x.view(1, n, 1, 64)
        tf.tf_kvq_write(rows, rows.flip(1).contiguous(), k, v, s, table, i32([0]))
        tf.tf_device_error()
        for y, codes, at in ((x, k, 0), (x.flip(0), v, 1)):
            whole, factor = qo.quantise(f64(y), bits)
            assert np.array_equal(f64(s).reshape(-1, 2)[:n, at], factor, equal_nan=True)
            assert np.array_equal(codes.cpu().numpy().reshape(-1, codes.shape[-1])[:n], qo.pack(whole, bits))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kh,d,page,layout", [(8, 128, 16, "hnd"), (3, 64, 7, "nhd"), (2, 256, 32, "both")])
def test_read_gives_the_values_and_leaves_the_rest(bits, dtype, kh, d, page, layout):
    lens = [0, 145, -1, 31, 200]
    c = Case(bits, dtype, lens, 1, kh, 1, d, page, seed=2, layout=layout)
    c.s[c.table[4, 0].long(), 0] = float("nan")
    val = [qo.unpack(x.cpu().numpy(), bits) * f64(c.s)[..., i, None] for i, x in enumerate((c.k, c.v))]
    for starts, slots in ((None, 150), ([0, 100, 0, 40, 7], 60), ([0, 144, 5, 30, 199], 1)):
        outs = [torch.full((5, slots, kh, d), 3.0, device="cuda").to(DT[dtype]) for _ in range(2)]
        if slots == 60:
            outs = [torch.full((5, kh, slots, d + 8), 3.0, device="cuda").to(DT[dtype])[..., :d].transpose(1, 2) for _ in range(2)]
        want = [f64(o) for o in outs]
        for i, ln in enumerate(lens):
            first = 0 if starts is None else starts[i]
            s = first + np.arange(max(0, min(slots, ln - first)))
            pg, rw = c.table[i].cpu().numpy()[s // page], s % page
            for w, x in zip(want, val):
                w[i, :len(s)] = f64(torch.tensor(x[pg, rw]).to(torch.float32).to(DT[dtype]))
        got = tf.tf_kvq_read(c.k, c.v, c.s, c.table, c.lengths, starts=None if starts is None else i32(starts),
                             k_out=outs[0], v_out=outs[1])
        tf.tf_device_error()
        assert got[0] is outs[0]
        for a, w in zip(got, want):
            assert np.array_equal(f64(a), w, equal_nan=True)
    a = tf.tf_kvq_read(c.k, c.v, c.s, c.table, c.lengths, slots=150, head_dim=d, dtype=DT[dtype])
    assert a[0].shape == (5, 150, kh, d) and (a[0][0] == 0).all() and (a[0][3, 31:] == 0).all()


def test_write_then_read_is_near_what_was_written():
    """Half a step of the row's factor, which is off by 2^-8 of itself at most,
    and the rounding of the value."""
    for bits, dtype in ((4, "fp16"), (8, "bf16")):
        c = Case(bits, dtype, [0, 50], 90, 2, 1, 128, 16, seed=8)
        tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, c.table, c.lengths)
        got = tf.tf_kvq_read(c.k, c.v, c.s, c.table, c.lengths + 90, starts=c.lengths, slots=90, head_dim=128, dtype=DT[dtype])
        for x, y in zip((c.k_new, c.v_new), got):
            top = x.double().abs().amax(-1, keepdim=True)
            step = top / (7 if bits == 4 else 127)
            assert ((x.double() - y.double()).abs() <= step * (0.5 + (7 if bits == 4 else 127) * 2.0 ** -8) + top * 2.0 ** -8).all()


def test_write_and_read_skip_bad_indices():
    c = Case(4, "fp16", [10, 10], 4, 1, 1, 64, 16, seed=1)
    k0, v0, s0 = c.k.clone(), c.v.clone(), c.s.clone()
    same = lambda: torch.equal(c.k, k0) and torch.equal(c.v, v0) and torch.equal(c.s, s0)  # noqa: E731
    for table, lens, counts in ((i32([[c.k.shape[0]], [-3]]), c.lengths, None), (c.table, i32([1 << 20, 2 ** 31 - 2]), None),
                                (c.table, i32([-1, -1]), i32([0, 0]))):
        tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, table, lens, counts=counts)
        if counts is None:
            raised()
        assert same()
    tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, c.table, c.lengths, counts=i32([-1, 5]))
    raised()
    at = int(c.table[1, 0])
    assert torch.equal(c.k[int(c.table[0, 0])], k0[int(c.table[0, 0])]) and not torch.equal(c.k[at], k0[at])
    outs = [torch.full((2, 20, 1, 64), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    for table, lens, starts in ((i32([[c.k.shape[0]], [-3]]), c.lengths, None), (c.table, c.lengths, i32([-1, -7])),
                                (c.table, i32([2 ** 31 - 1] * 2), i32([100, 1 << 30]))):
        tf.tf_kvq_read(c.k, c.v, c.s, table, lens, starts=starts, k_out=outs[0], v_out=outs[1])
        raised()
        assert all((o == 3).all() for o in outs)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("n,kh,d,page,layout", [(8, 8, 128, 16, "hnd"), (128, 2, 64, 7, "nhd"), (2, 1, 64, 1, "hnd"),
                                                (33, 3, 256, 32, "hnd"), (20, 2, 128, 16, "both")])
def test_keep_moves_the_path_together(bits, layers, n, kh, d, page, layout):
    rng = np.random.default_rng(n)
    lens = [0, 45, -1, 31, 8]
    b = len(lens)
    c = Case(bits, "bf16", lens, n, kh, 1, d, page, seed=n, layout=layout)
    if layers is None:
        bufs = [c.k, c.v, c.s]
    else:
        bufs = []
        for x in (c.k, c.v, c.s):
            y = torch.empty((layers, x.shape[0], kh, page, x.shape[3]), dtype=x.dtype, device="cuda").transpose(2, 3)
            for i in range(layers):
                y[i] = x if i == 0 else torch.roll(x, i, 0)
            bufs.append(y)
    counts = [n, int(rng.integers(1, n + 1)), 1, 0, max(1, n // 2)]
    path = np.full((b, n), -1)
    for i, m in enumerate(counts):
        path[i, :m] = np.sort(rng.permutation(n)[:m])
    want = [x.clone() for x in bufs]
    for w in want:
        w = w if layers is not None else w[None]
        for i, ln in enumerate(lens):
            if ln < 0:
                continue
            to = ln + torch.arange(counts[i], device="cuda")
            src = ln + torch.tensor(path[i, :counts[i]], device="cuda")
            at = lambda s: (c.table[i].long()[s // page], s % page)  # noqa: E731
            rows = w[:, at(src)[0], at(src)[1]].clone()
            w[:, at(to)[0], at(to)[1]] = rows
    new = tf.tf_kvq_keep(*bufs, c.table, c.lengths, i32(path), i32(counts))
    tf.tf_device_error()
    for x, w in zip(bufs, want):
        assert torch.equal(x, w)
    assert new.tolist() == [ln + m if ln >= 0 else ln for ln, m in zip(lens, counts)]


def test_keep_skips_bad_indices():
    c = Case(4, "fp16", [10, 10], 4, 1, 1, 64, 16, seed=1)
    k0, s0 = c.k.clone(), c.s.clone()
    new = tf.tf_kvq_keep(c.k, c.v, c.s, c.table, c.lengths, i32([[2, 1, 3, -1], [0, 1, 4, -1]]), i32([3, 9]))
    raised()
    pg = int(c.table[0, 0])
    k0[pg, 10], s0[pg, 10] = k0[pg, 12], s0[pg, 12]
    assert torch.equal(c.k, k0) and torch.equal(c.s, s0) and new.tolist() == [11, 12]


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("bits,dtype", [(4, "fp16"), (4, "bf16"), (8, "fp16"), (8, "bf16")])
@pytest.mark.parametrize("kh,group,d", [(8, 5, 128), (2, 1, 64), (1, 8, 128), (1, 3, 256), (3, 7, 64), (1, 16, 128), (1, 12, 256)])
@pytest.mark.parametrize("n,kind", [(1, "chain"), (5, "tree"), (16, "padded"), (40, "tree")])
def test_attention_heads_and_trees(bits, dtype, kh, group, d, n, kind):
    rng = np.random.default_rng(n * 100 + kh)
    lens = [200, 0, 77]
    Case(bits, dtype, lens, n, kh, group, d, 16, seed=n).check([tree(kind, n, rng) for _ in lens])


@pytest.mark.parametrize("page", [1, 7, 8, 16, 17, 24, 64, 128, 200, 256, 300])
@pytest.mark.parametrize("n", [1, 20])
def test_attention_page_sizes(page, n):
    rng = np.random.default_rng(page)
    lens = [page * 3 - 1, page, 129, 500]
    Case(4, "fp16", lens, n, 2, 4, 128, page, seed=page).check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("n", [1, 3, 64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [2, 127], [128, 126], [129, 63, 64, 65], [1000, 0, 5, 31, 32, 33]])
@pytest.mark.parametrize("bits,d", [(4, 128), (8, 64), (8, 128)])
def test_attention_lengths(n, lens, bits, d):
    rng = np.random.default_rng(len(lens))
    Case(bits, "bf16", lens, n, 2, 2, d, 32, seed=n).check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("n", [1, 30])
def test_attention_long_context_is_split_and_joined(n):
    rng = np.random.default_rng(5)
    Case(4, "bf16", [9001], n, 1, 4, 128, 64, seed=5).check([tree("tree", n, rng)])
    Case(8, "fp16", [7000, 3], n, 1, 5, 64, 16, seed=6).check([tree("tree", n, rng), tree("star", n, rng)])
    Case(4, "fp16", [5000, 3], n, 1, 5, 256, 16, seed=6).check([tree("tree", n, rng), tree("star", n, rng)])


@pytest.mark.parametrize("b,n", [(300, 1), (129, 6), (700, 2), (32, 1), (33, 12), (100, 2), (400, 12)])
def test_attention_large_batches(b, n):
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(-1, 90, b)]
    lens[7] = 400
    Case(4, "bf16", lens, n, 1, 2, 64, 16, seed=b).check(tree("chain", n, rng))


@pytest.mark.parametrize("kind", ["star", "roots", "holes", "padded", "chain"])
@pytest.mark.parametrize("n", [2, 33, 128])
def test_attention_tree_shapes(kind, n):
    rng = np.random.default_rng(n)
    lens = [130, 0, -1, 64]
    par = [tree(kind, n, rng) for _ in lens]
    par[1] = [-2] * n
    Case(4, "fp16", lens, n, 2, 3, 64, 16, seed=n + 1).check(par)


@pytest.mark.parametrize("layout", ["nhd", "both"])
@pytest.mark.parametrize("page,n,bits", [(16, 1, 4), (64, 24, 8), (7, 3, 4)])
def test_attention_cache_layouts(layout, page, n, bits):
    rng = np.random.default_rng(3)
    Case(bits, "bf16", [300, 41], n, 3, 4, 128, page, seed=3, layout=layout).check([tree("tree", n, rng)] * 2)


@pytest.mark.parametrize("n,group,bits,d", [(1, 4, 4, 128), (9, 4, 8, 64), (40, 5, 4, 128), (2, 2, 4, 256)])
def test_attention_unseen_slots_have_no_influence(n, group, bits, d):
    rng = np.random.default_rng(2)
    lens = [131, 0, 63, 255]
    c = Case(bits, "fp16", lens, n, 2, group, d, 32, seed=2, spoil=True)
    c.check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("group,d,bits", [(1, 64, 8), (5, 128, 4), (2, 256, 4)])
@pytest.mark.parametrize("n", [3, 24])
def test_attention_a_siblings_bad_row_stays_its_own(n, group, d, bits):
    """The last node's key or value is NaN: rows that see it are spoilt, the
    others keep the bits they have without it."""
    par = tree("tree", n, np.random.default_rng(4)) if n > 3 else [-1, 0, 0]
    seen = so.seen_nodes(par)
    for ln in (100, 0):
        for which in (0, 1):
            c = Case(bits, "bf16", [ln], n, 2, group, d, 16, seed=4)
            want, want_l = c.attend(i32(par))
            s = ln + n - 2
            c.s[int(c.table[0, s // 16]), s % 16, :, which] = float("nan")
            got, got_l = c.attend(i32(par))
            hit = torch.tensor(seen[:, n - 2], device="cuda")
            assert torch.equal(got[0, ~hit], want[0, ~hit]) and torch.equal(got_l[0, ~hit], want_l[0, ~hit])
            assert torch.isnan(got[0, hit]).all()
            assert torch.isnan(got_l[0, hit]).all() if which == 0 else torch.equal(got_l, want_l)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_large_values_beside_a_bad_sibling(bits, d, group, bad):
    """Tree nodes that see the context and themselves, after a context of small
    values: their own are 2^20 times as large, one of them is bad. With q = 0
    all weights are alike, so a row is the mean of the values it sees. More
    items than runs, so that the nodes come after a run's first tile."""
    g = torch.Generator(device="cuda").manual_seed(5)
    b, kh, n, ctx, page = 70, 8, 5, 200, 16
    per = -(-(ctx + n) // page)
    k, v, s = tf.tf_kvq_cache(b * per, page, kh, d, bits)
    table = torch.arange(b * per, dtype=torch.int32, device="cuda").view(b, per)
    zero, lens = i32([0] * b), i32([ctx] * b)
    rows = lambda m, size: (size * torch.randn((b, m, kh, d), device="cuda", generator=g)).to(torch.bfloat16)  # noqa: E731
    tf.tf_kvq_write(rows(ctx, 1.0), rows(ctx, 2.0 ** -10), k, v, s, table, zero)
    own = rows(n, 2.0 ** 10)
    own[:, 2, :, 3] = bad
    tf.tf_kvq_write(rows(n, 1.0), own, k, v, s, table, lens)
    q = torch.zeros((b, n, kh * group, d), dtype=torch.bfloat16, device="cuda")
    out, lse = tf.tf_kvq_attention(q, k, v, s, table, lens, i32([-1] * n))
    values = tf.tf_kvq_read(k, v, s, table, i32([ctx + n] * b), slots=ctx + n, head_dim=d, dtype=torch.bfloat16)[1].double()
    of_ctx, of_own = values[:, :ctx].sum(1, keepdim=True), values[:, ctx:]
    want = ((of_ctx + of_own) / (ctx + 1)).repeat_interleave(group, 2)
    mag = ((values[:, :ctx].abs().sum(1, keepdim=True) + of_own.abs()) / (ctx + 1)).repeat_interleave(group, 2)
    # bf16 has 8 significant bits: steps of 2^-7 at 1, half of one is 2^-8. So
    # values that were read back are off by 2^-8 and the result by 2^-8 again;
    # weights, in fp16, by 2^-11; sums in fp32 by 2^-14 at most.
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7)
    fine = [0, 1, 3, 4]
    assert ((out.double() - want).abs() <= tol)[:, fine].all(), ((out.double() - want).abs() / tol)[:, fine].max()
    assert torch.isnan(out[:, 2]).all()
    assert (lse.double() - np.log(ctx + 1)).abs().max() <= 2.0 ** -18
    tf.tf_device_error()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,group", [(1, 5), (4, 5), (40, 2)])
def test_attention_factors_over_a_wide_range(bits, dtype, n, group):
    """Factors of keys and values, and rows of q, that differ by many powers of
    two: what is largest is not what weighs most."""
    c = Case(bits, dtype, [700, 300], n, 2, group, 128, 16, seed=21)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(-9, 8, c.s.shape, device="cuda", generator=g).float()
    c.s[..., 1] = (c.s[..., 1].float() * torch.exp2(e[..., 1])).bfloat16()
    c.s[..., 0] = (c.s[..., 0].float() * torch.exp2(e[..., 0].clamp(-9, 0))).bfloat16()
    size = torch.exp2(torch.randint(-6, 3, c.q.shape[:3], device="cuda", generator=g).float())[..., None]
    c.q = (c.q.float() * size).to(c.q.dtype)
    c.check([tree("tree", n, np.random.default_rng(1))] * 2, scale=0.02)


@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** 60), ("bf16", 2.0 ** -60), ("fp16", 2.0 ** -20), ("fp16", 1000.0)])
def test_attention_large_and_small_queries(dtype, size):
    """A row of q far from 1, with a scale that brings the scores back."""
    c = Case(4, dtype, [300, 40], 3, 2, 4, 128, 16, seed=22)
    c.q = (c.q.float() * size).to(c.q.dtype)
    c.check([tree("tree", 3, np.random.default_rng(1))] * 2, scale=0.05 / size)
    c.q = c.q * 0
    c.check([tree("tree", 3, np.random.default_rng(1))] * 2)


@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** -70])
def test_attention_large_and_small_values(size):
    """Values that fp16 cannot hold."""
    c = Case(8, "bf16", [300, 40], 3, 2, 4, 64, 16, seed=23)
    c.s[..., 1] *= size
    c.check([tree("tree", 3, np.random.default_rng(1))] * 2)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("n,group", [(1, 4), (20, 4)])
def test_attention_scales(scale, n, group):
    c = Case(4, "bf16", [200, 7], n, 2, group, 128, 16, seed=24)
    c.check([tree("tree", n, np.random.default_rng(1))] * 2, scale=scale)


def test_attention_rising_and_falling_scores():
    """Scores that climb or fall by hundreds along the context: the running
    maximum has to move, and early or late parts vanish."""
    for sign in (1.0, -1.0):
        for n, bits in ((3, 4), (3, 8), (30, 4)):
            c = Case(bits, "bf16", [1500], n, 1, 2, 64, 16, seed=8)
            s = torch.arange(1500 + n, device="cuda")
            pages = c.table[0].long()[s // 16]
            c.q[..., :] = 1.0
            c.k[pages, s % 16] = 0x99 if bits == 4 else 129      # whole numbers 1
            c.s[pages, s % 16, :, 0] = (torch.linspace(-5, 5, 1500 + n, device="cuda") * sign).bfloat16()[:, None]
            c.check([tree("chain", n, None)], scale=1.0)


def test_attention_offsets_past_32_bits():
    """Pages whose offsets pass 2^32 bytes."""
    kh, d, page = 8, 128, 128
    pages = (1 << 32) // (kh * (d // 2) * page) + 40
    k, v, s = tf.tf_kvq_cache(pages, page, kh, d, 4)
    for n in (1, 20):
        c = Case(4, "bf16", [1000, 300], n, kh, 4, d, page, seed=11)
        lift = pages - c.k.shape[0]
        k[lift:], v[lift:], s[lift:] = c.k, c.v, c.s
        par = i32([tree("chain", n, None)] * 2)
        want, want_l = c.attend(par)
        got, got_l = tf.tf_kvq_attention(c.q, k, v, s, c.table + lift, c.lengths, par)
        assert torch.equal(got, want) and torch.equal(got_l, want_l)
        tf.tf_kvq_write(c.k_new, c.v_new, k, v, s, c.table + lift, c.lengths)
        tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, c.table, c.lengths)
        assert torch.equal(k[lift:], c.k) and torch.equal(v[lift:], c.v) and torch.equal(s[lift:], c.s)
        a = tf.tf_kvq_read(k, v, s, c.table + lift, c.lengths + n, slots=1000 + n, head_dim=d)
        b = tf.tf_kvq_read(c.k, c.v, c.s, c.table, c.lengths + n, slots=1000 + n, head_dim=d)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,group,d", [(1, 5, 128), (16, 6, 128), (3, 1, 64), (64, 5, 128), (2, 3, 256)])
def test_attention_same_bits_every_time_and_on_two_streams(n, group, d):
    rng = np.random.default_rng(1)
    lens = [3000, 17, 900]
    c = Case(4, "bf16", lens, n, 2, group, d, 32, seed=1)
    par = i32([tree("tree", n, rng) for _ in lens])
    want, want_l = c.attend(par)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(c.attend(par))
    got.append(c.attend(par, stream=streams[0]))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_l)


@pytest.mark.parametrize("n", [1, 24])
def test_attention_workspace_serves_other_sizes_and_a_graph(n):
    rng = np.random.default_rng(6)
    big = Case(4, "fp16", [5000, 100], n, 2, 5, 128, 64, seed=6)
    small = Case(8, "fp16", [40], 2, 1, 1, 64, 16, seed=7)
    ws = tf.tf_kvq_attention_workspace(2, n, 10, 2, 128)
    pb, ps = i32([tree("tree", n, rng)] * 2), i32([[-1, 0]])
    first = big.attend(pb, workspace=ws)
    small.attend(ps, workspace=ws)
    again = big.attend(pb, workspace=ws)
    assert torch.equal(first[0], again[0])
    outs = []
    for use in (ws, None):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(big.attend(pb, workspace=use))
        for _ in range(3):
            outs[-1][0].fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[-1][0], first[0]) and torch.equal(outs[-1][1], first[1])


def test_attention_one_workspace_for_many_sizes_in_turn():
    rng = np.random.default_rng(12)
    make = lambda: tf.tf_kvq_attention_workspace(64, 40, 40, 8, 256)  # noqa: E731
    ws = make()
    cases = [Case(4, "bf16", [200, 0, 77], 40, 8, 5, 128, 16, seed=1), Case(8, "bf16", [3000], 1, 1, 1, 64, 64, seed=2),
             Case(4, "bf16", [30] * 64, 3, 4, 4, 64, 16, seed=3), Case(4, "bf16", [900, 800], 20, 4, 2, 256, 32, seed=4),
             Case(4, "bf16", [5000], 16, 2, 8, 128, 64, seed=5)]
    trees = [i32([tree("tree", c.n, rng) for _ in c.lens]) for c in cases]
    fresh = [c.attend(t, workspace=make()) for c, t in zip(cases, trees)]
    for _ in range(2):
        for c, t, (o, l) in zip(cases, trees, fresh):
            o2, l2 = c.attend(t, workspace=ws)
            assert torch.equal(o, o2) and torch.equal(l, l2)
    for c, t in zip(cases, trees):
        c.check(t.tolist())


def test_attention_workspace_for_the_largest_sizes_serves_fewer_kv_heads():
    need = tf.lib().tf_kvq_attention_workspace_bytes
    rng = np.random.default_rng(3)
    for heads, kv, n, d in ((8, 8, 4, 64), (16, 8, 16, 128), (24, 6, 9, 256)):
        ws = tf.tf_kvq_attention_workspace(2, n, heads, kv, d)
        smaller = [need(2, m, h, k, e) for m in range(1, n + 1) for h in range(1, heads + 1) for k in range(1, kv + 1)
                   for e in (64, 128, 256) if h % k == 0 and e <= d]
        assert max(smaller) <= ws.numel()
        for k in (1, 2, kv):
            c = Case(4, "bf16", [700, 90], n, k, heads // k, d, 16, seed=k)
            par = [tree("tree", n, rng)] * 2
            got = c.attend(i32(par), workspace=ws)
            c.check(par, out=got[0], lse=got[1])
    assert tf.tf_kvq_attention_workspace(2, 4, 8, 3, 64).numel() == 1   # refused sizes
    c = Case(4, "bf16", [700, 90], 2, 2, 2, 128, 16)
    with pytest.raises(tf.TFError) as e:
        c.attend(i32([[-1, 0]] * 2), workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == tf.TF_ERR_SCRATCH


@pytest.mark.parametrize("n,group", [(4, 2), (4, 8)])
def test_attention_bad_indices_are_skipped_and_recorded(n, group):
    c = Case(4, "fp16", [100, 100], n, 1, group, 64, 16, seed=13)
    par = i32([[-1, 0, 1, 2]] * 2)
    want, _ = c.attend(par)
    table = c.table.clone()
    table[1, 2], table[1, 3] = c.k.shape[0], -1
    got, _ = tf.tf_kvq_attention(c.q, c.k, c.v, c.s, table, c.lengths, par)
    raised()
    tf.tf_device_error()
    assert torch.equal(got[0], want[0]) and torch.isfinite(got).all() and not torch.equal(got[1], want[1])
    wide = torch.cat([c.table, torch.full((2, 3), 1 << 30, dtype=torch.int32, device="cuda")], 1).contiguous()
    got, _ = tf.tf_kvq_attention(c.q, c.k, c.v, c.s, wide, c.lengths, par)
    tf.tf_device_error()
    assert torch.equal(got, want)
    got, _ = tf.tf_kvq_attention(c.q, c.k, c.v, c.s, c.table, i32([100, 10 ** 9]), par)
    raised()
    assert torch.equal(got[0], want[0]) and torch.isfinite(got).all()
    got, lse = c.attend(i32([[-1, 0, 1, 2], [-1, 1, 9, 0]]))
    raised()
    assert torch.equal(got[0], want[0]) and torch.isneginf(lse[1, 1:3]).all() and (got[1, 1:3] == 0).all()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (8, "fp16")])
def test_the_operators_in_a_row(bits, dtype):
    """A prompt in parts, then trees: normed and rotated, written, attended to,
    the accepted path kept, as a decoder runs them; against attention over the
    values that were read back, in a graph as well."""
    g = torch.Generator(device="cuda").manual_seed(1)
    b, kh, group, d, page, n = 3, 2, 4, 128, 16, 6
    h, pages = kh * group, 40
    k, v, s = tf.tf_kvq_cache(pages, page, kh, d, bits)
    table = torch.randperm(pages, device="cuda", generator=g)[:39].to(torch.int32).view(b, 13)
    freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    w = torch.ones((d,), dtype=DT[dtype], device="cuda")
    lengths, prompt = i32([0, 0, 0]), [100, 37, 1]

    def rows(m):
        x = torch.randn((b, m, h + 2 * kh, d), device="cuda", generator=g).to(DT[dtype])
        return x[:, :, :h], x[:, :, h:h + kh], x[:, :, h + kh:]

    for first in (0, 64):
        counts = i32([min(max(p - first, 0), 64) for p in prompt])
        _, k_new, v_new = rows(64)
        pos = (lengths[:, None] + torch.arange(64, device="cuda", dtype=torch.int32)).int()
        _, k_new = tf.tf_qk_norm_rope(k_new, k_new, pos, freq, w, w, hadamard=True)
        tf.tf_kvq_write(k_new, v_new, k, v, s, table, lengths, counts=counts)
        lengths = lengths + counts
    assert lengths.tolist() == prompt
    par = [-1, 0, 1, 0, 3, 3]
    depth = i32([0, 1, 2, 1, 2, 2])
    parents = i32(par)
    q_in, k_in, v_in = rows(n)
    pos = lengths[:, None] + depth

    def step():
        q, k_new = tf.tf_qk_norm_rope(q_in, k_in, pos, freq, w, w, hadamard=True)
        tf.tf_kvq_write(k_new, v_in, k, v, s, table, lengths)
        return (q,) + tf.tf_kvq_attention(q, k, v, s, table, lengths, parents)

    q, out, lse = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[1], out) and torch.equal(held[2], lse)
    kk, vv = tf.tf_kvq_read(k, v, s, table, lengths + n, slots=106, head_dim=d, dtype=torch.bfloat16)
    for i, ln in enumerate(prompt):
        seen = np.ones((n, ln + n), dtype=bool)
        seen[:, ln:] = so.seen_nodes(par)
        o, l, mag, _ = so.attend(f64(q[i]), f64(kk[i, :ln + n]), f64(vv[i, :ln + n]), seen, d ** -0.5)
        # keys and values were read back with one rounding to bf16 each: scores are off by 2^-8 of sum |q k|
        # scale (at most 0.1 here: |q| |k| scale <= sqrt(d) * 1.2, times 2^-8 and twice for weight and sum)
        e = 2.0 ** -8 * 1.2 * 1.2 * d ** 0.5
        assert np.all(np.abs(f64(lse[i]) - l) <= 1.1 * e)
        assert np.all(np.abs(f64(out[i]) - o) <= (2.2 * e + 2.0 ** -7) * mag + 1e-3)
    path = i32([[0, 3, 5, -1, -1, -1]] * b)
    new = tf.tf_kvq_keep(k, v, s, table, lengths, path, i32([3, 3, 3]))
    k2, v2 = tf.tf_kvq_read(k, v, s, table, new, starts=lengths, slots=3, head_dim=d, dtype=torch.bfloat16)
    for i, ln in enumerate(prompt):
        for j, node in enumerate((0, 3, 5)):
            assert torch.equal(k2[i, j], kk[i, ln + node]) and torch.equal(v2[i, j], vv[i, ln + node])
    tf.tf_device_error()
