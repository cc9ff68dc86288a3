"""Attention over a quantised cache where factors and queries differ by many
powers of two: what a row does not see has no influence whatever its size,
what it sees weighs what the definition says, and finite inputs give finite
results."""

import numpy as np
import pytest

import qcache_oracle as qo
import spec_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402
from test_gpu_qcache import Case, f64, i32, tree  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tf.lib()
    yield
    tf.tf_device_error()


# bits, head_dim, nodes, heads a kv head: both kernels, each width of rows
FORMS = [(4, 64, 24, 1), (4, 128, 9, 5), (4, 128, 64, 2), (4, 128, 3, 2), (8, 128, 24, 2), (8, 64, 3, 1), (4, 256, 9, 2)]
LARGE = [2.0 ** 20, 2.0 ** 40, 2.0 ** 100, float(torch.finfo(torch.bfloat16).max)]


def places(c, i, slots):
    """Pages and rows of slots of sequence i."""
    s = torch.as_tensor(slots, device="cuda")
    return c.table[i].long()[s // c.page], s % c.page


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("kind", ["sibling", "absent"])
@pytest.mark.parametrize("which", [0, 1])
def test_a_large_row_that_is_not_seen_changes_no_bit(bits, d, n, group, kind, which):
    """The key (value) factor of a sibling, or of the absent nodes, grows: rows
    that do not see it keep their bits."""
    lens = [0, 100, 200]
    par = tree("tree" if n > 3 else "star", n, np.random.default_rng(4))
    if kind == "absent":
        gone = list(range(2, n, 3))
        par = [-2 if j in gone else p if p not in gone else -1 for j, p in enumerate(par)]
    else:
        gone = [n - 2]
    hidden = ~so.seen_nodes(par)[:, gone].any(1) & (np.asarray(par) >= -1)
    assert hidden.sum() >= 1
    hidden = torch.tensor(hidden, device="cuda")
    c = Case(bits, "bf16", lens, n, 2, group, d, 16, seed=4)
    want, want_l = c.attend(i32(par))
    for size in LARGE:
        for i, ln in enumerate(lens):
            pg, rw = places(c, i, [ln + j for j in gone])
            c.s[pg, rw, :, which] = size
        got, got_l = c.attend(i32(par))
        assert torch.equal(got[:, hidden], want[:, hidden]) and torch.equal(got_l[:, hidden], want_l[:, hidden]), size
    tf.tf_device_error()


@pytest.mark.parametrize("bits,d,n,group", FORMS)
def test_a_pool_of_any_bits_under_absent_nodes(bits, d, n, group):
    """A pool whose memory held something else: only what a write's counts
    cover is ever written, and the rest has no influence."""
    g = torch.Generator(device="cuda").manual_seed(n)
    par = tree("padded", n, np.random.default_rng(3))
    there = int((np.asarray(par) >= -1).sum())
    c = Case(bits, "bf16", [131, 0, 45], n, 2, group, d, 16, seed=n)
    old = torch.randint(-32768, 32768, c.s.shape, device="cuda", generator=g, dtype=torch.int32).to(torch.int16)
    used = c.used(0)
    for i, ln in enumerate(c.lens):
        used[places(c, i, list(range(ln, ln + there)))] = True
    c.s.view(torch.int16)[~used] = old[~used]
    tf.tf_kvq_write(c.k_new, c.v_new, c.k, c.v, c.s, c.table, c.lengths, counts=i32([there] * 3))
    got = c.attend(i32(par))
    # (what the oracle multiplies by weights of 0 has to be finite there)
    c.s.view(torch.int16)[~used] = 0x3C00
    c.check([par] * 3, out=got[0], lse=got[1])
    tf.tf_device_error()


def laid_out(bits, dtype, ctx, n, group, d, scores, sizes, q=1.0, seed=0):
    """A chain whose slot s has the score scores[s] for every row (q is one
    number, scale 1, codes 1 or -1), random values of factor sizes[s]."""
    c = Case(bits, dtype, [ctx], n, 2, group, d, 16, seed=seed)
    pg, rw = places(c, 0, list(range(ctx + n)))
    c.q[...] = q
    low, high = (0x77, 0x99) if bits == 4 else (127, 129)
    sign = torch.tensor(scores, device="cuda")
    c.k[pg, rw] = torch.where(sign < 0, low, high).to(torch.uint8)[:, None, None]
    c.s[pg, rw, :, 0] = (sign.abs() / (d * q)).bfloat16()[:, None]
    c.s[pg, rw, :, 1] = torch.as_tensor(sizes, device="cuda", dtype=torch.float32).bfloat16()[:, None]
    return c


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("power", [24, 28, 40])
def test_a_large_value_that_weighs_nothing(bits, d, n, group, dtype, power):
    """Every seventh key of the context has a value 2^power as large as the
    others, and a weight smaller still: p |v| of it is 2^-20 of theirs."""
    ctx = 300
    s = np.arange(ctx + n)
    large = (s % 7 == 3) & (s < ctx)
    scores = np.where(large, -(power + 20) * np.log(2.0), 0.25 * np.cos(s))
    c = laid_out(bits, dtype, ctx, n, group, d, scores, np.where(large, 2.0 ** power, 1.0 / 8), seed=power)
    c.check([tree("chain", n, None)], scale=1.0)


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("power", [19, 30, 60])
def test_a_large_key_whose_score_is_nothing(bits, d, n, group, power):
    """Every seventh key has a factor 2^power as large as the others, and codes
    of 0 where q is not: its score is exactly 0."""
    c = Case(bits, "bf16", [300, 20], n, 2, group, d, 16, seed=power)
    par = tree("tree", n, np.random.default_rng(1)) if n > 3 else [-1, 0, 0]
    c.q[..., 8:] = 0
    zero = 0x88 if bits == 4 else 128
    oracle_s = f64(c.s)
    for i, ln in enumerate(c.lens):
        pg, rw = places(c, i, list(range(3, ln + n, 7)))
        c.k[pg, rw, :, : 8 * bits // 8] = zero
        c.s[pg, rw, :, 0] = 2.0 ** power
        oracle_s[pg.cpu().numpy(), rw.cpu().numpy(), :, 0] = 0.0
    out, lse = c.attend(i32(par))
    tf.tf_device_error()
    # (the bound of a score grows with its key's factor; here the products are 0 whatever that is)
    held, c.s = c.s, torch.tensor(oracle_s, device="cuda")
    c.check([par] * 2, out=out, lse=lse)
    c.s = held


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("dtype,size", [("fp16", 300.0), ("bf16", 300.0), ("bf16", 2.0 ** 60)])
@pytest.mark.parametrize("lower", [30.0, 60.0, 100.0])
def test_rows_of_zeros_before_large_values(bits, d, n, group, dtype, size, lower):
    """Rows of zeros, and after them large values far below the maximum: the
    weights of the largest scores are multiplied by nothing at all."""
    ctx = 300
    scores = np.where(np.arange(ctx + n) < 200, 0.0, -lower)
    sizes = np.where(np.arange(ctx + n) < 200, 0.0, size)
    c = laid_out(bits, dtype, ctx, n, group, d, scores, sizes, seed=3)
    out, lse = c.attend(i32(tree("chain", n, None)), scale=1.0)
    assert torch.isfinite(out).all()
    if lower < 80.0:
        c.check([tree("chain", n, None)], scale=1.0, out=out, lse=lse)
    else:   # a weight below 2^-126 is 0 in fp32: nothing is left, or what it would have been
        most = size * 2.0 ** (bits - 1) * 2.0 ** (-lower / np.log(2.0))
        assert (out.double().abs() <= most + 2.0 ** -24).all()


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("power", [110, 120, 124])
def test_large_queries_of_small_keys(bits, d, n, group, power):
    """Queries of 2^power and keys that are smaller by as much: the scores are ordinary ones."""
    c = Case(bits, "bf16", [300, 20], n, 2, group, d, 16, seed=power)
    c.q = (c.q.float().clamp(-3, 3) * 2.0 ** power).bfloat16()
    c.s[..., 0] = (c.s[..., 0].float() * 2.0 ** -power).bfloat16()
    c.check([tree("tree", n, np.random.default_rng(1)) if n > 3 else [-1, 0, 0]] * 2)


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("low,high", [(-40, 40), (-100, -20), (0, 25), (20, 90)])
def test_values_over_many_powers_of_two(bits, d, n, group, low, high):
    c = Case(bits, "bf16", [700, 131], n, 2, group, d, 16, seed=21)
    g = torch.Generator(device="cuda").manual_seed(3)
    e = torch.randint(low, high + 1, c.s.shape[:3], device="cuda", generator=g).float()
    c.s[..., 1] = (c.s[..., 1].float() * torch.exp2(e)).bfloat16()
    c.check([tree("tree", n, np.random.default_rng(1)) if n > 3 else [-1, 0, 0]] * 2, scale=0.5)


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("dtype,size", [("fp16", 300.0), ("bf16", 300.0), ("bf16", 2.0 ** 60)])
@pytest.mark.parametrize("lower", [30.0, 100.0])
def test_rows_of_zeros_before_large_values_in_one_run(bits, d, n, group, dtype, size, lower):
    """The same with more tiles than blocks, so that a block has rows of zeros first and large values in a later tile."""
    ctx, b = 700, 160
    c = Case(bits, dtype, [ctx] * b, n, 4, group, d, 16, seed=3)
    first = (torch.arange(c.k.shape[1] * c.table.shape[1], device="cuda") < 400).view(c.table.shape[1], -1)
    pages = c.table.long()
    low, high = (0x77, 0x99) if bits == 4 else (127, 129)
    c.q[...] = 1.0
    c.k[pages] = torch.where(first, high, low).to(torch.uint8)[None, :, :, None, None]
    c.s[pages, :, :, 0] = torch.where(first, 0.0, lower / d).bfloat16()[None, :, :, None]
    c.s[pages, :, :, 1] = torch.where(first, 0.0, size).bfloat16()[None, :, :, None]
    out, lse = c.attend(i32(tree("chain", n, None)), scale=1.0)
    tf.tf_device_error()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    if lower < 80.0:
        c.lens = c.lens[:1]
        c.check([tree("chain", n, None)], scale=1.0, out=out[:1], lse=lse[:1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [64, 90, 126])
def test_norm_rope_small_elements_of_large_rows(d, power):
    """One element of 2^power, the others from 2^-3 to 2^-115 of it: each keeps its bits, as far as bf16 has them."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((2, 7, 3, d), device="cuda", generator=g).double().clamp(-1.9, 1.9)
    x = x * torch.exp2(power - 3.0 - 112.0 * torch.rand(x.shape, device="cuda", generator=g).double())
    x[..., 5] = 1.5 * 2.0 ** power
    x = x.bfloat16()
    pos = torch.zeros((2, 7), dtype=torch.int32, device="cuda")
    got, _ = tf.tf_qk_norm_rope(x, None, pos, eps=0.0)
    tf.tf_device_error()
    want, mag = qo.norm_rope(f64(x), 1.0, np.zeros((2, 7)), [], 0.0, False, False)
    off = np.abs(f64(got) - want)
    assert np.all(off <= qo.norm_rope_bound(want, mag, "bf16", np.zeros((2, 7)), np.zeros(0), d))


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("which", [0, 1])
def test_factors_that_differ_in_some_places_only(bits, d, n, group, which):
    """Tiles whose keys are alike beside tiles, and parts of tiles, whose are not; factors of either sign."""
    c = Case(bits, "bf16", [900, 333], n, 2, group, d, 16, seed=31)
    g = torch.Generator(device="cuda").manual_seed(5)
    c.s *= torch.where(torch.rand(c.s.shape, device="cuda", generator=g) < 0.5, -1.0, 1.0).bfloat16()
    for i, ln in enumerate(c.lens):
        pg, rw = places(c, i, [s for s in range(ln) if 150 <= s < 170 or s % 211 == 3])
        c.s[pg, rw, :, which] *= 2.0 ** (-21 if which == 0 else 13)
        pg, rw = places(c, i, list(range(200, 230)))
        c.s[pg, rw, :, which] = 0.0
    c.check([tree("tree", n, np.random.default_rng(1)) if n > 3 else [-1, 0, 0]] * 2)


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("page", [16, 7])
def test_pages_outside_the_pool_are_left_out(bits, d, n, group, page):
    """The other slots weigh what they would if those of the page were not there, whatever lies beside them."""
    lens = [500, 40]
    c = Case(bits, "bf16", lens, n, 2, group, d, page, seed=17)
    par = tree("tree", n, np.random.default_rng(1)) if n > 3 else [-1, 0, 0]
    table = c.table.clone()
    bad = [[1, 2, 9, 30 // (page // 7)], [2]]
    for i, pages in enumerate(bad):
        for j, p in enumerate(pages):
            table[i, p] = (c.k.shape[0], -1, 1 << 30, -(1 << 31))[j]
    out, lse = tf.tf_kvq_attention(c.q, c.k, c.v, c.s, table, c.lengths, i32(par))
    with pytest.raises(tf.TFError) as e:
        tf.tf_device_error()
    assert e.value.status == tf.TF_ERR_INDEX
    kk, vv = (qo.unpack(x.cpu().numpy(), bits) for x in (c.k, c.v))
    ss, qq = f64(c.s), f64(c.q)
    for i, ln in enumerate(lens):
        total = ln + n
        pg, rw = so.slot_rows(c.table[i].cpu().numpy(), page, total)
        seen = np.ones((n, total), dtype=bool)
        seen[:, ln:] = so.seen_nodes(par)
        seen[:, np.isin(np.arange(total) // page, bad[i])] = False
        o, l, mag, err, top = qo.attend(qq[i], kk[pg, rw], ss[pg, rw, :, 0], vv[pg, rw], ss[pg, rw, :, 1], seen, d ** -0.5, bits)
        tol_o, tol_l = qo.attend_bounds(o, l, mag, err, top, "bf16", total, bits)
        assert np.all(np.abs(f64(lse[i]) - l) <= tol_l) and np.all(np.abs(f64(out[i]) - o) <= tol_o)


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("power", [10, 24, 28, 32, 40, 60, 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_any_size_find_the_largest(bits, d, n, group, power, sign):
    """Scores of +-2^power, one of them an eighth above the others: its value is the result, far from fp32's
    resolution at that size (from 10 on the others' weights are below 2^-100)."""
    ctx, top = 500, 321
    s = np.arange(ctx + n)
    scores = 2.0 ** power * (0.5 + 0.25 * np.cos(s) ** 2) if sign > 0 else -(2.0 ** power) * (1.0 + 0.25 * np.cos(s) ** 2)
    scores[top] = sign * 2.0 ** power * (1.0 if sign > 0 else 0.875)
    c = laid_out(bits, "bf16", ctx, n, group, d, scores, np.full(ctx + n, 0.5), seed=power)
    out, lse = c.attend(i32(tree("chain", n, None)), scale=1.0)
    tf.tf_device_error()
    pg, rw = places(c, 0, [top])
    value = 0.5 * qo.unpack(c.v[pg, rw].cpu().numpy(), bits)[0]                       # [kh, d]
    want = np.repeat(value, group, 0)[None]
    # codes of up to 7 bits times a half are exact in bf16; the others weigh 2^-100 in all
    assert np.array_equal(f64(out[0]), np.broadcast_to(want, (n, 2 * group, d)))
    most = f64(c.s[pg, rw, :, 0])[0] * d * sign                                       # bf16 factors times d: exact
    want_l = np.broadcast_to(np.repeat(most, group)[None], (n, 2 * group))
    assert np.all(np.abs(f64(lse[0]) - want_l) <= (2 * d + 4) * 2.0 ** -24 * np.abs(want_l) * (1 + 2.0 ** (bits - 1)))


@pytest.mark.parametrize("bits,d,n,group", FORMS)
@pytest.mark.parametrize("power", [12, 34, 60])
@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -60, 2.0 ** 90])
@pytest.mark.parametrize("mixed", [False, True])
def test_values_of_any_size_under_large_scores(bits, d, n, group, power, size, mixed):
    """The value of the one key that weighs is the result, where scores are so large that a value's exponent is
    less than their resolution; mixed: values beside it are larger or smaller by many powers."""
    ctx, top = 500, 321
    s = np.arange(ctx + n)
    scores = 2.0 ** power * (0.5 + 0.25 * np.cos(s) ** 2)
    scores[top] = 2.0 ** power
    sizes = size * np.where(mixed & (s % 3 == 1), 2.0 ** -20, 1.0) * np.where(mixed & (s % 5 == 1), 2.0 ** 20, 1.0)
    sizes[top] = size
    c = laid_out(bits, "bf16", ctx, n, group, d, scores, sizes, seed=power)
    out, lse = c.attend(i32(tree("chain", n, None)), scale=1.0)
    tf.tf_device_error()
    pg, rw = places(c, 0, [top])
    value = size * qo.unpack(c.v[pg, rw].cpu().numpy(), bits)[0]
    assert np.array_equal(f64(out[0]), np.broadcast_to(np.repeat(value, group, 0)[None], (n, 2 * group, d)))
    assert torch.isfinite(lse).all()
