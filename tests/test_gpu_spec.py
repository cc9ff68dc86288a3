"""The cache, tree attention and draft verification operators on the GPU,
against the plain 64-bit forms of spec_oracle.py: types, head layouts,
lengths from nothing to long, odd pages and strides, trees with absent nodes,
what is masked holding NaN and infinities, offsets past 32 bits, streams and
graphs, and the refusals."""

import numpy as np
import pytest

import spec_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


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
    if kind == "roots":            # nodes without a parent, each alone
        return [-1] * n
    par = [-1] + [int(rng.integers(max(0, j - 6), j)) for j in range(1, n)]
    if kind == "padded":
        for j in range(n - max(1, n // 3), n):
            par[j] = -2
    if kind == "holes":            # an absent node inside: its children see no further up than themselves
        for j in range(2, n, 3):
            par[j] = -5
    return par


class Case:
    """A paged cache with scattered pages and the sequences' own parts of it."""

    def __init__(self, dtype, lens, n, kh, group, d, page, seed=0, spare=2, layout="nhd", fill=None, layers=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.lens, self.n, self.kh, self.h, self.d, self.page = dtype, lens, n, kh, kh * group, d, page
        b = len(lens)
        per = max(1, -(-(max(max(lens), 0) + n) // page))
        pages = b * per + spare
        dt = DT[dtype]
        if layout == "nhd":
            shape = (pages, page, kh, d)
            self.k = torch.randn(shape, device="cuda", generator=g).to(dt)
            self.v = torch.randn(shape, device="cuda", generator=g).to(dt)
        elif layout == "hnd":
            shape = (pages, kh, page, d)
            self.k = torch.randn(shape, device="cuda", generator=g).to(dt).transpose(1, 2)
            self.v = torch.randn(shape, device="cuda", generator=g).to(dt).transpose(1, 2)
        else:   # both in one tensor, rows padded
            both = torch.randn((pages, 2, page, kh, d + 8), device="cuda", generator=g).to(dt)
            self.k, self.v = both[:, 0, :, :, :d], both[:, 1, :, :, :d]
        perm = torch.randperm(pages, device="cuda", generator=g)[: b * per]
        self.table = perm.to(torch.int32).view(b, per).contiguous()
        self.lengths = i32(lens)
        rows = torch.randn((b, n, (self.h + 2 * kh) * d), device="cuda", generator=g).to(dt)
        self.q = rows[:, :, : self.h * d].view(b, n, self.h, d)
        if fill is not None:       # every slot that no row may see
            used = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
            for i, ln in enumerate(lens):
                if ln < 0:
                    continue
                s = torch.arange(ln + n, device="cuda")
                used[self.table[i].long()[s // page], s % page] = True
            self.k[~used] = fill
            self.v[~used] = fill

    def check(self, parents, scale=None, out=None, lse=None):
        b = len(self.lens)
        par = np.broadcast_to(np.asarray(parents, dtype=np.int64), (b, self.n))
        if out is None:
            out, lse = tf.tf_tree_attention(self.q, self.k, self.v, self.table, self.lengths, i32(parents),
                                            scale=scale)
            tf.tf_device_error()
        scale = self.d ** -0.5 if scale is None else scale
        kk, vv, qq, tb = f64(self.k), f64(self.v), f64(self.q), self.table.cpu().numpy()
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
            k, v = kk[pg, rw], vv[pg, rw]
            o, l, mag, err = so.attend(qq[i], k, v, seen, scale)
            tol_o, tol_l = so.attend_bounds(o, l, mag, err, self.dtype, total)
            assert np.array_equal(np.isneginf(got_l[i]), np.isneginf(l)), i
            fin = np.isfinite(l)
            off = np.abs(got_l[i][fin] - l[fin])
            assert np.all(off <= tol_l[fin]), (i, off.max())
            bad = ~(np.abs(got_o[i] - o) <= tol_o)
            assert not bad.any(), (i, np.argwhere(bad)[:4].tolist(), np.abs(got_o[i] - o).max())
            assert np.all(got_o[i][~fin] == 0)
        return out, lse


# --------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kh,group,d", [(8, 5, 128), (2, 1, 64), (1, 8, 128), (1, 3, 256), (3, 7, 64), (1, 16, 128)])
@pytest.mark.parametrize("n,kind", [(1, "chain"), (5, "tree"), (16, "padded"), (40, "tree")])
def test_attention_heads_and_trees(dtype, kh, group, d, n, kind):
    rng = np.random.default_rng(n * 100 + kh)
    lens = [200, 0, 77]
    Case(dtype, lens, n, kh, group, d, 16, seed=n).check([tree(kind, n, rng) for _ in lens])


@pytest.mark.parametrize("page", [1, 7, 8, 16, 17, 24, 64, 128, 200, 256, 300])
@pytest.mark.parametrize("n", [1, 20])
def test_attention_page_sizes(page, n):
    rng = np.random.default_rng(page)
    lens = [page * 3 - 1, page, 129, 500]
    Case("fp16", lens, n, 2, 4, 128, page, seed=page).check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("n", [1, 3, 64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [2, 127], [128, 126], [129, 63, 64, 65], [1000, 0, 5, 31, 32, 33]])
def test_attention_lengths(n, lens):
    rng = np.random.default_rng(len(lens))
    Case("bf16", lens, n, 2, 2, 128, 32, seed=n).check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("n", [1, 30])
def test_attention_long_context_is_split_and_joined(n):
    rng = np.random.default_rng(5)
    Case("bf16", [9001], n, 1, 4, 128, 64, seed=5).check([tree("tree", n, rng)])
    Case("fp16", [7000, 3], n, 1, 5, 64, 16, seed=6).check([tree("tree", n, rng), tree("star", n, rng)])


@pytest.mark.parametrize("b,n", [(300, 1), (129, 6), (700, 2), (32, 1), (33, 12), (100, 2), (400, 12)])
def test_attention_large_batches(b, n):
    """More sequences than a block scans at once, lengths of all kinds."""
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(-1, 90, b)]
    lens[7] = 400
    Case("bf16", lens, n, 1, 2, 64, 16, seed=b).check(tree("chain", n, rng))


@pytest.mark.parametrize("kind", ["star", "roots", "holes", "padded", "chain"])
@pytest.mark.parametrize("n", [2, 33, 128])
def test_attention_tree_shapes(kind, n):
    rng = np.random.default_rng(n)
    lens = [130, 0, -1, 64]
    par = [tree(kind, n, rng) for _ in lens]
    par[1] = [-2] * n                     # nothing present: every row empty
    Case("fp16", lens, n, 2, 3, 64, 16, seed=n + 1).check(par)


def test_attention_one_tree_for_all_and_strided_parents():
    rng = np.random.default_rng(9)
    c = Case("bf16", [50, 60, 70], 12, 2, 4, 128, 16, seed=9)
    par = tree("tree", 12, rng)
    o, l = c.check(par)
    wide = torch.full((3, 20), -7, dtype=torch.int32, device="cuda")
    wide[:, :12] = i32(par)
    o2, l2 = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, wide[:, :12])
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("layout", ["hnd", "both"])
@pytest.mark.parametrize("page,n", [(16, 1), (64, 24), (7, 3)])
def test_attention_cache_layouts(layout, page, n):
    rng = np.random.default_rng(3)
    Case("bf16", [300, 41], n, 3, 4, 128, page, seed=3, layout=layout).check([tree("tree", n, rng)] * 2)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 65504.0])
@pytest.mark.parametrize("n,group", [(1, 4), (9, 4), (40, 5)])
def test_attention_unseen_slots_have_no_influence(fill, n, group):
    rng = np.random.default_rng(2)
    lens = [131, 0, 63, 255]
    Case("fp16", lens, n, 2, group, 128, 32, seed=2, fill=fill).check([tree("tree", n, rng) for _ in lens])


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("group,d", [(1, 64), (5, 128), (2, 256)])
def test_attention_a_siblings_bad_row_stays_its_own(fill, group, d):
    """Node 3's key and value are not finite: rows that see it are spoilt,
    the others keep the bits they have without it."""
    rng = np.random.default_rng(4)
    n = 24
    par = tree("tree", n, rng)
    seen = so.seen_nodes(par)
    for ln in (100, 0):
        c = Case("bf16", [ln], n, 2, group, d, 16, seed=4)
        want, want_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par))
        s = ln + 3
        pg = int(c.table[0, s // 16])
        c.v[pg, s % 16] = fill
        got, got_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par))
        hit = torch.tensor(seen[:, 3], device="cuda")
        assert torch.equal(got[0, ~hit], want[0, ~hit]) and torch.equal(got_l, want_l)
        assert not torch.isfinite(got[0, hit]).any()
        c.k[pg, s % 16] = float("nan")
        got, got_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par))
        assert torch.equal(got[0, ~hit], want[0, ~hit]) and torch.equal(got_l[0, ~hit], want_l[0, ~hit])
        assert torch.isnan(got[0, hit]).all() and torch.isnan(got_l[0, hit]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(3, 2), (4, 5), (40, 4)])
def test_attention_weights_over_the_whole_range(dtype, d, n, group):
    """Scores from the maximum down to weights that vanish, in shuffled slots:
    every place of a tile meets large, small and vanished weights. An infinite
    key's score of -inf is a weight of 0, as that of -160 is in fp32."""
    ln = 700
    c = Case(dtype, [ln], n, 1, group, d, 16, seed=12)
    g = torch.Generator(device="cuda").manual_seed(5)
    score = (torch.randint(-640, 1, (ln + n,), device="cuda", generator=g) / 4).to(c.k.dtype)
    score[::7] = score[::7] / 8
    score[3::50] = -160.0
    score[0] = 0.0
    score[ln:] = -1.0
    s = torch.arange(ln + n, device="cuda")
    c.q.zero_()
    c.q[..., 0] = 1.0
    c.k[c.table[0].long()[s // 16], s % 16] = 0.0
    c.k[c.table[0].long()[s // 16], s % 16, :, 0] = score[:, None]
    par = [tree("tree", n, np.random.default_rng(1))]
    want, want_l = c.check(par, scale=1.0)
    score[3::50] = -float("inf")
    score[ln:] = -1.0
    c.k[c.table[0].long()[s // 16], s % 16, :, 0] = score[:, None]
    got, got_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par), scale=1.0)
    assert torch.equal(got, want) and torch.equal(got_l, want_l)


def test_attention_rising_and_falling_scores():
    """Scores that climb or fall by hundreds along the context: the running
    maximum has to move, and early or late parts vanish."""
    for sign in (1.0, -1.0):
        c = Case("bf16", [1500], 3, 1, 2, 64, 16, seed=8)
        ramp = torch.linspace(-20, 20, 1503, device="cuda") * sign
        s = torch.arange(1503, device="cuda")
        pages = c.table[0].long()[s // 16]
        c.q[..., 0] = 8.0
        c.k[pages, s % 16, :, 0] = ramp[:, None].to(torch.bfloat16)
        c.check([[-1, 0, 1]], scale=1.0)


def test_attention_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31 and byte offsets 2^32."""
    kh, d, page = 8, 128, 128
    pages = (1 << 31) // (kh * d * page) + 40
    k = torch.empty((pages, page, kh, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for n in (1, 20):
        c = Case("bf16", [1000, 300], n, kh, 4, d, page, seed=11)
        lift = pages - c.k.shape[0]
        k[lift:] = c.k
        v[lift:] = c.v
        par = [tree("chain", n, None)] * 2
        want, want_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par))
        got, got_l = tf.tf_tree_attention(c.q, k, v, c.table + lift, c.lengths, i32(par))
        assert torch.equal(got, want) and torch.equal(got_l, want_l)
        new = torch.randn((2, n, kh, d), device="cuda").bfloat16()
        tf.tf_kv_write(new, -new, k, v, c.table + lift, c.lengths)
        tf.tf_kv_write(new, -new, c.k, c.v, c.table, c.lengths)
        assert torch.equal(k[lift:], c.k) and torch.equal(v[lift:], c.v)


@pytest.mark.parametrize("n,group,d", [(1, 5, 128), (16, 6, 128), (3, 1, 64), (64, 5, 128)])
def test_attention_same_bits_every_time_and_on_two_streams(n, group, d):
    rng = np.random.default_rng(1)
    lens = [3000, 17, 900]
    c = Case("bf16", lens, n, 2, group, d, 32, seed=1)
    par = i32([tree("tree", n, rng) for _ in lens])
    want, want_l = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, par)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, par))
    got.append(tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, par, stream=streams[0]))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_l)
    tf.tf_device_error()


@pytest.mark.parametrize("n", [1, 24])
def test_attention_workspace_serves_other_sizes_and_a_graph(n):
    rng = np.random.default_rng(6)
    big = Case("fp16", [5000, 100], n, 2, 5, 128, 64, seed=6)
    small = Case("fp16", [40], 2, 1, 1, 64, 16, seed=7)
    ws = tf.tf_tree_attention_workspace(2, n, 10, 2, 128)
    pb, ps = i32([tree("tree", n, rng)] * 2), i32([[-1, 0]])
    first = tf.tf_tree_attention(big.q, big.k, big.v, big.table, big.lengths, pb, workspace=ws)
    tf.tf_tree_attention(small.q, small.k, small.v, small.table, small.lengths, ps, workspace=ws)
    again = tf.tf_tree_attention(big.q, big.k, big.v, big.table, big.lengths, pb, workspace=ws)
    assert torch.equal(first[0], again[0])
    outs = []
    for use in (ws, None):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(tf.tf_tree_attention(big.q, big.k, big.v, big.table, big.lengths, pb, workspace=use))
        for _ in range(3):
            outs[-1][0].fill_(7)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[-1][0], first[0]) and torch.equal(outs[-1][1], first[1])
    tf.tf_device_error()


def test_attention_one_workspace_for_many_sizes_in_turn():
    """Counters and parts of calls of different sizes must not lie over one
    another: one workspace, calls of many sizes in turn, twice."""
    rng = np.random.default_rng(12)
    ws = tf.tf_tree_attention_workspace(64, 40, 40, 8, 128)
    cases = [Case("bf16", [200, 0, 77], 40, 8, 5, 128, 16, seed=1), Case("bf16", [3000], 1, 1, 1, 64, 64, seed=2),
             Case("bf16", [30] * 64, 3, 4, 4, 64, 16, seed=3), Case("bf16", [900, 800], 20, 4, 2, 128, 32, seed=4),
             Case("bf16", [5000], 16, 2, 8, 128, 64, seed=5)]
    trees = [i32([tree("tree", c.n, rng) for _ in c.lens]) for c in cases]
    fresh = [tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, t,
                                  workspace=tf.tf_tree_attention_workspace(64, 40, 40, 8, 128))
             for c, t in zip(cases, trees)]
    for _ in range(2):
        for c, t, (o, l) in zip(cases, trees, fresh):
            o2, l2 = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, t, workspace=ws)
            assert torch.equal(o, o2) and torch.equal(l, l2)
    for c, t in zip(cases, trees):
        c.check(t.tolist())


def test_attention_workspace_for_the_largest_sizes_serves_fewer_kv_heads():
    need = tf.lib().tf_tree_attention_workspace_bytes
    rng = np.random.default_rng(3)
    for heads, kv, n, d in ((8, 8, 4, 64), (16, 8, 16, 128), (24, 6, 9, 128)):
        ws = tf.tf_tree_attention_workspace(2, n, heads, kv, d)
        smaller = [need(2, m, h, k, e) for m in (1, n) for h in (heads // 2, heads) for k in range(1, kv + 1)
                   for e in (64, d) if h % k == 0]
        assert max(smaller) <= ws.numel()
        for k in (1, 2, kv):
            c = Case("bf16", [700, 90], n, k, heads // k, d, 16, seed=k)
            par = [tree("tree", n, rng)] * 2
            got = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32(par), workspace=ws)
            c.check(par, out=got[0], lse=got[1])
    assert tf.tf_tree_attention_workspace(2, 4, 8, 3, 64).numel() == 1   # refused sizes


def test_attention_bad_indices_are_skipped_and_recorded():
    c = Case("fp16", [100, 100], 4, 1, 2, 64, 16, seed=13)
    par = i32([[-1, 0, 1, 2]] * 2)
    want, _ = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, par)
    table = c.table.clone()
    table[1, 2], table[1, 3] = c.k.shape[0], -1
    got, _ = tf.tf_tree_attention(c.q, c.k, c.v, table, c.lengths, par)
    with pytest.raises(tf.TFError) as e:
        tf.tf_device_error()
    assert e.value.status == tf.TF_ERR_INDEX
    tf.tf_device_error()
    assert torch.equal(got[0], want[0]) and torch.isfinite(got).all() and not torch.equal(got[1], want[1])
    # pages past the end that no row needs are not looked at
    wide = torch.cat([c.table, torch.full((2, 3), 1 << 30, dtype=torch.int32, device="cuda")], 1).contiguous()
    got, _ = tf.tf_tree_attention(c.q, c.k, c.v, wide, c.lengths, par)
    tf.tf_device_error()
    assert torch.equal(got, want)
    # a context longer than the table, and a parent that is no earlier node
    got, _ = tf.tf_tree_attention(c.q, c.k, c.v, c.table, i32([100, 10 ** 9]), par)
    with pytest.raises(tf.TFError):
        tf.tf_device_error()
    assert torch.equal(got[0], want[0]) and torch.isfinite(got).all()
    got, lse = tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, i32([[-1, 0, 1, 2], [-1, 1, 9, 0]]))
    with pytest.raises(tf.TFError):
        tf.tf_device_error()
    assert torch.equal(got[0], want[0]) and torch.isneginf(lse[1, 1:3]).all() and (got[1, 1:3] == 0).all()


# ------------------------------------------------------------------- cache
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,kh,d,page,layout", [(1, 8, 128, 16, "nhd"), (5, 3, 64, 7, "hnd"), (64, 2, 256, 32, "both"),
                                                (17, 1, 8, 1, "nhd")])
def test_write_puts_every_node_in_its_slot(dtype, n, kh, d, page, layout):
    lens = [0, 45, -1, 31]
    c = Case(dtype, lens, n, kh, 1, d, page, seed=n, layout=layout)
    rows = torch.randn((4, n, 5 * kh * d), device="cuda").to(DT[dtype])
    kn, vn = rows[..., kh * d: 2 * kh * d].view(4, n, kh, d), rows[..., 3 * kh * d: 4 * kh * d].view(4, n, kh, d)
    want_k, want_v = c.k.clone(), c.v.clone()
    for i, ln in enumerate(lens):
        if ln < 0:
            continue
        s = ln + torch.arange(n, device="cuda")
        pg = c.table[i].long()[s // page]
        want_k[pg, s % page], want_v[pg, s % page] = kn[i], vn[i]
    tf.tf_kv_write(kn, vn, c.k, c.v, c.table, c.lengths)
    tf.tf_device_error()
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("n,kh,d,page", [(8, 8, 128, 16), (128, 2, 64, 7), (2, 1, 8, 1), (33, 3, 128, 32)])
def test_keep_moves_the_path_together(layers, n, kh, d, page):
    rng = np.random.default_rng(n)
    lens = [0, 45, -1, 31, 8]
    b = len(lens)
    c = Case("bf16", lens, n, kh, 1, d, page, seed=n)
    k = c.k if layers is None else torch.stack([c.k + i for i in range(layers)])
    v = c.v if layers is None else torch.stack([c.v - i for i in range(layers)])
    counts = [n, int(rng.integers(1, n + 1)), 1, 0, max(1, n // 2)]
    path = np.full((b, n), -1)
    for i, m in enumerate(counts):
        path[i, :m] = np.sort(rng.permutation(n)[:m])
    want_k, want_v = k.clone(), v.clone()
    wk, wv = want_k.view((-1,) + c.k.shape), want_v.view((-1,) + c.v.shape)
    for i, ln in enumerate(lens):
        if ln < 0:
            continue
        to = ln + torch.arange(counts[i], device="cuda")
        src = ln + torch.tensor(path[i, :counts[i]], device="cuda")
        at = lambda s: (c.table[i].long()[s // page], s % page)  # noqa: E731
        for w in (wk, wv):
            rows = w[:, at(src)[0], at(src)[1]].clone()
            w[:, at(to)[0], at(to)[1]] = rows
    new = tf.tf_kv_keep(k, v, c.table, c.lengths, i32(path), i32(counts))
    tf.tf_device_error()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
    assert new.tolist() == [ln + m if ln >= 0 else ln for ln, m in zip(lens, counts)]


def test_keep_and_write_skip_bad_indices():
    c = Case("fp16", [10, 10], 4, 1, 1, 64, 16, seed=1)
    k0, v0 = c.k.clone(), c.v.clone()
    new = tf.tf_kv_keep(c.k, c.v, c.table, c.lengths, i32([[2, 1, 3, -1], [0, 1, 4, -1]]), i32([3, 9]))
    with pytest.raises(tf.TFError) as e:
        tf.tf_device_error()
    assert e.value.status == tf.TF_ERR_INDEX
    pg = int(c.table[0, 0])
    k0[pg, 10], v0[pg, 10] = k0[pg, 12], v0[pg, 12]
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0) and new.tolist() == [11, 12]
    kn = torch.ones((2, 4, 1, 64), dtype=torch.float16, device="cuda")
    table = i32([[c.k.shape[0]], [-3]])
    tf.tf_kv_write(kn, kn, c.k, c.v, table, c.lengths)
    with pytest.raises(tf.TFError):
        tf.tf_device_error()
    tf.tf_kv_write(kn, kn, c.k, c.v, c.table, i32([1 << 20, 2 ** 31 - 2]))
    with pytest.raises(tf.TFError):
        tf.tf_device_error()
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)


# ------------------------------------------------------------ verification
def logits_like(b, n, v, dtype, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = spread * torch.randn((b, n, v), device="cuda", generator=g)
    at = torch.randint(0, v, (b, n, min(6, v)), device="cuda", generator=g)
    x.scatter_add_(2, at, 4 + 6 * torch.rand((b, n, min(6, v)), device="cuda", generator=g))
    d = x + 0.7 * torch.randn((b, n, v), device="cuda", generator=g)
    return x.to(DT[dtype]), d.to(DT[dtype]), g


def verify_and_check(x, tokens, par, us, temperature, d=None, ua=None, name=""):
    b, n, v = x.shape
    got = tf.tf_verify_draft(x, tokens, i32(par), us, temperature=temperature, draft_logits=d, u_accept=ua)
    tf.tf_device_error()
    c, p, o, l = [t.cpu().numpy() for t in got]
    par = np.broadcast_to(np.asarray(par), (b, n))
    for i in range(b):
        so.check_walk(f64(x[i]), tokens[i].tolist(), list(par[i]), us[i].tolist() if us is not None else None,
                      temperature, None if d is None else f64(d[i]), None if ua is None else ua[i].tolist(),
                      (int(c[i]), p[i], o[i], l[i]), "seq %d %s" % (i, name))
    return got


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("v", [1, 2, 31, 1000, 4097, 50001, 129280])
@pytest.mark.parametrize("temperature", [0.0, 0.7, 1.0])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_walks(dtype, v, temperature, with_draft):
    b, n = (6, 9) if v < 20000 else (3, 5)
    rng = np.random.default_rng(v)
    x, d, g = logits_like(b, n, v, dtype, v + n)
    par = [tree(("tree", "chain", "star")[i % 3], n, rng) for i in range(b)]
    if b > 4:
        par[4] = tree("padded", n, rng)
        par[5][0] = -2                                  # an idle sequence
    up = torch.tensor(par, device="cuda").clamp(min=0)
    if with_draft:
        rows = torch.gather(d.float(), 1, up[:, :, None].expand(b, n, v)) / max(temperature, 0.5)
        tok = (rows - torch.log(-torch.log(torch.rand(rows.shape, device="cuda", generator=g).clamp(1e-9, 1 - 1e-6)))).argmax(-1)
    else:
        k = min(3, v)
        best = torch.topk(x.float(), k, dim=-1).indices
        tok = torch.gather(best, 1, up[:, :, None].expand(b, n, k))
        tok = torch.gather(tok, 2, torch.randint(0, k, (b, n, 1), device="cuda", generator=g))[..., 0]
    us = torch.rand((b, n), device="cuda", generator=g)
    ua = torch.rand((b, n), device="cuda", generator=g) if with_draft else None
    verify_and_check(x, tok.int(), par, us, temperature, d if with_draft else None, ua)


@pytest.mark.parametrize("dtype,off", [("fp32", 0), ("fp32", 1), ("bf16", 3), ("fp16", 0)])
@pytest.mark.parametrize("b,n", [(10, 20), (32, 9), (60, 5), (200, 3)])   # 8, 4, 2 blocks a sequence, and 1
@pytest.mark.parametrize("mode", ["greedy", "sampled", "draft"])
def test_verify_large_batches_walk_down_their_trees(dtype, off, b, n, mode):
    """More rows than SMs: a cluster walks down a sequence's tree, from node to
    node with refusals on the way. Against the definition, and bit for bit
    against the same sequences a few at a time, which are not walked. Padded
    and idle sequences among them; rows that begin off a 16-byte boundary."""
    assert b * n > torch.cuda.get_device_properties(0).multi_processor_count
    v, rng = 2003, np.random.default_rng(b)
    x, d, g = logits_like(b, n, v + 8, dtype, b + n, spread=1.0)
    x, d = x[:, :, off:off + v], d[:, :, off:off + v]
    par = [tree(("chain", "tree", "star", "padded")[i % 4], n, rng) for i in range(b)]
    for i in range(7, b, 10):
        par[i] = [-2] + par[i][1:]
    up = torch.tensor(par, device="cuda").clamp(min=0)
    if mode == "draft":    # drawn from the parent's draft row
        rows = torch.gather(d.float(), 1, up[:, :, None].expand(b, n, v)) / 0.8
        u = torch.rand(rows.shape, device="cuda", generator=g).clamp(1e-9, 1 - 1e-6)
        tok = (rows - torch.log(-torch.log(u))).argmax(-1)
    else:                  # one of the parent's two best
        best = torch.gather(torch.topk(x.float(), 2, dim=-1).indices, 1, up[:, :, None].expand(b, n, 2))
        tok = torch.gather(best, 2, torch.randint(0, 2, (b, n, 1), device="cuda", generator=g))[..., 0]
    tok = tok.int()
    us, ua = (torch.rand((b, n), device="cuda", generator=g) for _ in range(2))
    t = 0.0 if mode == "greedy" else 0.8
    dr = d if mode == "draft" else None
    got = verify_and_check(x, tok, par, us, t, dr, ua if mode == "draft" else None)
    assert int(got[0].max()) >= 2 and int(got[0].min()) == 0   # some went down, some are idle
    few = 100 // n
    for i in range(0, b, few):
        at = slice(i, i + few)
        part = tf.tf_verify_draft(x[at], tok[at], i32(par[at]), us[at], temperature=t,
                                  draft_logits=None if dr is None else dr[at],
                                  u_accept=ua[at] if mode == "draft" else None)
        assert all(torch.equal(p, q[at]) for p, q in zip(part, got)), i
    tf.tf_device_error()


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("temperature", [0.6, 0.8, 1.0, 1.3])
@pytest.mark.parametrize("v", [257, 129280])
def test_verify_one_row_is_the_definition_to_the_last_bit(dtype, temperature, v):
    """Every step of the definition is one fp32 operation or exact, so the
    tokens and log-probabilities are those of the same steps done one by one."""
    x, _, g = logits_like(8, 3, v, dtype, v + 1)
    us = torch.rand((8, 3), device="cuda", generator=g)
    tok = torch.zeros((8, 3), dtype=torch.int32, device="cuda")
    _, _, out, logp = tf.tf_verify_draft(x.view(24, 1, v), tok.view(24, 1), i32([[-1]] * 24), us.view(24, 1),
                                         temperature=temperature)
    z = x.float() * torch.tensor(1.0 / temperature, dtype=torch.float32, device="cuda")
    top = z.amax(-1, keepdim=True)
    w = torch.round(torch.exp(z - top) * 2.0 ** 30).long()
    mass = w.sum(-1)
    goal = torch.floor(us.double() * mass.double()).long()
    want = (torch.cumsum(w, -1) <= goal[..., None]).sum(-1)
    assert torch.equal(out.view(8, 3).long(), want)
    lp = (torch.gather(z, 2, want[..., None])[..., 0] - top[..., 0]) - torch.log(mass.float() * 2.0 ** -30)
    assert torch.equal(logp.view(8, 3), lp)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("v", [300, 50003])
def test_verify_the_rest_of_a_distribution_is_the_definition_to_the_last_bit(dtype, v):
    """A refused child (u = 1 - 2^-24 against a token the target finds
    unlikely): the token comes from max(round(p) - round(q), 0)."""
    x, d, g = logits_like(16, 2, v, dtype, v + 2)
    q = torch.softmax(d[:, 0].float(), -1)
    tok = (q / torch.softmax(x[:, 0].float(), -1)).argmax(-1).int()[:, None].expand(16, 2).contiguous()
    us = torch.rand((16, 2), device="cuda", generator=g)
    ua = torch.full((16, 2), 1 - 2.0 ** -24, device="cuda")
    counts, _, out, _ = tf.tf_verify_draft(x, tok, i32([-1, 0]), us, draft_logits=d, u_accept=ua)
    assert counts.tolist() == [1] * 16

    def weights(y):
        z = y.float()
        return torch.exp(z - z.amax(-1, keepdim=True)), torch.round(torch.exp(z - z.amax(-1, keepdim=True)) * 2.0 ** 30).long().sum(-1)

    e, mass = weights(x[:, 0])
    f, qmass = weights(d[:, 0])
    p = torch.round(e * (2.0 ** 61 / mass.double()).float()[:, None]).long()
    r = (p - torch.round(f * (2.0 ** 61 / qmass.double()).float()[:, None]).long()).clamp(min=0)
    goal = torch.floor(us[:, 0].double() * r.sum(-1).double()).long()
    assert torch.equal(out[:, 0].long(), (torch.cumsum(r, -1) <= goal[:, None]).sum(-1))


def test_verify_strided_rows_and_shared_tree():
    """A padded head (rows longer than the vocabulary, so that a row starts
    off a 16-byte boundary) gives what a contiguous copy gives."""
    for dtype in ("fp32", "fp16", "bf16"):
        x, d, g = logits_like(3, 4, 5003, dtype, 5)
        par = [-1, 0, 0, 1]
        tok = x[:, :1, :].float().argmax(-1).int().expand(3, 4).contiguous()
        us, ua = (torch.rand((3, 4), device="cuda", generator=g) for _ in range(2))
        for v, off in ((4999, 0), (4999, 1), (4098, 3)):
            for dr in (None, d):
                a = tf.tf_verify_draft(x[:, :, off:off + v], tok, i32(par), us, draft_logits=None if dr is None else dr[:, :, off:off + v],
                                       u_accept=None if dr is None else ua)
                c = tf.tf_verify_draft(x[:, :, off:off + v].contiguous(), tok, i32([par] * 3), us,
                                       draft_logits=None if dr is None else dr[:, :, off:off + v].contiguous(),
                                       u_accept=None if dr is None else ua)
                assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_verify_extreme_logits():
    inf, low = float("inf"), torch.finfo(torch.float32).min
    nan = float("nan")
    rows = [[-inf] * 8, [nan] * 8, [low] * 8, [-inf, 1.0, -inf, nan, 2.0, low, -inf, -inf],
            [0.0, inf, 1.0, inf, -inf, nan, 3.0, 2.0], [-inf, -inf, -inf, 5.0, -inf, -inf, -inf, -inf],
            [3.0e38, -3.0e38, 3.0e38, 0.0, 0.0, 0.0, 0.0, 0.0], [1.0] * 8]
    x = torch.tensor(rows, device="cuda")[:, None, :].contiguous()
    tok = torch.zeros((8, 1), dtype=torch.int32, device="cuda")
    for u in (0.0, 0.3, 0.9999999, 1.0, 7.0, -1.0, nan):
        us = torch.full((8, 1), u, device="cuda")
        for t in (0.0, 0.5, 1.0):
            c, p, o, l = tf.tf_verify_draft(x, tok, i32([[-1]] * 8), us, temperature=t)
            o = o[:, 0].tolist()
            assert c.tolist() == [1] * 8 and o[0] == o[1] == -1 and o[5] == 3
            assert o[3] in (1, 4) and o[4] in (1, 3) and o[6] in (0, 2)
            assert l[0, 0] == 0 and l[5, 0] == 0 and abs(float(l[7, 0]) + np.log(8)) < 1e-6
            if t == 0:
                assert o[2] == 0 and o[4] == 1 and o[6] == 0 and o[7] == 0 and o[3] == 4
            else:
                uu = min(max(u if u == u else 0.0, 0.0), 0.99999994)
                assert o[7] == int(uu * 8)
                # z = logit / T: the lowest value is a value at T = 1 and overflows to -inf at 1/2
                assert o[2] == (int(uu * 8) if t == 1.0 else -1)
    tf.tf_device_error()


def test_verify_ties_go_to_the_lowest_index():
    v = 70001
    x = torch.zeros((1, 3, v), device="cuda")
    x[0, 0, [61234, 9, 40000]] = 5.0
    x[0, 1, [70000, 69999]] = 4.0
    tok = i32([[0, 9, 9]])
    c, p, o, _ = tf.tf_verify_draft(x, tok, i32([[-1, 0, 0]]), None, temperature=0.0)
    assert o.tolist() == [[9, 69999, -1]] and p.tolist() == [[0, 1, -1]] and c.tolist() == [2]


def test_verify_passes_over_tokens_outside_the_vocabulary():
    x, d, g = logits_like(2, 4, 100, "fp32", 3)
    tok = i32([[0, -1, 100, 2 ** 31 - 1]] * 2)
    us = torch.rand((2, 4), device="cuda")
    for dr in (None, d):
        verify_and_check(x, tok, [-1, 0, 0, 0], us, 1.0, dr, None if dr is None else torch.zeros((2, 4), device="cuda"))


def test_verify_equal_distributions_and_a_refusal_without_a_rest():
    """Draft and target alike: any u below 1 accepts. u = 1 refuses although
    nothing is left of the distribution: the token then comes from p itself."""
    x, _, g = logits_like(2, 3, 1000, "fp32", 8)
    tok = x[:, 0].argmax(-1).int()[:, None].expand(2, 3).contiguous()
    us = torch.full((2, 3), 0.25, device="cuda")
    ua = torch.full((2, 3), 0.999, device="cuda")
    c, p, o, _ = tf.tf_verify_draft(x, tok, i32([-1, 0, 0]), us, draft_logits=x, u_accept=ua)
    assert c.tolist() == [2, 2] and p[:, 1].tolist() == [1, 1]
    c, p, o, _ = tf.tf_verify_draft(x, tok, i32([-1, 0, 0]), us, draft_logits=x, u_accept=torch.ones_like(ua))
    want = tf.tf_verify_draft(x, tok, i32([-1, -2, -2]), us)
    assert c.tolist() == [1, 1] and o[:, 0].tolist() == want[2][:, 0].tolist()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_clamps_the_numbers_that_accept(dtype):
    """A child whose token has no weight in the target (5), one that the target
    finds 24 times likelier than the draft (7), or an ordinary one (9, 1.2
    times). u_accept outside [0, 1] counts as the nearer end, a NaN as 0."""
    v = 64
    x = torch.zeros((1, 4, v), device="cuda")
    d = torch.zeros((1, 4, v), device="cuda")
    x[..., 5], d[..., 5] = -float("inf"), 3.0
    x[..., 7], d[..., 7] = 2.0, -1.0
    x, d = x.to(DT[dtype]), d.to(DT[dtype])
    us = torch.full((1, 4), 0.5, device="cuda")

    def first(child_token, u):
        tok, ua = i32([[0, child_token, 0, 0]]), torch.full((1, 4), u, device="cuda")
        return [t.tolist() for t in tf.tf_verify_draft(x, tok, i32([[-1, 0, -2, -2]]), us, draft_logits=d, u_accept=ua)]

    nan, inf = float("nan"), float("inf")
    for low in (-0.0, -1e-30, -0.5, -7.0, -inf, nan):
        got = first(5, low)
        assert got[0] == [1] and got[2][0][0] != 5, low   # a weight of 0 is never accepted
        for t in (7, 9):
            got = first(t, low)
            assert got[0] == [2] and got[1][0][:2] == [0, 1] and got[2][0][0] == t == first(t, 0.0)[2][0][0], low
    for high in (1.0, 1.5, 40.0, inf):
        assert first(5, high)[0] == [1] and first(7, high)[0] == [2], high
        for t in (5, 7, 9):
            assert first(t, high) == first(t, 1.0), (t, high)
    tf.tf_device_error()


def test_verify_parent_out_of_order_is_recorded():
    x, _, _ = logits_like(1, 3, 50, "fp32", 8)
    tok = x[:, 0].argmax(-1).int()[:, None].expand(1, 3).contiguous()
    c, p, _, _ = tf.tf_verify_draft(x, tok, i32([[-1, 1, 0]]), None, temperature=0.0)
    with pytest.raises(tf.TFError) as e:
        tf.tf_device_error()
    assert e.value.status == tf.TF_ERR_INDEX and p.tolist()[0][:2] == [0, 2]


def test_verify_parent_out_of_order_is_recorded_in_large_batches():
    """The same where a batch has more rows than the GPU has SMs and is walked
    down, so that the malformed node is never come to."""
    b = 200
    x, _, _ = logits_like(1, 3, 50, "fp32", 8)
    x = x.expand(b, 3, 50).contiguous()
    tok = x[:, 0].argmax(-1).int()[:, None].expand(b, 3).contiguous()
    good = [[-1, 0, 0]] * b
    tf.tf_verify_draft(x, tok, i32(good), None, temperature=0.0)
    tf.tf_device_error()
    for at, par, kept in ((0, [-1, 1, 0], [0, 2]), (b - 1, [-1, -2, 2], [0]), (77, [0, 0, 0], [])):
        c, p, _, _ = tf.tf_verify_draft(x, tok, i32(good[:at] + [par] + good[at + 1:]), None, temperature=0.0)
        with pytest.raises(tf.TFError) as e:
            tf.tf_device_error()
        assert e.value.status == tf.TF_ERR_INDEX
        assert p[at].tolist() == kept + [-1] * (3 - len(kept)) and c[at] == len(kept)


@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_emits_tokens_with_the_targets_probabilities(with_draft):
    """The point of it all: over many sequences the first emitted token has
    the target's distribution, whatever the drafts were (three children drawn
    from the draft distribution, or its three best ones)."""
    b, v = 60000, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((v,), device="cuda", generator=g) * 1.5
    d = torch.randn((v,), device="cuda", generator=g) * 1.5
    p, q = torch.softmax(x.double(), 0), torch.softmax(d.double(), 0)
    if with_draft:
        tok = torch.multinomial(q.float().expand(b, v), 4, replacement=True, generator=g).int()
    else:
        tok = torch.topk(d, 4).indices.int().expand(b, 4).contiguous()
    us, ua = (torch.rand((b, 4), device="cuda", generator=g) for _ in range(2))
    rows = x.expand(b, 4, v).contiguous()
    kw = dict(draft_logits=d.expand(b, 4, v).contiguous(), u_accept=ua) if with_draft else {}
    c, path, out, _ = tf.tf_verify_draft(rows, tok, i32([-1, 0, 0, 0]), us, **kw)
    freq = torch.bincount(out[:, 0].long(), minlength=v).double() / b
    sd = (p * (1 - p) / b).sqrt()
    assert ((freq - p).abs() <= 5 * sd).all(), (freq, p)
    went = float((c > 1).double().mean())
    if with_draft:
        assert 0.3 < went < 1.0
    else:
        share = float(p[tok[0, 1:].long()].sum())
        assert abs(went - share) <= 5 * (share * (1 - share) / b) ** 0.5
    tf.tf_device_error()


@pytest.mark.parametrize("b,n,v,with_draft", [(2, 16, 129280, True), (40, 9, 20001, False), (1, 1, 129280, False)])
def test_verify_same_bits_every_time_on_streams_and_in_a_graph(b, n, v, with_draft):
    rng = np.random.default_rng(0)
    x, d, g = logits_like(b, n, v, "bf16", 4)
    par = i32([tree("tree", n, rng) for _ in range(b)])
    tok = torch.topk(d.float(), 1, dim=-1).indices[:, :, 0].int().roll(1, 1).contiguous()
    us, ua = (torch.rand((b, n), device="cuda", generator=g) for _ in range(2))
    kw = dict(draft_logits=d, u_accept=ua) if with_draft else {}
    want = tf.tf_verify_draft(x, tok, par, us, temperature=0.9, **kw)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(tf.tf_verify_draft(x, tok, par, us, temperature=0.9, **kw))
    torch.cuda.synchronize()
    ws = tf.tf_verify_draft_workspace(b, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = tf.tf_verify_draft(x, tok, par, us, temperature=0.9, workspace=ws, **kw)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        got.append([t.clone() for t in res])
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))
    tf.tf_device_error()


def test_verify_one_workspace_for_the_largest_and_all_smaller_sizes():
    """A program that makes its workspace once, for its largest batch of
    trees, verifies whatever part of it there is in a step."""
    sizes = [(32, 16), (8, 16), (1, 24), (16, 9), (152, 1), (17, 9), (1, 1), (32, 16), (9, 16)]
    ws = tf.tf_verify_draft_workspace(152, 24)
    rng = np.random.default_rng(2)
    for b, n in sizes:
        x, _, g = logits_like(b, n, 500, "bf16", b + n)
        par = i32([tree("tree", n, rng) for _ in range(b)])
        tok = x.float().argmax(-1).int().roll(1, 1).contiguous()
        us = torch.rand((b, n), device="cuda", generator=g)
        want = tf.tf_verify_draft(x, tok, par, us, workspace=tf.tf_verify_draft_workspace(b, n))
        got = tf.tf_verify_draft(x, tok, par, us, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), (b, n)
    assert not ws.any()   # ready for the next call
    # No smaller size needs more than a larger one.
    need = [[tf.lib().tf_verify_draft_workspace_bytes(b, n) for n in (1, 2, 7, 16, 31, 128)]
            for b in (1, 2, 8, 32, 151, 152, 153, 4000)]
    assert all(x <= y for row in need for x, y in zip(row, row[1:]))
    assert all(x <= y for r0, r1 in zip(need, need[1:]) for x, y in zip(r0, r1))
    tf.tf_device_error()


def test_a_graph_of_a_stream_that_is_not_the_current_one_has_its_own_workspaces():
    """A side stream is captured while another stream is the current one: the
    graph must not hold the workspaces that the binding keeps for the side
    stream, which a larger call replaces."""
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    rng = np.random.default_rng(4)
    c = Case("bf16", [3000, 40], 3, 2, 4, 64, 16, seed=3)
    par = i32([tree("tree", 3, rng)] * 2)
    x, _, g = logits_like(2, 3, 1000, "bf16", 6)
    tok, us = x.float().argmax(-1).int(), torch.rand((2, 3), device="cuda", generator=g)
    big = Case("bf16", [900], 100, 2, 4, 128, 64, seed=4)
    big_par = i32([tree("tree", 100, rng)])

    def calls():
        return [*tf.tf_tree_attention(c.q, c.k, c.v, c.table, c.lengths, par, stream=side),
                *tf.tf_verify_draft(x, tok, par, us, stream=side)]

    torch.cuda.synchronize()
    want = calls()   # the side stream's workspaces are made here
    torch.cuda.synchronize()
    kept = {k: w[0] for k, w in tf.spec._workspaces.items() if k[2] == side.cuda_stream}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        graph.capture_begin(capture_error_mode="relaxed")
        with torch.cuda.stream(other):
            got = calls()
        graph.capture_end()
    assert kept == {k: w[0] for k, w in tf.spec._workspaces.items() if k[2] == side.cuda_stream} and len(kept) == 2
    tf.tf_tree_attention(big.q, big.k, big.v, big.table, big.lengths, big_par, stream=side)
    torch.cuda.synchronize()
    for _ in range(2):
        for t in got:
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    tf.tf_device_error()


# -------------------------------------------------------- refusals, empties
def test_empty_batches_launch_nothing():
    k = torch.zeros((2, 16, 1, 64), dtype=torch.float16, device="cuda")
    t, ln = torch.zeros((0, 1), dtype=torch.int32, device="cuda"), torch.zeros((0,), dtype=torch.int32, device="cuda")
    par = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    o, l = tf.tf_tree_attention(torch.zeros((0, 3, 2, 64), dtype=torch.float16, device="cuda"), k, k, t, ln, par)
    assert o.shape == (0, 3, 2, 64) and l.shape == (0, 3, 2)
    tf.tf_kv_write(torch.zeros((0, 3, 1, 64), dtype=torch.float16, device="cuda"),
                   torch.zeros((0, 3, 1, 64), dtype=torch.float16, device="cuda"), k, k, t, ln)
    got = tf.tf_verify_draft(torch.zeros((0, 3, 10), device="cuda"), par, par, torch.zeros((0, 3), device="cuda"))
    assert got[0].shape == (0,) and got[1].shape == (0, 3)
    assert tf.tf_kv_keep(k, k, t, ln, par, ln).shape == (0,)


def test_refusals_reach_the_caller_before_any_launch():
    c = Case("fp16", [20], 4, 2, 2, 64, 16, seed=1)
    par = i32([-1, 0, 1, 2])
    call = lambda **k: tf.tf_tree_attention(**{**dict(q=c.q, k_cache=c.k, v_cache=c.v, page_table=c.table,  # noqa: E731
                                                      lengths=c.lengths, parents=par), **k})
    for bad in (dict(q=c.q[..., :32]), dict(q=c.q.transpose(2, 3)), dict(v_cache=c.v[:, :8]), dict(parents=par[:3]),
                dict(page_table=c.table[0]), dict(out=torch.empty(3, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=c.q.bfloat16()), dict(lengths=c.lengths.long()), dict(parents=par.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad, status in ((dict(q=c.q[:, :, :3]), tf.TF_ERR_SHAPE), (dict(scale=float("nan")), tf.TF_ERR_SHAPE),
                        (dict(workspace=torch.zeros(0, dtype=torch.uint8, device="cuda")), tf.TF_ERR_NULL),
                        (dict(workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")[16:]), tf.TF_ERR_ALIGN),
                        (dict(lengths=torch.tensor([20], dtype=torch.int32)), tf.TF_ERR_POINTER)):
        with pytest.raises(tf.TFError) as e:
            call(**bad)
        assert e.value.status == status, bad
    with pytest.raises(tf.TFError) as e:
        tf.tf_kv_keep(c.k, c.v, c.table, c.lengths, i32([[0, 1]]), i32([2]), new_lengths=c.lengths)
    assert e.value.status == tf.TF_ERR_POINTER
