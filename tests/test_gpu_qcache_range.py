"""Attention over a quantised cache where factors and queries differ by many
powers of two: what a row does not see has no influence whatever its size,
what it sees weighs what the definition says, and finite inputs give finite
results."""

import numpy as np
import pytest

import spec_oracle as so

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402
from test_gpu_qcache import Case, i32, tree  # noqa: E402


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
