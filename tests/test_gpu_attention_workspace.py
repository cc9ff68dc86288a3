"""One workspace for the attention over a 16-bit cache and over a quantised
one, in turn: a model may hold some of its layers in each."""

import numpy as np
import pytest

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


def calls():
    """(call over 16 bits, call over 4 or 8), each with items cut between blocks."""
    g = torch.Generator(device="cuda").manual_seed(1)
    out = []
    for lens, n, group, bits in (([4000], 1, 2, 4), ([900] * 300, 1, 1, 4), ([700] * 40, 4, 2, 8), ([2500, 9], 20, 3, 4)):
        c = Case(bits, "bf16", lens, n, 1, group, 128, 32, seed=n)
        par = i32(tree("chain", n, None))
        k, v = (torch.randn(c.k.shape[:3] + (128,), device="cuda", generator=g).bfloat16() for _ in range(2))
        out.append((lambda ws, c=c, par=par, k=k, v=v: tf.tf_tree_attention(c.q, k, v, c.table, c.lengths, par, workspace=ws),
                    lambda ws, c=c, par=par: c.attend(par, workspace=ws)))
    return out


def test_the_two_attentions_share_a_workspace():
    make = lambda: torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")  # noqa: E731
    pairs = calls()
    want = [[call(make()) for call in pair] for pair in pairs]
    ws = make()
    for order in (np.arange(len(pairs)), np.arange(len(pairs))[::-1]):
        for i in order:
            for j in range(len(pairs)):
                pairs[j][0](ws)
                got = pairs[i][1](ws)
                assert torch.equal(got[0], want[i][1][0]) and torch.equal(got[1], want[i][1][1]), (i, j)
                got = pairs[j][0](ws)
                assert torch.equal(got[0], want[j][0][0]) and torch.equal(got[1], want[j][0][1]), (i, j)
    tf.tf_device_error()
