"""Tree attention where scores are large, up to what tf_spec.h says they may be:
the key whose score is far above the others is found."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tf.lib()
    yield
    tf.tf_device_error()


@pytest.mark.parametrize("d,n,group", [(64, 24, 1), (128, 9, 5), (128, 3, 2), (64, 40, 3), (256, 9, 2)])
@pytest.mark.parametrize("dtype,power", [("bf16", 10), ("bf16", 24), ("bf16", 29), ("fp16", 10), ("fp16", 25)])
@pytest.mark.parametrize("top", [3, 321])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_of_any_size_find_the_largest(d, n, group, dtype, power, top, sign):
    """Scores of about +-2^power, one an eighth above the others, whose weights are below 2^-100 in all."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(power)
    kh, page, ctx = 2, 16, 500
    per = -(-(ctx + n) // page)
    s = np.arange(per * page)
    scores = 0.5 + 0.25 * np.cos(s) ** 2 if sign > 0 else -(1.0 + 0.25 * np.cos(s) ** 2)
    scores[top] = 1.0 if sign > 0 else -0.875
    half = 2.0 ** (power // 2)                       # q and k share the size
    k = torch.empty((per, page, kh, d), dtype=dt, device="cuda")
    k[...] = (torch.tensor(scores, device="cuda") * half / d).to(dt).view(per, page, 1, 1)
    v = torch.randn(k.shape, device="cuda", generator=g).to(dt)
    q = torch.full((1, n, kh * group, d), 2.0 ** (power - power // 2), dtype=dt, device="cuda")
    table = torch.arange(per, dtype=torch.int32, device="cuda")[None]
    out, lse = tf.tf_tree_attention(q, k, v, table, torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                                    torch.arange(n, dtype=torch.int32, device="cuda") - 1, scale=1.0)
    tf.tf_device_error()
    want = v.view(-1, kh, d)[top].repeat_interleave(group, 0)
    # the weight and the result are rounded to the dtype, by half a step each
    assert ((out[0].double() - want.double()).abs() <= torch.finfo(dt).eps * (1 + 2.0 ** -6) * want.double().abs()).all()
    most = k.view(-1, kh, d)[top, :, 0].double() * d * 2.0 ** (power - power // 2)
    want_l = most.repeat_interleave(group)
    # d products summed, one factor and the logarithm's, in fp32
    assert ((lse[0].double() - want_l).abs() <= (d + 4) * 2.0 ** -24 * want_l.abs()).all()
