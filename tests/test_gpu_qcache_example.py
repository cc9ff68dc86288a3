"""The operators of the quantised cache together as a user runs them: the
decoding example with head norms, positions and a cache in 4 or 8 bits."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bits", [4, 8])
def test_decoding_with_a_quantised_cache(bits):
    """Runs, in fewer steps with trees than without; the first token comes from
    one pass over the same inputs and has to be the same."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    plain, plain_steps, tokens, steps = example.run(count=24, batch=3, cache_bits=bits)
    assert plain_steps == 24 and steps < 24
    assert plain.shape == tokens.shape == (3, 24)
    assert ((tokens >= 0) & (tokens < example.VOCAB)).all()
    assert torch.equal(plain[:, 0], tokens[:, 0])
    assert example.depths(9) == [0, 1, 2, 3, 4, 1, 2, 3, 4] and example.depths(1) == [0]


@pytest.mark.parametrize("bits", [4, 8])
def test_trees_leave_in_the_cache_what_single_tokens_leave(bits):
    """The tokens of a decoding with trees, fed one by one into another model:
    the rows of the first layer, which no attention comes before, are the same
    bits, wherever in a tree they were written and kept from; those of the
    second differ by what two roundings of nearly the same numbers may.

    Nearly: with the same rows and queries in the first layer, two attentions
    differ by 2^-9 of the mean size of values (weights and result are rounded
    to 11 bits each, twice), which is 4 times the result's at most for 12 slots
    whose values cancel; two projections, a sum and their roundings to fp16
    leave it below 2^-5 of a row's norm with a factor of 4 to spare. Half a step
    for each of two roundings, and 2^-8 of it for their factors, come on top."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    count, batch = 12, 3
    first = torch.arange(1, batch + 1, device="cuda")
    make = lambda: ex.Model(batch, count + 2 * len(ex.TREE), cache_bits=bits)  # noqa: E731
    none = lambda done: torch.zeros((batch, 0), dtype=torch.int32, device="cuda")  # noqa: E731
    truth, _ = ex.decode(make(), first, count, [-1], none)
    padded = torch.cat([truth, torch.zeros((batch, 8), dtype=truth.dtype, device="cuda")], dim=1)
    calls = []

    def draft(done):
        """By turns a right child beside a wrong one, and one below two right ones of the chain."""
        ahead = padded.gather(1, done.clamp(max=count)[:, None] + torch.arange(4, device="cuda"))
        wrong = (ahead + 1) % ex.VOCAB
        calls.append(None)
        right = [5] if len(calls) % 2 else [1, 2, 7]
        nodes = torch.cat([wrong, wrong], dim=1)
        for j in right:
            nodes[:, j - 1] = ahead[:, (j - 1) % 4]
        return nodes

    trees, moved = make(), 0
    keep = trees.keep

    def watched(lengths, path, counts):
        nonlocal moved
        k = torch.arange(path.shape[1], device="cuda")
        moved += int(((path != k) & (k < counts[:, None])).sum())
        return keep(lengths, path, counts)

    trees.keep = watched
    tokens, steps = ex.decode(trees, first, count, ex.TREE, draft)
    assert moved >= batch and steps < count     # (the first token is right, so each first child is kept from node 5)
    singles, lengths = make(), torch.zeros((batch,), dtype=torch.int32, device="cuda")
    root = torch.full((batch, 1), -1, dtype=torch.int32, device="cuda")
    fed = torch.cat([first[:, None].to(torch.int32), tokens[:, : count - 1]], dim=1)
    for t in range(count):
        singles.logits(fed[:, t : t + 1].contiguous(), root, lengths)
        lengths = lengths + 1
    most = 2 ** (bits - 1) - 1
    for layer in range(ex.LAYERS):
        rows = [ex.tf.tf_kvq_read(m.k[layer], m.v[layer], m.scales[layer], m.table, lengths, slots=count,
                                  head_dim=ex.DIM, dtype=torch.bfloat16 if layer else torch.float16) for m in (trees, singles)]
        for x, y in zip(*rows):
            if layer == 0:
                assert torch.equal(x, y)
                continue
            x, y = x.double(), y.double()
            step = torch.maximum(x.abs().amax(-1), y.abs().amax(-1)) / most
            # (and the reading's rounding to bf16, 2^-8 of each)
            tol = 2.0 ** -5 * y.norm(dim=-1) + ex.DIM ** 0.5 * step * (1 + 2.0 ** -8 * most) + 2 * 2.0 ** -8 * y.norm(dim=-1)
            assert ((x - y).norm(dim=-1) <= tol).all(), ((x - y).norm(dim=-1) / tol).max()
    ex.tf.tf_device_error()
