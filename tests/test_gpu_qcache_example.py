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
