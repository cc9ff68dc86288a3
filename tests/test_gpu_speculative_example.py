"""The operators together as a user runs them: greedy decoding with drafted
trees gives the tokens of one-token decoding, in fewer steps."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_speculative_decoding_gives_the_tokens_of_plain_decoding():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    plain, plain_steps, spec_tokens, steps = example.run(count=40, batch=3)
    assert plain_steps == 40 and steps < 25
    assert torch.equal(plain, spec_tokens)
    assert len(set(plain.flatten().tolist())) > 10        # not one token for ever
