"""GPU: the example that runs the cache, the attention and the verification
together with the quantized linears."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROMPT = [3, 141, 59, 26, 53, 3, 141, 59]


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", [0, 1])
def test_drafts_do_not_change_the_text(example, fmt):
    # A place's random number draws its token with and without a tree of
    # drafts, and near temperature 0 a chain keeps just the likeliest tokens.
    for kind, temperature in (("tree", 0.5), ("tree", 1e-3), ("chain", 1e-3)):
        plain, passes = example.generate(example.Decoder(format=fmt), PROMPT, 64, "none",
                                         temperature=temperature)
        assert passes == 64
        text, fewer = example.generate(example.Decoder(format=fmt), PROMPT, 64, kind,
                                       temperature=temperature)
        assert text == plain
        assert fewer <= passes


def test_a_text_that_repeats_itself_takes_fewer_passes(example):
    # near temperature 0 a small decoder soon runs in a circle, and what
    # followed a token before is what follows it again
    text, passes = example.generate(example.Decoder(), PROMPT, 160, "tree", temperature=1e-3)
    assert len(text) == 160
    assert all(0 <= t < 512 for t in text)
    assert passes < 160
