"""The example that runs the attention operators with the experts' products."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_prompts_then_tokens_give_the_whole_sequences_outputs():
    """Tokens served one by one from the cache leave the layers as they do within
    a prompt: to BF16 roundings (each layer's operators round a few times at
    2^-8) with a BF16 cache; with an E4M3 cache (2^-4 a key and value) to what its
    codes keep."""
    spec = importlib.util.spec_from_file_location("moe_decoder", os.path.join(ROOT, "examples", "moe_decoder.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    off = ex.main()
    assert off[False] < 2.0 ** -6
    assert off[True] < 2.0 ** -3
