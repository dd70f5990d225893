"""The hybrid stack of examples/hybrid_layers.py: decoding token by token gives the hidden states of
prefilling everything at once."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


# Both ways round every layer's output to bf16 (2^-8 of a value, eight layers of residual sums), and a 4-bit
# key or value may round the other way where its bf16 source did: one step is up to a third of a value, in one
# of some hundred tokens.
@pytest.mark.parametrize("cache,window,sinks,tol", [("bf16", 0, 0, 8 * 2.0 ** -8), ("bf16", 100, 4, 8 * 2.0 ** -8), ("fp4", 0, 0, 16 * 2.0 ** -8)])
def test_decode_continues_prefill(cache, window, sinks, tol):
    diff = _example().run(prompts=(130, 7, 201), steps=5, width=512, cache=cache, window=window, sinks=sinks, verbose=False)
    assert 0 <= diff <= tol
