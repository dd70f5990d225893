"""The recurrent layers of examples/hybrid_layers.py with a convolution before and a gated norm behind the recurrence:
decoding token by token gives the hidden states of prefilling everything at once."""
import pytest

from tests.test_gpu_hybrid_example import _example

pytestmark = pytest.mark.gpu


# Both ways round every layer's output to bf16 (2^-8 of a value, eight layers of residual sums), and each layer rounds its
# convolution's and its norm's results too: two further half steps a layer.
@pytest.mark.parametrize("kind,steps", [("conv", 5), ("ssm", 5)])
@pytest.mark.parametrize("prompts", [(130, 7, 201), (3, 1, 1, 2)])
def test_decode_continues_prefill(kind, steps, prompts):
    diff = _example().run(prompts=prompts, steps=steps, width=512, kind=kind, verbose=False)
    assert 0 <= diff <= 3 * 8 * 2.0 ** -8
