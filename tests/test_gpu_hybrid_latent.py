"""The hybrid example with rotated and with latent attention layers: decoding step by step
through states and caches gives what one pass over the whole sequences gives.

Tolerance: as for the plain layers, both ways round each layer's operands and outputs to
bf16 (2^-8 each, at random). A latent layer's two ways (expanded heads; queries and outputs
multiplied by the expansion) round two operands more, about ten roundings a layer: over 8 layers
sqrt(80) 2^-8 = 3.5 % of the rms, and 0.25 of it for the largest of all entries.
"""
import pytest

from gated_delta_rule_57_gb300 import hybrid_example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("attention", ["rope", "latent"])
@pytest.mark.parametrize("kw", [dict(), dict(prompts=1, tokens=64, steps=70), dict(prompts=5, tokens=31, steps=3, d=128, hq=8),
                                dict(prompts=2, tokens=300, steps=5, hq=6, hkv=2, layers=4)])
def test_steps_equal_one_pass(attention, kw):
    off, status = hybrid_example.run(attention=attention, **kw)
    assert status == 0
    assert off <= 0.25
