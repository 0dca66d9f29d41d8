"""The hybrid example: decoding step by step through states and paged cache gives
what one pass over the whole sequences gives.

Tolerance: both ways round each layer's operands and outputs to bf16 (2^-8 each,
about eight roundings a layer, at random); over 8 layers the residual stream
differs by about sqrt(64) 2^-8 = 3 % of its rms at worst entries of a few
sigmas, so 0.25 of the rms for the largest of all entries.
"""
import pytest

from gated_delta_rule_57_gb300 import hybrid_example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(prompts=1, tokens=64, steps=70), dict(prompts=5, tokens=31, steps=3, d=128, hq=8),
                                dict(prompts=2, tokens=300, steps=5, hq=6, hkv=2, layers=4)])
def test_steps_equal_one_pass(kw):
    off, status = hybrid_example.run(**kw)
    assert status == 0
    assert off <= 0.25
