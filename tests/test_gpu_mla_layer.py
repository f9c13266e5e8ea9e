"""The example layer: a prompt in the expanded form and steps in the absorbed form against the layer in 64 bits.

Tolerance of the outputs (largest difference over largest value): the expanded form rounds q, k and v to bf16
(2^-8 each of the value; scores of a few units move by about 2^-8 of themselves and the probabilities alike) and the
probabilities to bf16; errors of 128 x 16 independent terms average in the o projection, so 3 x 2^-8 bounds
them amply.  The absorbed form keeps the cache's values and rounds q and the probabilities alone: the same bound."""
import os
import sys

import pytest

from gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("hidden,heads,prompt,steps", [(512, 4, 70, 5), (256, 16, 300, 3), (256, 40, 1, 2)])
def test_example_layer(e4m3, hidden, heads, prompt, steps):
    cuda_or_skip()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mla_layer
    e_prompt, e_step, *_ = mla_layer.run(hidden, heads, prompt, steps, e4m3, seed=heads)
    assert e_prompt <= 3 * 2.0 ** -8 and e_step <= 3 * 2.0 ** -8
