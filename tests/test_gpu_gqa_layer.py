"""The example layer: a prompt, steps over the 4-bit cache, an eviction by their weights and more steps, against the layer in
64 bits from the same cached rows.

Tolerance of the outputs (largest difference over largest value): the prompt rounds q, k, v and the probabilities to f16 (2^-11
each of the value, the scores move by as much of themselves); the steps round q to f16, the probabilities and their products with
the scales to bf16 (2^-8 each).  Errors of the independent terms of the o projection average, so 2^-8 bounds the prompt and
3 x 2^-8 the steps amply."""
import os
import sys

import pytest

from gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,heads,kv,prompt,steps,keep", [(512, 8, 2, 70, 6, 40), (256, 14, 2, 300, 4, 100), (256, 4, 4, 1, 4, 2), (256, 16, 1, 130, 4, 200)])
def test_example_layer(hidden, heads, kv, prompt, steps, keep):
    cuda_or_skip()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import gqa_layer
    e_prompt, e_step, right, *_ = gqa_layer.run(hidden, heads, kv, prompt, steps, keep, seed=heads)
    assert e_prompt <= 2.0 ** -8 and e_step <= 3 * 2.0 ** -8
    assert right
