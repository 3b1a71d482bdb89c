"""GPU: the example that runs a recurrent layer and an attention layer through segments and decode
steps gives what one call of each over the whole prompt gives.

Bars (2-norm of the difference over that of the result): the recurrence's own for its outputs and
states; an attention output carries two independent roundings to bf16, of the weights and of
itself, each of at most 2^-8 / sqrt 3 in the root mean square, and two such outputs are compared:
2 x 2.3e-3, and twice that as margin."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,segment,steps,store", [(700, 256, 3, "fp8"), (300, 128, 5, "bf16")])
def test_segments_and_steps_match_the_whole_prompt(tokens, segment, steps, store):
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off = m.run(tokens, segment, steps, store)
    assert off["recurrent"] <= 1e-3 and off["state"] <= 1e-3, off
    assert off["attention"] <= 9e-3, off
