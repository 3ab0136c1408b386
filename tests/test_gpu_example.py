"""The example layer runs as written: its outputs lie as near the plain layer as
the rows' roundings leave them, and its balance loss falls.

Bound of the serving steps: a row's FP8 codes are off by at most 2^-4 of a
value and its MXFP4 codes by at most 1/4 (a value in the lowest normal binade,
half a step of 1/2; a block's smaller values less in absolute terms), each with
independent signs, so the layer's output is within their root sum of squares."""
import math
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu


def test_serving_steps():
    import moe_layer
    for name, off in moe_layer.serve(tokens=1000, decode_tokens=17).items():
        print("example", name, off, flush=True)
        assert off <= math.hypot(2.0 ** -4 * math.sqrt(2), 0.25), name


def test_training_steps():
    import moe_layer
    losses = moe_layer.train(tokens=777, steps=12)
    print("example balance loss", losses, flush=True)
    # two of the three sequences hold tokens, and each one's loss is at least
    # about 1 where scores are even; a biased router lies above
    assert all(b < a for a, b in zip(losses[:6], losses[1:6])) and losses[-1] < losses[0]
