"""The training example runs the bridge codec, the clipping and AdamW
together, replayed from a HIP graph, and learns with both kinds of moments."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_example_learns_with_both_states():
    import ddp_adamw
    last = {}
    for state in ("f32", "e4m3"):
        losses = ddp_adamw.train(state, "fp8", 150)
        assert np.isfinite(losses).all()
        last[state] = float(np.mean(losses[-10:]))
        # a teacher's sine has variance about 1/2: learning shows far below the start
        assert last[state] < 0.5 * losses[0], (state, losses[0], last)
    assert last["e4m3"] < 1.5 * last["f32"] + 0.01, last
