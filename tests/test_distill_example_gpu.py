"""The example runs the calls together, and its head learns what each part asks for."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_head.py")


def test_the_head_learns(cuda_lib):
    run = runpy.run_path(PATH)["run"]
    losses, scores = run(tokens=256, vocab=5000, hidden=256, top_k=16, steps=8)
    assert losses[-1] < losses[0] and scores[-1] > scores[0]
    assert all(x == x for x in losses + scores)
