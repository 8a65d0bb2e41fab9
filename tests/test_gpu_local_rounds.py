"""The operators together, as a user runs them: examples/local_rounds.py learns."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_rounds_lower_the_held_out_loss():
    import local_rounds
    lines = []
    losses = local_rounds.run(rounds=6, peers=3, local_steps=8, report=lines.append)
    assert len(lines) == 6 and abs(losses[0] - 7.6) < 0.1     # log 2000 at the start
    assert all(b < a for a, b in zip(losses, losses[1:]))
    again = local_rounds.run(rounds=2, peers=3, local_steps=8, report=lambda s: None)
    assert abs(again[2] - losses[2]) < 1e-3
