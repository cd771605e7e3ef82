"""The post-training example: distillation loss falls, the rewarded tokens gain."""
import math

import pytest

pytestmark = pytest.mark.gpu


def test_post_training_example_learns():
    from nvfp4_token_routed_gb300.examples import post_training
    h = post_training.run()
    assert all(math.isfinite(v) for vs in h.values() for v in vs)
    assert h["distill"][-1] < 0.5 * h["distill"][0], h["distill"]
    assert h["reward"][-1] > h["reward"][0] + 0.02, h["reward"]
