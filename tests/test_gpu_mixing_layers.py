"""The example's two layers: a packed prompt and then single tokens give what
one longer prompt gives.  Both sides store y in bf16 after a chain of bf16
products (the projection of the convolved inputs among them), whose roundings
can fall either way where fp32 sums differ in order: a few half ulps of 2^-9
each, 1e-2 together in the 2-norm."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,steps", [(200, 8), (70, 3), (3, 5)])
def test_steps_continue_the_prompt(tokens, steps):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import gated_delta_rule_09_gb300 as gdn
    import mixing_layers
    for name, (parts, whole) in mixing_layers.run(tokens, steps).items():
        for a, b in zip(parts, whole):
            assert a.shape == b.shape and torch.isfinite(a.float()).all(), name
            assert (a - b).float().norm() <= 1e-2 * b.float().norm(), name
    assert gdn.gdn_get_device_status() == 0
