"""bf16 prompts on the tensor cores: outputs are off by their own rounding and by
little else, as fp32 arithmetic rounded once would be."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from linattn_exact import agrees, walk
from test_gpu_linattn import make, on_tensor_cores

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,dk,dv", [(2, 2, 128, 128), (2, 1, 96, 192), (4, 2, 64, 64), (3, 3, 8, 8), (2, 1, 40, 72)])
@pytest.mark.parametrize("T", [1, 100, 129, 517])
@pytest.mark.parametrize("segment", [0, 128])
def test_outputs_are_off_by_their_rounding(H, G, dk, dv, T, segment):
    """Every entry within half a step of bf16 and 2^-16 of the sum of magnitudes behind it."""
    x = make((1, T), H, G, dk, dv, "bf16", seed=T + dk)
    assert on_tensor_cores(x)
    S0 = torch.randn(1, H, dv, dk, device="cuda")
    o, S = gdn.gdn_linattn_fwd(**x, scale=dk ** -0.5, state_in=S0, segment=segment)
    ro, bo, rS, bS = walk(**x, scale=dk ** -0.5, state_in=S0, parts=True, pieces=1 + (segment > 0))
    assert agrees(o, ro, bo) <= 1 and agrees(S[0], rS[0], bS[0]) <= 1
    assert gdn.gdn_get_device_status() == 0


def test_outputs_round_as_one_rounding_would():
    """The 2-norm of the error against that of rounding the exact outputs once: entries near
    a border between two roundings go the other way, few of them, and nothing else."""
    x = make((2, 600), 4, 4, 128, 128, "bf16", seed=3)
    o, _ = gdn.gdn_linattn_fwd(**x, scale=128 ** -0.5)
    ro = torch.from_numpy(walk(**x, scale=128 ** -0.5, parts=True)[0])
    off, own = (float((t.double().cpu() - ro).norm() / ro.norm()) for t in (o, ro.bfloat16()))
    # 2^-16 of a sum's magnitudes at random, against 2^-8 / sqrt(12) or so of the outputs: 1 % together, if the
    # magnitudes' root sum of squares is up to ten times the output
    assert off <= 1.01 * own, (off, own)
