"""Slots of calls that keep no states: nothing is addressed, so nothing is past the end."""
import pytest
import torch

import layer_reference as R
import test_gpu_conv as conv
import test_gpu_ssm as ssm
from test_gpu_ssm import gdn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("segment", [0, 64])
def test_scan_without_states(gdn, segment):  # noqa: F811
    a = ssm.draw(1, (3, 130), 40, 16)
    slots = torch.tensor([0, 7, -1], dtype=torch.int32, device="cuda")
    y, s = gdn.gdn_ssm_fwd(**a, slots=slots, want_final_state=False, segment=segment)
    assert s is None and gdn.gdn_get_device_status() == 0
    y0, bound, _, _ = ssm.reference(a, pieces=3)
    assert R.inside(y, y0, bound) <= 1


def test_convolution_without_states(gdn):  # noqa: F811
    x, w, b, _ = conv.draw(2, (3, 50), 64, 4, "bf16")
    slots = torch.tensor([0, 7, -1], dtype=torch.int32, device="cuda")
    y, s = gdn.gdn_conv_fwd(x, w, b, slots=slots, want_final_state=False)
    assert s is None and gdn.gdn_get_device_status() == 0
    y0, bound, _ = R.conv(x, w, b, None, None, None, "silu")
    assert R.inside(y, y0, bound) <= 1
