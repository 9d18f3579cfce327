"""So many channels that their blocks go on in the grid's third dimension."""
import numpy as np
import pytest
import torch

import layer_reference as R
import test_gpu_conv as conv
import test_gpu_ssm as ssm
from test_gpu_ssm import gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def test_scan_step(gdn):  # noqa: F811
    """65 540 blocks of four channels."""
    a = ssm.draw(1, (1, 1), 4 * 65540, 65, pool=1)
    y0, bound, new, eb = ssm.reference(a)
    y, s = gdn.gdn_ssm_step(**{k: (v[:, 0] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()})
    assert gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1 and R.inside(s, np.stack(new), np.stack(eb)) <= 1


def test_convolution(gdn):  # noqa: F811
    """65 537 blocks of 256 channels, the last with one: prompts and a step."""
    C = 256 * 65536 + 1
    x, w, _, s = conv.draw(2, (1, 3), C, 2, "bf16", bias=False, pool=1)
    taps = torch.cat([s, x], 1).float()
    want = taps[:, :-1] * w[:, 0] + taps[:, 1:] * w[:, 1]
    y, out = gdn.gdn_conv_fwd(x, w, state_in=s, act="none")
    assert (y.float() - want).abs().max() <= 2.0 ** -8 * want.abs().max()
    assert torch.equal(out[:, 0], x[:, 2])
    y, out = gdn.gdn_conv_step(x[:, 0], w, state_in=s, act="none")
    assert (y.float() - want[:, 0]).abs().max() <= 2.0 ** -8 * want.abs().max()
    assert torch.equal(out[:, 0], x[:, 0]) and gdn.gdn_get_device_status() == 0
