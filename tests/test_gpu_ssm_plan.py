"""Which scans the library cuts into pieces."""
import pytest
import torch

import layer_reference as R
from test_gpu_ssm import draw, gdn, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,cut", [(1, True), (64, False)])
def test_blocks_of_groups_are_counted(gdn, groups, cut):  # noqa: F811
    """Four prompts of 4096 tokens x 512 channels: 32 blocks in one group, which
    leaves SMs without one unless it is cut; 256 blocks in 64 groups."""
    a = draw(groups, (4, 4096), 512, 16, groups, pool=4)
    y, s = gdn.gdn_ssm_fwd(**a)
    assert gdn.gdn_last_launch_count() == (2 if cut else 1, 7)
    small = {k: (v[:1, :300] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    y0, bound, _, _ = reference(dict(small, state_in=a["state_in"][:1]), pieces=2)
    assert R.inside(y[:1, :300], y0, bound) <= 1


@pytest.mark.parametrize("ch,groups", [(70, 7), (512, 64), (203, 7), (4096, 2), (60, 60)])
@pytest.mark.parametrize("T", [600, 5000])
def test_workspace_is_enough_for_any_groups(gdn, ch, groups, T):  # noqa: F811
    """The size knows nothing of groups; the call takes it."""
    a = draw(ch, (2, T), ch, 16, groups)
    need = gdn.gdn_ssm_fwd_workspace_size(2, T, ch, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y, _ = gdn.gdn_ssm_fwd(**a, workspace=ws)
    small = {k: (v[:1, :100] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    y0, bound, _, _ = reference(small, pieces=2)
    assert R.inside(y[:1, :100], y0, bound) <= 1 and gdn.gdn_get_device_status() == 0
