"""The scan's workspace in the Python binding (CPU only)."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from test_layer_cpu import host_only, ssm_args  # noqa: F401


@pytest.mark.parametrize("workspace", [
    torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0],              # a column: its neighbours would be written
    torch.zeros(1, dtype=torch.uint8).expand(1 << 16),             # past its storage
    torch.zeros(256, 512, dtype=torch.uint8)[:, :256]])
def test_strided_workspace_is_refused(host_only, workspace):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.gdn_ssm_fwd(**ssm_args(), segment=64, workspace=workspace)


def test_other_types_are_refused(host_only):  # noqa: F811
    with pytest.raises(TypeError):
        gdn.gdn_ssm_fwd(**ssm_args(), segment=64, workspace=torch.zeros(1 << 16))


def test_plain_workspace_reaches_the_library(host_only):  # noqa: F811
    with pytest.raises(RuntimeError, match="reached the library"):
        gdn.gdn_ssm_fwd(**ssm_args(), segment=64, workspace=torch.zeros(1 << 16, dtype=torch.uint8))
