"""Malformed packs of linear attention: spans that fall or leave the rows are flagged and
left alone, the others are computed."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from test_gpu_linattn import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("segment", [0, 128])
@pytest.mark.parametrize("cu", [[0, 150, 90, 90], [0, 150, -5, 150], [0, 150, 301, 150], [0, 150, -2 ** 31, 2 ** 31 - 1]])
@pytest.mark.parametrize("before", [0, 70])
def test_spans_that_fall_are_left_alone(dtype, segment, cu, before):
    """The first span of the four offsets is right.  ``before`` empty sequences ahead of it: more than are ranked."""
    x = make((1, 300), 2, 1, 64, 64, dtype, seed=51)
    N = before + 3
    offsets = torch.tensor([0] * before + cu, dtype=torch.int32, device="cuda")
    S0 = torch.randn(N, 2, 64, 64, device="cuda")
    out, o = torch.full_like(S0, 7.0), torch.full_like(x["v"].contiguous(), 5.0)
    gdn.gdn_linattn_fwd(**x, state_in=S0, state_out=out, o=o, cu_seqlens=offsets, segment=segment)
    assert gdn.gdn_get_device_status() == 1                              # GDN_DEV_BAD_SEQLENS
    want, final = gdn.gdn_linattn_fwd(**{n: t[:, :150].contiguous() for n, t in x.items()}, state_in=S0[before:before + 1],
                                      segment=segment)
    assert torch.equal(o[:, :150], want) and bool((o[:, 150:] == 5).all())
    assert torch.equal(out[before], final[0]) and torch.equal(out[:before], S0[:before])
    for n in range(1, 3):
        lo, hi = cu[n], cu[n + 1]
        assert torch.equal(out[before + n], S0[before + n]) if 0 <= lo == hi else bool((out[before + n] == 7).all())
