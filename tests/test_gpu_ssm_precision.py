"""What bf16 scans may be off beside the rounding of y: the sum over states is
taken in fp32, for prompts as for single tokens.

The bounds are ``layer_reference``'s for fp32 arithmetic (the same inputs seen
as fp32, which is exact), then one rounding to bf16."""
import numpy as np
import pytest
import torch

import layer_reference as R
from test_gpu_ssm import draw, gdn  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = ("x", "delta", "B", "C", "z")


def fp32_arithmetic(a, pieces=1):
    """(y, bound) of fp32 arithmetic with y rounded once to bf16, new states and theirs."""
    f = {k: (v.float() if k in ROWS and v is not None else v) for k, v in a.items()}
    y, bound, new, eb = R.ssm(f["x"], f["delta"], f["A"], f["B"], f["C"], f["D"], f["z"], f["delta_bias"],
                              f["delta_softplus"], f["state_in"], None, None, pieces)
    return y, R.stored(y, bound, torch.bfloat16), new, eb


@pytest.mark.parametrize("segment", [0, 64])
@pytest.mark.parametrize("S,ch", [(1, 64), (13, 40), (16, 64), (16, 43), (24, 64), (32, 72), (64, 64), (100, 40), (128, 64)])
def test_prompt_sums_states_in_fp32(gdn, S, ch, segment):  # noqa: F811
    """C of either sign: y is often far smaller than the terms it is the sum of."""
    a = draw(S + ch, (2, 150), ch, S, pool=2)
    pieces = 3 if segment else 1
    y0, bound, new, eb = fp32_arithmetic(a, pieces)
    y, s = gdn.gdn_ssm_fwd(**a, segment=segment)
    assert gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0, bound) <= 1
    assert R.inside(s, np.stack(new), np.stack(eb)) <= 1


@pytest.mark.parametrize("S", [4, 16, 100, 128])
def test_step_sums_states_in_fp32(gdn, S):  # noqa: F811
    a = draw(S, (30, 1), 64, S, pool=30)
    y0, bound, _, _ = fp32_arithmetic(a)
    y, _ = gdn.gdn_ssm_step(**{k: (v[:, 0] if k in ROWS else v) for k, v in a.items()})
    assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1


@pytest.mark.parametrize("S", [16, 32, 128])
def test_prompt_outputs_are_not_shifted(gdn, S):  # noqa: F811
    """The mean of (y - exact) / exact over 2^17 outputs that are sums of positive
    terms.  Rounding y to nearest is off by at most 2^-9 of it and by at most
    2^-9 / sqrt(3) in RMS, in either direction: the mean of n is within six
    standard errors.  Beside that only fp32's own errors, below 2^-18 here."""
    T, ch = 512, 256
    a = draw(S, (1, T), ch, S, z=False)
    a.update({k: a[k].abs() for k in ("x", "B", "C")}, D=None)
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
    d = torch.nn.functional.softplus(f["delta"] + f["delta_bias"], threshold=1e9)[0]
    h, rows = torch.zeros(ch, S, dtype=torch.float64, device="cuda"), []
    for t in range(T):
        h = torch.exp(d[t][:, None] * f["A"]) * h + (d[t] * f["x"][0, t])[:, None] * f["B"][0, t]
        rows.append(h @ f["C"][0, t, 0])
    exact = torch.stack(rows)
    y, _ = gdn.gdn_ssm_fwd(**a, segment=T)
    off = (y[0].double() - exact) / exact
    assert torch.isfinite(off).all()
    assert abs(float(off.mean())) <= 6 * 2.0 ** -9 / np.sqrt(3 * off.numel()) + 2.0 ** -18
