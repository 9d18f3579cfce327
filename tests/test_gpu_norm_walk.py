"""Group norm of so many rows that every team walks down several turns of them,
for each team that a group's width selects.  The definition in fp64 on the GPU
with ``layer_reference.norm``'s bound."""
import pytest
import torch

import layer_reference as R
from test_gpu_norm import draw, gdn  # noqa: F401

pytestmark = pytest.mark.gpu
U, EX = R.U, R.EX


def silu_error(v):
    return (v * torch.sigmoid(v)).abs() * (8 * U + EX + 2 * U * v.abs())


def definition(a, groups, rms, act):
    """(y, bound), the formulas of ``layer_reference.norm``."""
    X = a["x"].double()
    rows = X.unflatten(1, (groups, -1))
    k = (rows.shape[-1] / 32 + 8) * U
    mean = 0 if rms else rows.mean(-1, keepdim=True)
    c = rows - mean
    var = (c * c).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(var + 1e-5)
    emean = torch.zeros_like(rows) if rms else k * rows.abs().mean(-1, keepdim=True) + U * rows.abs()
    u = c * r
    er = 0.5 * (2 * k * var + (2 * emean * c.abs()).mean(-1, keepdim=True) + (emean ** 2).mean(-1, keepdim=True)) * r * r + 4 * U
    off = (emean * r + u.abs() * (er + 2 * U)).flatten(1)
    u = u.flatten(1)
    if a["weight"] is not None:
        w = a["weight"].double()
        off = off * w.abs() + U * (u * w).abs()
        u = u * w
    if a["bias"] is not None:
        u = u + a["bias"].double()
        off = off + U * u.abs()
    if act == "silu":
        off = 1.1 * off + silu_error(u)
        u = u * torch.sigmoid(u)
    if a["gate"] is not None:
        z = a["gate"].double()
        g = z * torch.sigmoid(z)
        off = (off + 2 * U * u.abs()) * g.abs() + u.abs() * silu_error(z)
        u = u * g
    if a["x"].dtype == torch.bfloat16:   # half an ulp of the stored value
        half = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"),
                           (torch.frexp(u.abs() + off).exponent - 9).clamp(min=-134))
    else:
        half = U * (u.abs() + off)
    return u, off + half + 1e-37


def check(gdn, a, groups, rms=False, act="none"):  # noqa: F811
    y = gdn.gdn_group_norm(a["x"], groups, a["weight"], a["bias"], a["gate"], rms=rms, act=act)
    assert gdn.gdn_last_launch_count() == (1, 8) and gdn.gdn_get_device_status() == 0
    u, bound = definition(a, groups, rms, act)
    assert float(((y.double() - u).abs() / bound).max()) <= 1
    return y


# one width or more per team: words of 16 bytes, of two elements, single ones
WIDTHS = [8, 64, 128, 256, 512, 1024, 2048, 4096, 8192, 34, 122, 186, 250, 314, 378, 506, 762, 1018, 2042,
          5, 31, 61, 95, 127, 159, 191, 255, 383, 511, 1021, 2051]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_teams_walk_rows(gdn, width, dtype):  # noqa: F811
    """6001 rows of about 4000 channels: 4 turns of the widest teams and up, the last one ragged."""
    groups = max(1, 4000 // width)
    a = draw(width, 6001, groups * width, dtype)
    y = check(gdn, a, groups)
    for name in ("x", "gate"):                       # in place: the next rows are read while these are stored
        b = dict(a, **{name: a[name].clone()})
        assert torch.equal(gdn.gdn_group_norm(b["x"], groups, a["weight"], a["bias"], b["gate"], y=b[name]), y)
    check(gdn, dict(a, weight=None, gate=None), groups, rms=True, act="silu")


@pytest.mark.parametrize("rows", [1, 2, 911, 912, 913, 1824, 4001])
def test_ragged_ends(gdn, rows):  # noqa: F811
    a = draw(rows, rows, 2048, "bf16")
    y = check(gdn, a, 1)
    x = a["x"].clone()
    assert torch.equal(gdn.gdn_group_norm(x, 1, a["weight"], a["bias"], a["gate"], y=x), y)
