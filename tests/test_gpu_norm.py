"""GPU parity of gdn_group_norm with the definition in fp64 (bounds:
``layer_reference``)."""
import pytest
import torch

import layer_reference as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_09_gb300 as g
    return g


def draw(seed, rows, C, dtype, gate=True, affine=True, extra=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    cut = lambda m: m.to(DT[dtype])[:, extra:]  # noqa: E731
    return dict(x=cut(r(rows, C + extra) + r(rows, 1)), gate=cut(r(rows, C + extra)) if gate else None,
                weight=1 + 0.2 * r(C) if affine else None, bias=0.2 * r(C) if affine else None)


def check(gdn, a, groups, rms=False, act="none", eps=1e-5, **kw):
    y = gdn.gdn_group_norm(a["x"], groups, weight=a["weight"], bias=a["bias"], gate=a["gate"], eps=eps, rms=rms,
                           act=act, **kw)
    assert gdn.gdn_last_launch_count() == (1, 8) and gdn.gdn_get_device_status() == 0
    ref, bound = R.norm(a["x"], groups, a["weight"], a["bias"], a["gate"], eps, rms, act)
    assert R.inside(y, ref, bound) <= 1
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 2, 3, 4, 7, 8, 9, 16, 24, 31, 32, 33, 61, 64, 96, 128, 192, 200, 256, 257, 264, 512,
                                   513, 1000, 1024, 2048, 2056, 2500, 4096, 8192, 8200, 10007, 20000])
def test_group_widths(gdn, width, dtype):
    groups = 3 if width < 5000 else 1
    check(gdn, draw(width, 5, groups * width, dtype), groups)
    check(gdn, draw(width, 5, groups * width, dtype, gate=False), groups, rms=True, act="silu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 3, 31, 255, 1000])
@pytest.mark.parametrize("groups", [1, 2, 5, 16])
def test_rows_and_groups(gdn, rows, groups, dtype):
    check(gdn, draw(rows + groups, rows, groups * 64, dtype), groups)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_variants(gdn, act, rms, gate, affine, dtype):
    check(gdn, draw(5, 7, 512, dtype, gate, affine), 4, rms=rms, act=act)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups,extra", [(512, 4, 64), (512, 4, 3), (63, 7, 5), (1925, 7, 0)])
def test_strides(gdn, C, groups, extra, dtype):
    check(gdn, draw(C, 9, C, dtype, extra=extra), groups)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", [(512, 4), (63, 7), (9000, 1)])
def test_in_place(gdn, C, groups, dtype):
    a = draw(C, 9, C, dtype)
    want = check(gdn, a, groups)
    x = a["x"].clone()
    assert torch.equal(gdn.gdn_group_norm(x, groups, a["weight"], a["bias"], a["gate"], y=x), want)
    g = a["gate"].clone()
    assert torch.equal(gdn.gdn_group_norm(a["x"], groups, a["weight"], a["bias"], g, y=g), want)


def test_large_mean(gdn):
    """A mean a thousand times the spread: the variance is taken about it."""
    a = draw(6, 20, 512, "f32", gate=False)
    a["x"] = a["x"] + 1000
    check(gdn, a, 4)


def test_constant_and_zero_groups(gdn):
    a = draw(7, 4, 256, "f32", gate=False, affine=False)
    a["x"][:, :64] = 3.0
    a["x"][:, 64:128] = 0.0
    y = check(gdn, a, 4)
    assert (y[:, :128] == 0).all()
    assert (gdn.gdn_group_norm(a["x"], 4, rms=True)[:, 64:128] == 0).all()


def test_groups_do_not_see_one_another(gdn):
    a = draw(8, 6, 256, "f32")
    clean = check(gdn, a, 4)
    a["x"][2, 70] = float("nan")
    a["x"][3, 10] = float("inf")
    y = gdn.gdn_group_norm(a["x"], 4, a["weight"], a["bias"], a["gate"])
    assert torch.isnan(y[2, 64:128]).all() and torch.isnan(y[3, :64]).any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[2, 64:128] = keep[3, :64] = False
    assert torch.equal(y[keep], clean[keep])


def test_output_slice_and_leading_dimensions(gdn):
    a = draw(9, 12, 96, "bf16")
    wide = torch.full((12, 110), float("nan"), dtype=torch.bfloat16, device="cuda")
    check(gdn, a, 3, y=wide[:, 7:103])
    assert torch.isnan(wide[:, :7]).all() and torch.isnan(wide[:, 103:]).all()
    y = gdn.gdn_group_norm(a["x"].reshape(2, 3, 2, 96), 3, a["weight"], a["bias"], a["gate"].reshape(2, 3, 2, 96))
    assert y.shape == (2, 3, 2, 96) and torch.equal(y.reshape(12, 96), wide[:, 7:103])


def test_offsets_past_32_bits(gdn):
    ld = (1 << 31) // 6 + 64
    a = draw(10, 7, 128, "bf16", gate=False)
    big = torch.empty(7 * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((7, 128), (ld, 1))
    x.copy_(a["x"])
    check(gdn, dict(a, x=x), 2, y=big.as_strided((7, 128), (ld, 1), 128))


def test_another_stream(gdn):
    a = draw(11, 64, 1024, "bf16")
    want = check(gdn, a, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = gdn.gdn_group_norm(a["x"], 8, a["weight"], a["bias"], a["gate"], stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_empty(gdn):
    assert gdn.gdn_group_norm(torch.empty(0, 64, device="cuda"), 4).shape == (0, 64)
