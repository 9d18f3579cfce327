"""Norms around a block against their definition in fp64."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from layer_reference import inside
from linattn_reference import block_norm

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(rows, C, dtype, stream, seed=0, gate=True, scale=True, bias=True, affine=True, post=True, pre=True, extra=0):
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *s, dt=torch.float32: torch.randn(*s, generator=g, device="cuda", dtype=dt)  # noqa: E731
    rowsof = lambda dt: normal(rows, C + extra, dt=dt)[:, extra:]  # noqa: E731
    return dict(y=rowsof(DT[dtype]) + normal(rows, 1, dt=DT[dtype]), residual=rowsof(DT[stream]) * 3,
                gate=rowsof(DT[dtype]) if gate else None, scale=normal(C) if scale else None,
                post_weight=1 + 0.1 * normal(C) if affine and post else None,
                post_bias=0.1 * normal(C) if affine and bias and post else None,
                pre_weight=1 + 0.1 * normal(C) if affine and pre else None,
                pre_bias=0.1 * normal(C) if affine and bias and pre else None)


def check(x, gate_act="sigmoid", residual_scale=0.7, eps=1e-5, rms=True, post=True, pre=True, **outs):
    want = block_norm(**x, gate_act=gate_act, residual_scale=residual_scale, eps=eps, rms=rms, post=post, pre=pre)
    r, h = gdn.gdn_block_norm(**x, gate_act=gate_act, residual_scale=residual_scale, eps=eps, rms=rms, post=post, pre=pre,
                              **outs)
    assert inside(r, *want[:2]) <= 1
    if pre:
        assert inside(h, *want[2:]) <= 1
    else:
        assert h is None
    return r, h


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
WIDTHS = [1, 2, 7, 64, 96, 130, 255, 256, 512, 1000, 1025, 1925, 2048, 4096, 4100, 8192, 8200, 12288]


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_every_width(dtype, stream, C):
    check(make(37, C, dtype, stream, seed=C), rms=C % 2 == 0)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate_act", [None, "none", "sigmoid", "silu"])
def test_every_choice(dtype, stream, rms, post, pre, gate_act):
    x = make(21, 320, dtype, stream, gate=gate_act is not None, post=post, pre=pre, scale=rms, bias=not rms)
    check(x, gate_act or "sigmoid", rms=rms, post=post, pre=pre)


@pytest.mark.parametrize("rows", [1, 2, 3, 1000, 5001])
@pytest.mark.parametrize("C", [64, 1024])
def test_row_counts(rows, C):
    check(make(rows, C, "bf16", "bf16", seed=rows))


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("extra", [1, 2, 8])
def test_slices_of_wider_rows(dtype, stream, extra):
    check(make(19, 264, dtype, stream, extra=extra))


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("C", [96, 1925, 12288])
def test_in_place(dtype, stream, C):
    x = make(300, C, dtype, stream)
    r, h = check({k: None if v is None else v.clone() for k, v in x.items()})
    same = {k: None if v is None else v.clone() for k, v in x.items()}
    r2, h2 = gdn.gdn_block_norm(**same, residual_scale=0.7, residual_out=same["residual"], h=same["y"])
    assert r2 is same["residual"] and h2 is same["y"] and torch.equal(r, r2) and torch.equal(h, h2)
    if dtype == stream:
        same = {k: None if v is None else v.clone() for k, v in x.items()}
        r2, h2 = gdn.gdn_block_norm(**same, residual_scale=0.7, residual_out=same["gate"], h=same["residual"])
        assert torch.equal(r, r2) and torch.equal(h, h2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_block_without_a_residual(dtype):
    x = make(9, 200, dtype, dtype)
    x["residual"] = None
    r, _ = check(x)
    assert r.dtype is DT[dtype]
    r32 = torch.empty(9, 200, device="cuda")
    got, _ = gdn.gdn_block_norm(**x, residual_out=r32)
    assert got is r32 and torch.equal(r32.to(DT[dtype]), r)


def test_rows_do_not_touch_one_another():
    x = make(64, 512, "bf16", "bf16")
    r, h = check(x)
    y = {k: None if v is None else v.clone() for k, v in x.items()}
    y["y"][10] = float("nan")
    y["residual"][20] = float("inf")
    r2, h2 = gdn.gdn_block_norm(**y, residual_scale=0.7)
    keep = [i for i in range(64) if i not in (10, 20)]
    assert torch.equal(r[keep], r2[keep]) and torch.equal(h[keep], h2[keep])
    assert bool(torch.isnan(h2[10]).all()) and bool(torch.isnan(h2[20]).all())


def test_constant_rows():
    x = make(5, 128, "f32", "f32", gate=False, scale=False, bias=False, affine=False)
    x["y"][:] = 2.0
    x["residual"][:] = 1.0
    r, h = gdn.gdn_block_norm(**x, rms=False)
    assert bool((r == 1).all()) and bool((h == 0).all())
