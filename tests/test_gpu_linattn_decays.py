"""Decays that rise, fall and fall again within a block of 32 tokens: finite inputs
give finite outputs, and what lies behind a steep token is neither lost nor less
precise.  Against the definition in fp64."""
import numpy as np
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from layer_reference import EX, U, stored
from linattn_exact import agrees, walk
from test_gpu_linattn import check, make, on_tensor_cores

pytestmark = pytest.mark.gpu


def decayed(dtype, T, at, seed, base=-0.05):
    x = {n: t.clone() for n, t in make((1, T), 2, 1, 64, 64, dtype, seed=seed).items()}
    x["log_decay"][:] = base
    for t, g in at.items():
        x["log_decay"][0, t] = g
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [{5: 55.0, 6: -55.0, 7: -55.0}, {40: 55.0, 41: -55.0, 42: -55.0, 43: 54.0},
                                {96: 60.0, 100: -61.0, 127: -55.0}, {3: 30.0, 40: 30.0, 70: -62.0, 100: -62.0}])
def test_a_rise_then_a_fall_within_a_block(dtype, at):
    """Sums of decays of both signs, none over 128 tokens above 80: all of it is finite."""
    x = decayed(dtype, 200, at, seed=31)
    for t in at:                                  # what the rise multiplies stays of ordinary size
        x["k"][0, :t] *= 2.0 ** -30 if at[t] > 0 else 1.0
    check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fall,second", [(-62.0, -28.0), (-40.0, -60.0), (-61.0, -61.0), (-30.0, -62.0)])
def test_tokens_seen_over_two_steep_ones(dtype, fall, second):
    """A fall early in a block and another early in the next: what is left of the tokens between is all there is."""
    x = decayed(dtype, 200, {1: fall, 33: second}, seed=33, base=-0.01)
    x["v"][0, :2] = 0
    x["v"][0, 32:64] = 0
    o, S = gdn.gdn_linattn_fwd(**x, scale=0.25)
    assert gdn.gdn_get_device_status() == 0
    ro, bo, rS, bS = walk(**x, scale=0.25, parts=on_tensor_cores(x))
    assert agrees(o, ro, bo) <= 1 and agrees(S[0], rS[0], bS[0] + 1e-37) <= 1


@pytest.mark.parametrize("scale", [2.0 ** 40, 2.0 ** -60, -3.0, 0.0])
def test_scales_of_every_size(scale):
    """Steep and flat decays under a scale that no factor may take along past what fp32 holds."""
    x = decayed("bf16", 200, {1: -61.0, 40: 10.0, 70: -30.0}, seed=37)
    o, _ = gdn.gdn_linattn_fwd(**x, scale=scale)
    ro, bo, _, _ = walk(**x, scale=scale, parts=True)
    assert agrees(o, ro, bo) <= 1 and gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("steep", [-50.0, -60.0, -80.0, -87.0])
@pytest.mark.parametrize("where", [range(8), range(0, 16, 2), range(1), range(0, 24, 3)])
def test_flat_decays_behind_steep_ones(dtype, steep, where):
    """Outputs of a single term: the factor of two tokens depends on what lies between them, not on what the
    block of 32 began with."""
    T, at, dk, dv = 96, 25, 8, 64
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator("cuda").manual_seed(41)
    q = torch.zeros(1, T, 1, dk, device="cuda", dtype=dt)
    q[..., 0] = 1
    v = torch.zeros(1, T, 1, dv, device="cuda", dtype=dt)
    v[0, at, 0] = torch.randn(dv, generator=gen, device="cuda").to(dt)
    g = -0.05 * torch.rand(1, T, 1, generator=gen, device="cuda")
    g[0, list(where)] = steep
    o, _ = gdn.gdn_linattn_fwd(q, q, v, g)
    sums = np.cumsum(g[0, :, 0].double().cpu().numpy())
    D = np.maximum(sums[at] - sums, 0)                       # between the token and the output
    want = np.where(np.arange(T) >= at, np.exp(-D), 0)[:, None] * v[0, at, 0].double().cpu().numpy()
    # the factor's exponential and those that carry a state on (twice a block: 6 and 6), the roundings of the sum
    # between, and three products; on tensor cores what two parts leave, twice
    rel = (14 * EX + 12 * U * D + 16 * U + (2.0 ** -15 if dtype == "bf16" else 0))[:, None]
    assert agrees(o[0, :, 0], want, stored(want, rel * np.abs(want), dt)) <= 1
