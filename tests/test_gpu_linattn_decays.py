"""Decays that rise, fall and fall again within a block of 32 tokens: finite inputs
give finite outputs.  Against the definition in fp64."""
import pytest

from test_gpu_linattn import check, make

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
