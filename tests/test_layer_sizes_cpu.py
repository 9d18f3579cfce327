"""Sizes that the operators around the recurrence refuse or take, on the host (CPU only)."""
import pytest

from test_layer_cpu import P, conv_fwd, conv_step, lib, ssm_fwd, ssm_step  # noqa: F401

TOP = 2 ** 31 - 2 ** 16
FAR = dict(x=1 << 50, y=1 << 52)


@pytest.mark.parametrize("count", [TOP + 1, 2 ** 31 - 1])
def test_counts_past_32_bit_arithmetic_are_refused(lib, count):  # noqa: F811
    """Token numbers run a few tiles past the end of a sequence."""
    for cu in (None, P["cu"]):
        assert conv_fwd(lib, B=1, T=count, C=1, ldx=1, ldy=1, W=1, cu=cu, **FAR) == 2
        assert ssm_fwd(lib, B=1, T=count, C=1, S=1, ld=(1,) * 6, cu=cu, delta=1 << 54, Bm=1 << 55, Cm=1 << 56, **FAR) == 2
    assert conv_fwd(lib, B=count, T=0) == 2 and ssm_fwd(lib, B=count, T=0) == 2
    assert conv_step(lib, N=count, C=1, W=1, ldx=1, ldy=1, **FAR) == 2
    assert ssm_step(lib, N=count, C=1, S=1, ld=(1,) * 6, delta=1 << 54, Bm=1 << 55, Cm=1 << 56, **FAR) == 2


def test_large_counts_are_taken(lib):  # noqa: F811
    """No sequences of the longest length, or the most sequences without tokens and states."""
    assert conv_fwd(lib, B=0, T=TOP) == 0 and ssm_fwd(lib, B=0, T=TOP) == 0
    assert conv_fwd(lib, B=TOP, T=0) == 0 and ssm_fwd(lib, B=TOP, T=0) == 0


def test_rows_of_b_past_32_bits_are_refused(lib):  # noqa: F811
    """Columns of B and C are numbered in 32 bits."""
    G = 1 << 24
    kw = dict(C=G, G=G, S=128, A=1 << 40, delta=1 << 54, Bm=1 << 55, Cm=1 << 56, **FAR)
    ld = (G, G, G * 128, G * 128, G, G)
    assert ssm_fwd(lib, B=1, T=1, ld=ld, **kw) == 2 and ssm_step(lib, N=1, ld=ld, so=1 << 57, pool=1, **kw) == 2
