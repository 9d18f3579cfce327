"""Scans long enough to come round their ring of tiles several times, on rows
of every alignment and in packs of many sequences, against the recurrence in
fp64 (bounds: ``layer_reference``)."""
import numpy as np
import pytest
import torch

from test_gpu_ssm import check, draw, gdn, reference  # noqa: F401

pytestmark = pytest.mark.gpu

# (channels, states, groups, dtype): words of two, single elements, odd numbers of states, groups
# that end inside a block of 64 channels, more states per lane, states in two parts
SHAPES = [(44, 16, 1, "bf16"), (43, 16, 1, "bf16"), (64, 13, 1, "bf16"), (70, 16, 7, "bf16"), (66, 5, 2, "bf16"), (43, 3, 1, "bf16"),
          (43, 24, 1, "bf16"), (46, 50, 1, "bf16"), (43, 100, 1, "bf16"), (64, 27, 1, "bf16"), (64, 24, 1, "bf16"), (136, 128, 1, "bf16"),
          (43, 16, 1, "f32"), (66, 13, 3, "f32"), (64, 16, 1, "f32"), (43, 50, 1, "f32"), (43, 100, 1, "f32"), (64, 32, 1, "f32")]


@pytest.mark.parametrize("T", [81, 96, 97, 113, 250])
@pytest.mark.parametrize("ch,S,G,dtype", SHAPES)
def test_ring_comes_round(gdn, ch, S, G, dtype, T):  # noqa: F811
    a = draw(ch + T, (2, T), ch, S, G, dtype, pool=2)
    ref = reference(a)
    check(gdn, a, segment=T, ref=ref)
    check(gdn, a, segment=T, ref=ref, in_place=True)
    check(gdn, dict(a, z=None, state_in=None), segment=T, pieces=1)


@pytest.mark.parametrize("segment", [256, 1000])
@pytest.mark.parametrize("ch,S,G,dtype", SHAPES)
def test_long_pieces(gdn, ch, S, G, dtype, segment):  # noqa: F811
    """700 tokens whole, or in pieces of 16 tiles."""
    a = draw(ch + S, (1, 700), ch, S, G, dtype, pool=1)
    check(gdn, a, segment=segment, pieces=3 if segment < 700 else 1)
    assert gdn.gdn_last_launch_count()[0] == (2 if segment < 700 else 1)


@pytest.mark.parametrize("segment", [0, 128])
@pytest.mark.parametrize("ch,S,G,dtype", [(44, 16, 1, "bf16"), (43, 13, 1, "bf16"), (70, 16, 7, "bf16"), (43, 16, 1, "f32"),
                                          (64, 16, 1, "bf16")])
def test_packs(gdn, ch, S, G, dtype, segment):  # noqa: F811
    """Ends inside a tile after several rounds of the ring; odd offsets."""
    lengths = [205, 1, 0, 131, 97, 16, 250]
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    a = draw(ch, (1, sum(lengths)), ch, S, G, dtype, pool=9)
    slots = torch.tensor([8, 2, 5, -1, 0, 7, 3], dtype=torch.int32, device="cuda")
    check(gdn, a, slots=slots, cu=cu, segment=segment, pieces=4)
    check(gdn, a, slots=slots, cu=cu, segment=segment, pieces=4, in_place=True)


@pytest.mark.parametrize("N", [64, 65, 130])
def test_packs_of_many_sequences(gdn, N):  # noqa: F811
    lengths = [(7 * i) % 23 + (90 if i % 29 == 0 else 0) for i in range(N)]
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    a = draw(N, (1, sum(lengths)), 40, 16, pool=N)
    check(gdn, a, cu=cu, pieces=2)
    check(gdn, a, cu=cu, segment=64, in_place=True, pieces=2)
