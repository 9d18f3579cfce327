"""Convolution of rows read in words of two elements and in words of 16 bytes,
over several tiles: rows of even widths, slices that start off 16 bytes, packs."""
import numpy as np
import pytest
import torch

from test_gpu_conv import check, draw, gdn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("C,extra", [(2, 0), (66, 0), (70, 2), (258, 0), (1030, 6), (64, 2)])
def test_words_of_two(gdn, C, extra, W, dtype):  # noqa: F811
    x, w, b, s = draw(C + W, (2, 75), C, W, dtype, extra=extra, pool=2)
    check(gdn, x, w, b, s)
    check(gdn, x, w, None, None, act="none")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [63, 66, 72])
@pytest.mark.parametrize("T", [1, 4, 5, 8, 9, 127, 129, 300])
def test_lengths(gdn, T, C, dtype):  # noqa: F811
    x, w, b, s = draw(T + C, (2, T), C, 4, dtype, pool=2)
    check(gdn, x, w, b, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [66, 67])
def test_packs(gdn, C, dtype):  # noqa: F811
    lengths = [1, 133, 0, 64, 2, 301, 32, 3] * 5
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    x, w, b, s = draw(C, (1, sum(lengths)), C, 4, dtype, pool=len(lengths))
    check(gdn, x, w, b, s, cu=cu)
    check(gdn, x, w, b, s, cu=cu, in_place=True)
