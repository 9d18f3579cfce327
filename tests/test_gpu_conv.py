"""GPU parity of gdn_conv_fwd and gdn_conv_step with the definition in fp64
(bounds: ``layer_reference``)."""
import numpy as np
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


def draw(seed, lead, C, W, dtype, extra=0, bias=True, pool=None):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = int(np.prod(lead))
    x = r(rows, C + extra).to(DT[dtype])[:, extra:].unflatten(0, lead)
    return (x, r(C, W) / W ** 0.5, 0.3 * r(C) if bias else None,
            None if pool is None else r(pool, W - 1, C).to(DT[dtype]))


def check(gdn, x, w, b, state_in, slots=None, cu=None, act="silu", in_place=False):
    y0, bound, new = R.conv(x, w, b, state_in, slots, cu, act)
    before = None if state_in is None else state_in.clone()
    state = state_in.clone() if in_place else state_in
    out = state if in_place else (None if slots is None else torch.full_like(state_in, 7))
    y, s = gdn.gdn_conv_fwd(x, w, b, state_in=state, state_out=out, slots=slots, cu_seqlens=cu, act=act)
    assert gdn.gdn_last_launch_count() == (1, 6)
    assert gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0, bound) <= 1
    if s.shape[1] == 0:
        return y, s
    touched = set()
    for i, e in enumerate(R.entries(slots, len(new))):
        if e >= 0:
            assert np.array_equal(R.f64(s[e]), new[i]), i
            touched.add(e)
    for e in set(range(s.shape[0])) - touched:  # nothing else in the pool changes
        assert torch.equal(s[e], before[e] if in_place else torch.full_like(s[e], 7))
    if not in_place and state_in is not None:
        assert torch.equal(state_in, before)
    return y, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", range(1, 9))
def test_widths(gdn, W, dtype):
    x, w, b, s = draw(W, (2, 70), 64, W, dtype, pool=2)
    check(gdn, x, w, b, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 31, 32, 33, 64, 65, 257])
def test_lengths(gdn, T, dtype):
    """Lengths below, at and above the taps, the loads in flight and the tiles."""
    x, w, b, s = draw(T, (2, T), 136, 4, dtype, pool=2)
    check(gdn, x, w, b, s)
    check(gdn, x, w, None, None, act="none")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,extra", [(1, 0), (3, 0), (7, 1), (8, 8), (63, 0), (64, 3), (129, 0), (1031, 5),
                                     (2056, 0), (4096, 64)])
def test_channels_and_strides(gdn, C, extra, dtype):
    """Odd channel counts, rows that start off 16 bytes, slices of wider rows."""
    x, w, b, s = draw(C, (2, 41), C, 3, dtype, extra=extra, pool=2)
    check(gdn, x, w, b, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[5], [0], [0, 0, 3, 0], [1, 33, 0, 64, 2, 100, 32], [31] * 40, [3] * 70])
def test_packed(gdn, lengths, dtype):
    """Empty sequences, sequences shorter than the taps, ends inside and at a tile, over 32 sequences."""
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    x, w, b, s = draw(sum(lengths), (1, sum(lengths)), 72, 4, dtype, pool=len(lengths))
    check(gdn, x, w, b, s, cu=cu)
    check(gdn, x, w, b, s, cu=cu, in_place=True)


def test_slots(gdn):
    """States in a pool: permuted, in place and from one pool to another; a
    negative slot keeps none; a slot past the pool raises the bit."""
    lengths = [4, 0, 90, 2]
    cu = torch.tensor([0, 4, 4, 94, 96], dtype=torch.int32, device="cuda")
    x, w, b, s = draw(3, (1, 96), 80, 4, "bf16", pool=9)
    slots = torch.tensor([8, 2, 5, -1], dtype=torch.int32, device="cuda")
    check(gdn, x, w, b, s, slots=slots, cu=cu)
    check(gdn, x, w, b, s, slots=slots, cu=cu, in_place=True)
    bad = torch.tensor([8, 2, 9, -1], dtype=torch.int32, device="cuda")
    pool = s.clone()
    y, _ = gdn.gdn_conv_fwd(x, w, b, state_in=pool, slots=bad, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == 0x10
    ref, bound, _ = R.conv(x, w, b, s, torch.tensor([8, 2, -1, -1]), cu, "silu")
    assert R.inside(y, ref, bound) <= 1
    assert torch.equal(pool[[0, 1, 3, 4, 5, 6, 7]], s[[0, 1, 3, 4, 5, 6, 7]]), lengths


def test_bad_span_skips_its_sequence(gdn):
    x, w, b, s = draw(4, (1, 50), 64, 4, "f32", pool=3)
    cu = torch.tensor([0, 20, 60, 50], dtype=torch.int32, device="cuda")
    y = torch.full_like(x, 5)
    gdn.gdn_conv_fwd(x, w, b, state_in=s, y=y, cu_seqlens=cu)
    assert gdn.gdn_get_device_status() == 0x1
    ref, bound, _ = R.conv(x[:, :20], w, b, s[:1], None, None, "silu")
    assert R.inside(y[:, :20], ref, bound) <= 1
    assert (y[:, 20:] == 5).all()


def test_sequences_do_not_see_one_another(gdn):
    """NaN and infinity in one sequence stay there."""
    x, w, b, s = draw(5, (3, 40), 64, 4, "f32", pool=3)
    clean, _ = gdn.gdn_conv_fwd(x, w, b, state_in=s)
    x[1] = float("nan")
    s[1] = float("inf")
    y, _ = gdn.gdn_conv_fwd(x, w, b, state_in=s)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[2], clean[2]) and torch.isnan(y[1]).all()


def test_output_slice_leaves_its_neighbours(gdn):
    x, w, b, s = draw(6, (2, 37), 100, 4, "bf16", extra=28, pool=2)
    wide = torch.full((2, 37, 120), float("nan"), dtype=x.dtype, device="cuda")
    gdn.gdn_conv_fwd(x, w, b, state_in=s, y=wide[..., 9:109])
    ref, bound, _ = R.conv(x, w, b, s, None, None, "silu")
    assert R.inside(wide[..., 9:109], ref, bound) <= 1
    assert torch.isnan(wide[..., :9]).all() and torch.isnan(wide[..., 109:]).all()


def test_offsets_past_32_bits(gdn):
    """Rows and pool entries beyond 2^31 elements."""
    C, T = 64, 40
    ld = (1 << 31) // T + 64
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, T, C), (T * ld, ld, 1))
    x.copy_(torch.randn(1, T, C, device="cuda"))
    entry = (1 << 31) // (3 * C) + 3
    pool = torch.empty(entry + 1, 3, C, dtype=torch.bfloat16, device="cuda")
    pool[entry] = torch.randn(3, C, device="cuda")
    slots = torch.tensor([entry], dtype=torch.int32, device="cuda")
    _, w, b, _ = draw(7, (1, 1), C, 4, "bf16")
    ref, bound, new = R.conv(x, w, b, pool[entry:], None, None, "silu")
    step_ref, step_bound, step_new = R.conv(x[:, :1], w, b, torch.as_tensor(new[0][None]), None, None, "silu")
    y, s = gdn.gdn_conv_fwd(x, w, b, state_in=pool, slots=slots)
    assert R.inside(y, ref, bound) <= 1 and np.array_equal(R.f64(s[entry]), new[0])
    y, s = gdn.gdn_conv_step(x[:, 0], w, b, state_in=pool, slots=slots)
    assert R.inside(y, step_ref[:, 0], step_bound[:, 0]) <= 1 and np.array_equal(R.f64(s[entry]), step_new[0])
    assert gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,C,W,extra", [(1, 64, 4, 0), (5, 1, 2, 0), (3, 1031, 3, 7), (65, 512, 4, 64), (2, 40, 8, 0),
                                         (3, 16, 1, 0), (300, 24, 4, 0)])
def test_step(gdn, N, C, W, extra, dtype):
    x, w, b, s = draw(N + C, (N,), C, W, dtype, extra=extra, pool=N)
    ref, bound, new = R.conv(x[:, None], w, b, s, None, None, "silu")
    keep = s.clone()
    y, out = gdn.gdn_conv_step(x, w, b, state_in=s)
    assert gdn.gdn_last_launch_count() == (1, 6)
    assert R.inside(y, ref[:, 0], bound[:, 0]) <= 1 and np.array_equal(R.f64(out), np.stack(new))
    assert torch.equal(s, keep)
    y2, same = gdn.gdn_conv_step(x, w, b, state_in=s, state_out=s)  # in place
    assert same is s and torch.equal(y, y2) and torch.equal(s, out)
    y3, out3 = gdn.gdn_conv_step(x, w, b, act="none")  # no state yet
    ref, bound, new = R.conv(x[:, None], w, b, None, None, None, "none")
    assert R.inside(y3, ref[:, 0], bound[:, 0]) <= 1 and np.array_equal(R.f64(out3), np.stack(new))
    assert gdn.gdn_get_device_status() == 0


def test_step_slots(gdn):
    x, w, b, s = draw(8, (4,), 96, 4, "bf16", pool=6)
    slots = torch.tensor([5, -1, 0, 3], dtype=torch.int32, device="cuda")
    ref, bound, new = R.conv(x[:, None], w, b, s, slots, None, "silu")
    pool = s.clone()
    y, out = gdn.gdn_conv_step(x, w, b, state_in=pool, slots=slots)
    assert out is pool and R.inside(y, ref[:, 0], bound[:, 0]) <= 1
    for i, e in ((0, 5), (2, 0), (3, 3)):
        assert np.array_equal(R.f64(pool[e]), new[i])
    assert torch.equal(pool[[1, 2, 4]], s[[1, 2, 4]])
    assert gdn.gdn_get_device_status() == 0
    gdn.gdn_conv_step(x, w, b, state_in=pool, slots=torch.tensor([6, 1, 2, 3], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_get_device_status() == 0x10


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps_is_the_whole_prompt(gdn, dtype):
    x, w, b, _ = draw(9, (3, 50), 72, 4, dtype)
    whole, end = gdn.gdn_conv_fwd(x, w, b)
    y, s = gdn.gdn_conv_fwd(x[:, :2].contiguous(), w, b)
    parts = [y]
    y, s = gdn.gdn_conv_fwd(x[:, 2:40].contiguous(), w, b, state_in=s, state_out=s)
    parts.append(y)
    for t in range(40, 50):
        y, s = gdn.gdn_conv_step(x[:, t], w, b, state_in=s, state_out=s)
        parts.append(y[:, None])
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, end)


def test_another_stream(gdn):
    x, w, b, s = draw(10, (2, 300), 512, 4, "bf16", pool=2)
    y, out = gdn.gdn_conv_fwd(x, w, b, state_in=s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        y2, out2 = gdn.gdn_conv_fwd(x, w, b, state_in=s, stream=stream)
        side.synchronize()
        assert torch.equal(y, y2) and torch.equal(out, out2)


def test_empty(gdn):
    x, w, b, s = draw(11, (2, 0), 16, 4, "f32", pool=2)
    y, out = gdn.gdn_conv_fwd(x, w, b, state_in=s)
    assert y.shape == x.shape and torch.equal(out, s)
    x, w, b, s = draw(11, (0, 5), 16, 4, "f32", pool=0)
    assert gdn.gdn_conv_fwd(x, w, b)[0].shape == x.shape
    assert gdn.gdn_conv_step(x[:, 0], w, b)[0].shape == (0, 16)
