"""GPU parity of gdn_ssm_fwd and gdn_ssm_step with the recurrence in fp64
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


def draw(seed, lead, ch, S, G=1, dtype="bf16", z=True, pool=None, extra=0):
    """One call's tensors: x, z and delta as slices of wider rows (``extra``), B
    and C side by side, step sizes of 1e-3 to 1e-1 after softplus."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows, dt = int(np.prod(lead)), DT[dtype]
    cut = lambda m: m.to(dt)[:, extra:].unflatten(0, lead)  # noqa: E731
    step = torch.exp(torch.rand(ch, generator=g, device="cuda") * 4.6 - 6.9)
    bc = r(rows, 2 * G * S + extra).to(dt)[:, extra:]
    return dict(x=cut(r(rows, ch + extra)), delta=cut(0.5 * r(rows, ch + extra)),
                A=-torch.arange(1, S + 1, device="cuda") * torch.exp(0.1 * r(ch, S)),
                B=bc[:, :G * S].unflatten(1, (G, S)).unflatten(0, lead),
                C=bc[:, G * S:].unflatten(1, (G, S)).unflatten(0, lead),
                D=1 + 0.1 * r(ch), z=cut(r(rows, ch + extra)) if z else None,
                delta_bias=step + torch.log(-torch.expm1(-step)), delta_softplus=True,
                state_in=None if pool is None else r(pool, ch, S))


def reference(a, slots=None, cu=None, pieces=1):
    return R.ssm(a["x"], a["delta"], a["A"], a["B"], a["C"], a["D"], a["z"], a["delta_bias"],
                 a["delta_softplus"], a["state_in"], slots, cu, pieces)


def check(gdn, a, slots=None, cu=None, in_place=False, segment=0, pieces=None, ref=None):
    """``pieces``: how many a sequence may be cut into (bounds grow with it)."""
    T = a["x"].shape[1]
    if pieces is None:
        pieces = max(1, -(-T // 64))
    y0, bound, new, eb = ref or reference(a, slots, cu, pieces)
    given = a["state_in"]
    state = given.clone() if in_place else given
    out = state if in_place else (None if slots is None else torch.full_like(given, 7))
    kw = dict(a, state_in=state, state_out=out)
    y, s = gdn.gdn_ssm_fwd(**kw, slots=slots, cu_seqlens=cu, segment=segment)
    assert gdn.gdn_last_launch_count()[1] == 7
    assert gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0, bound) <= 1
    touched = set()
    for i, e in enumerate(R.entries(slots, len(new))):
        if e >= 0:
            assert R.inside(s[e], new[i], eb[i]) <= 1, i
            touched.add(e)
    for e in set(range(s.shape[0])) - touched:
        assert torch.equal(s[e], given[e] if in_place else torch.full_like(s[e], 7))
    return y, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 2, 3, 4, 5, 8, 13, 16, 17, 31, 32, 48, 64, 65, 100, 128])
def test_state_sizes(gdn, S, dtype):
    check(gdn, draw(S, (2, 37), 40, S, dtype=dtype, pool=2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 400])
def test_lengths(gdn, T, dtype):
    a = draw(T, (2, T), 72, 16, dtype=dtype, pool=2)
    check(gdn, a)
    check(gdn, dict(a, z=None, D=None, state_in=None))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ch,G,extra", [(1, 1, 0), (3, 3, 0), (7, 1, 1), (31, 1, 0), (32, 2, 8), (33, 11, 0), (64, 4, 3),
                                        (65, 5, 0), (203, 7, 0), (256, 1, 64), (1026, 2, 0)])
def test_channels_groups_strides(gdn, ch, G, extra, dtype):
    """Odd channel counts, groups that end inside a block, rows off 16 bytes."""
    check(gdn, draw(ch + G, (2, 21), ch, 16, G, dtype, pool=2, extra=extra))
    check(gdn, draw(ch + G, (1, 70), ch, 5, G, dtype, extra=extra))


@pytest.mark.parametrize("segment", [0, 64, 128, 1000])
@pytest.mark.parametrize("lengths", [[0], [5], [0, 0, 3, 0], [1, 65, 0, 64, 2, 200, 63], [3] * 40, [64, 128, 192]])
def test_packed(gdn, lengths, segment):
    """Empty and one-token sequences, ends inside and at a piece, over 32 sequences."""
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    a = draw(sum(lengths), (1, sum(lengths)), 40, 16, pool=len(lengths))
    check(gdn, a, cu=cu, segment=segment)
    check(gdn, a, cu=cu, segment=segment, in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,segment,S", [(64, 64, 16), (65, 64, 16), (300, 64, 16), (300, 100, 16), (300, 299, 16),
                                         (513, 256, 16), (200, 64, 3), (200, 64, 50), (130, 64, 128)])
def test_pieces(gdn, T, segment, S, dtype):
    """A sequence cut into pieces gives what one piece gives, state included."""
    a = draw(T + S, (2, T), 48, S, 2, dtype, pool=2)
    ref = reference(a, pieces=-(-T // 64))
    check(gdn, a, segment=segment, ref=ref)
    n = gdn.gdn_last_launch_count()[0]
    assert n == (2 if T > (segment + 63) // 64 * 64 else 1)
    check(gdn, dict(a), segment=segment, in_place=True, ref=ref)


def test_many_pieces(gdn):
    a = draw(77, (1, 64 * 40 + 9), 40, 16, pool=1)
    check(gdn, a, segment=64)


def test_plain_step_sizes(gdn):
    """delta taken as it is: zero keeps the state, a negative one grows it, a
    huge one forgets it."""
    a = draw(12, (2, 60), 40, 16, dtype="f32", pool=2)
    a.update(delta_softplus=False, delta_bias=None, delta=a["delta"].abs() * 0.1)
    a["delta"][:, 10:20] = 0
    a["delta"][:, 30] = 1e4
    a["delta"][:, 40] = -0.05
    check(gdn, a)
    a["delta"] = torch.zeros_like(a["delta"])
    _, s = check(gdn, a)
    assert torch.equal(s, a["state_in"])


@pytest.mark.parametrize("shift", [-30.0, -12.0, 0.0, 12.0, 80.0])
def test_softplus_range(gdn, shift):
    """Step sizes from 1e-13 to 80: small ones keep their relative precision."""
    a = draw(13, (2, 40), 40, 16, dtype="f32", pool=2)
    a["delta_bias"] = torch.full_like(a["delta_bias"], shift)
    check(gdn, a)


def test_growing_state(gdn):
    """A positive A makes the state grow."""
    a = draw(14, (1, 50), 24, 8, dtype="f32", pool=1)
    check(gdn, dict(a, A=-0.2 * a["A"]))


def test_slots(gdn):
    cu = torch.tensor([0, 4, 4, 154, 156], dtype=torch.int32, device="cuda")
    a = draw(15, (1, 156), 40, 16, pool=9)
    slots = torch.tensor([8, 2, 5, -1], dtype=torch.int32, device="cuda")
    for segment in (0, 64):
        check(gdn, a, slots=slots, cu=cu, segment=segment)
        check(gdn, a, slots=slots, cu=cu, segment=segment, in_place=True)
        bad = torch.tensor([8, 2, 9, -1], dtype=torch.int32, device="cuda")
        pool = a["state_in"].clone()
        y, _ = gdn.gdn_ssm_fwd(**dict(a, state_in=pool), slots=bad, cu_seqlens=cu, segment=segment)
        assert gdn.gdn_get_device_status() == 0x10
        y0, bound, _, _ = reference(a, torch.tensor([8, 2, -1, -1]), cu, 3)
        assert R.inside(y, y0, bound) <= 1
        assert torch.equal(pool[[0, 1, 3, 4, 5, 6, 7]], a["state_in"][[0, 1, 3, 4, 5, 6, 7]])


@pytest.mark.parametrize("segment", [0, 64])
def test_bad_span_skips_its_sequence(gdn, segment):
    a = draw(16, (1, 150), 40, 16, pool=3, dtype="f32")
    cu = torch.tensor([0, 100, 160, 150], dtype=torch.int32, device="cuda")
    y = torch.full_like(a["x"], 5)
    gdn.gdn_ssm_fwd(**a, y=y, cu_seqlens=cu, segment=segment)
    assert gdn.gdn_get_device_status() == 0x1
    part = {k: (v[:, :100] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    y0, bound, _, _ = reference(dict(part, state_in=a["state_in"][:1]), pieces=2)
    assert R.inside(y[:, :100], y0, bound) <= 1
    assert (y[:, 100:] == 5).all()


def test_sequences_and_channels_do_not_see_one_another(gdn):
    a = draw(17, (3, 80), 40, 16, dtype="f32", pool=3)
    clean, cs = gdn.gdn_ssm_fwd(**a)
    a["x"][1] = float("nan")
    a["state_in"][1] = float("inf")
    a["x"][2, 30:, 7] = float("inf")
    y, s = gdn.gdn_ssm_fwd(**a)
    assert torch.equal(y[0], clean[0]) and torch.equal(s[0], cs[0])
    assert torch.equal(y[2, :30], clean[2, :30])
    others = [c for c in range(40) if c != 7]
    assert torch.equal(y[2][:, others], clean[2][:, others]) and torch.equal(s[2][others], cs[2][others])


def test_output_slice_leaves_its_neighbours(gdn):
    a = draw(18, (2, 70), 100, 16, pool=2)
    wide = torch.full((2, 70, 120), float("nan"), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_ssm_fwd(**a, y=wide[..., 9:109])
    y0, bound, _, _ = reference(a, pieces=2)
    assert R.inside(wide[..., 9:109], y0, bound) <= 1
    assert torch.isnan(wide[..., :9]).all() and torch.isnan(wide[..., 109:]).all()


def test_offsets_past_32_bits(gdn):
    ch, S, T = 64, 16, 70
    a = draw(19, (1, T), ch, S, pool=1)
    ref = reference(a, pieces=2)
    ld = (1 << 31) // T + 64
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((1, T, ch), (T * ld, ld, 1))
    x.copy_(a["x"])
    delta = big.as_strided((1, T, ch), (T * ld, ld, 1), 64)
    delta.copy_(a["delta"])
    entry = (1 << 31) // (ch * S) + 3
    pool = torch.empty(entry + 1, ch, S, device="cuda")
    pool[entry] = a["state_in"][0]
    slots = torch.tensor([entry], dtype=torch.int32, device="cuda")
    y, s = gdn.gdn_ssm_fwd(**dict(a, x=x, delta=delta, state_in=pool), slots=slots)
    assert gdn.gdn_get_device_status() == 0
    assert R.inside(y, ref[0], ref[1]) <= 1 and R.inside(s[entry], ref[2][0], ref[3][0]) <= 1
    pool[entry] = a["state_in"][0]
    one = lambda v: v[:, 0]  # noqa: E731
    b = dict(a, x=one(x), delta=one(delta), B=one(a["B"]), C=one(a["C"]), z=one(a["z"]), state_in=pool)
    y, s = gdn.gdn_ssm_step(**b, slots=slots)
    first = {k: (v[:, :1] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    ref = reference(first)
    assert R.inside(y, ref[0][:, 0], ref[1][:, 0]) <= 1 and R.inside(s[entry], ref[2][0], ref[3][0]) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,ch,S,G,extra", [(1, 64, 16, 1, 0), (5, 1, 1, 1, 0), (3, 203, 13, 7, 0), (65, 128, 16, 2, 64),
                                            (2, 40, 128, 1, 0), (3, 33, 64, 3, 5), (300, 24, 16, 1, 0), (7, 50, 6, 5, 3)])
def test_step(gdn, N, ch, S, G, extra, dtype):
    a = draw(N + ch, (N, 1), ch, S, G, dtype, pool=N, extra=extra)
    y0, bound, new, eb = reference(a)
    b = {k: (v[:, 0] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    keep = a["state_in"].clone()
    y, s = gdn.gdn_ssm_step(**b)
    assert gdn.gdn_last_launch_count() == (1, 7) and gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1 and R.inside(s, np.stack(new), np.stack(eb)) <= 1
    assert torch.equal(a["state_in"], keep)
    y2, same = gdn.gdn_ssm_step(**b, state_out=b["state_in"])
    assert same is b["state_in"] and torch.equal(y2, y) and torch.equal(same, s)
    y3, s3 = gdn.gdn_ssm_step(**dict(b, state_in=None, z=None, D=None))
    y0, bound, new, eb = reference(dict(a, state_in=None, z=None, D=None))
    assert R.inside(y3, y0[:, 0], bound[:, 0]) <= 1 and R.inside(s3, np.stack(new), np.stack(eb)) <= 1


def test_step_slots(gdn):
    a = draw(20, (4, 1), 48, 16, pool=6)
    slots = torch.tensor([5, -1, 0, 3], dtype=torch.int32, device="cuda")
    y0, bound, new, eb = reference(a, slots)
    pool = a["state_in"].clone()
    b = {k: (v[:, 0] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
    y, out = gdn.gdn_ssm_step(**dict(b, state_in=pool), slots=slots)
    assert out is pool and gdn.gdn_get_device_status() == 0
    assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1
    for i, e in ((0, 5), (2, 0), (3, 3)):
        assert R.inside(pool[e], new[i], eb[i]) <= 1
    assert torch.equal(pool[[1, 2, 4]], a["state_in"][[1, 2, 4]])
    gdn.gdn_ssm_step(**dict(b, state_in=pool), slots=torch.tensor([6, 1, 2, 3], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_get_device_status() == 0x10


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps_is_the_whole_prompt(gdn, dtype):
    T0, T1 = 130, 10
    a = draw(21, (3, T0 + T1), 72, 16, dtype=dtype, pool=3)
    y0, bound, new, eb = reference(a, pieces=3)
    cut = lambda lo, hi: {k: (v[:, lo:hi].contiguous() if k in ("x", "delta", "B", "C", "z") else v)  # noqa: E731
                          for k, v in a.items()}
    y, s = gdn.gdn_ssm_fwd(**cut(0, T0))
    parts = [y]
    for t in range(T0, T0 + T1):
        b = {k: (v[:, t] if k in ("x", "delta", "B", "C", "z") else v) for k, v in a.items()}
        y, s = gdn.gdn_ssm_step(**dict(b, state_in=s), state_out=s)
        parts.append(y[:, None])
    assert R.inside(torch.cat(parts, 1), y0, bound) <= 1
    assert R.inside(s, np.stack(new), np.stack(eb)) <= 1


def test_repeats_bit_for_bit_and_on_another_stream(gdn):
    a = draw(22, (2, 700), 256, 16, pool=2)
    for segment in (0, 128):
        y, s = gdn.gdn_ssm_fwd(**a, segment=segment)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            y2, s2 = gdn.gdn_ssm_fwd(**a, segment=segment, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and torch.equal(s, s2)


def test_empty(gdn):
    a = draw(23, (2, 0), 24, 16, pool=2)
    y, s = gdn.gdn_ssm_fwd(**a)
    assert y.shape == a["x"].shape and torch.equal(s, a["state_in"])
    a = draw(23, (0, 5), 24, 16)
    assert gdn.gdn_ssm_fwd(**a)[0].shape == (0, 5, 24)


@pytest.mark.parametrize("segment", [4096, 512])
def test_long_memory_does_not_drift(gdn, segment):
    """States alone, decaying by 2^-v, v in [2^-11, 2^-10], for 4096 tokens: the
    decays' errors may not add up in one direction by more than 1/16 of an ulp
    (2^-28) per token on average, beside 2^-24 of the exponents' sum of 2 to 4
    and as much again for the constants' rounding."""
    T, ch = 4096, 256
    g = torch.Generator("cuda").manual_seed(24)
    zero = torch.zeros(1, T, ch, device="cuda")
    delta = (1 + torch.rand(1, T, ch, generator=g, device="cuda")) * (np.log(2) * 2.0 ** -11)
    A = -torch.ones(ch, 16, device="cuda")
    bc = torch.zeros(1, T, 1, 16, device="cuda")
    h = 1 + torch.rand(1, ch, 16, generator=g, device="cuda")
    _, s = gdn.gdn_ssm_fwd(zero, delta, A, bc, bc, state_in=h, segment=segment)
    exact = h.double() * torch.exp(-delta.double().sum(1))[..., None]
    mean = float(((s.double() - exact) / exact).mean())
    assert abs(mean) <= T * 2.0 ** -28 + 2 * 4 * 2.0 ** -24
