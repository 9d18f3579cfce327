"""Linear attention with a decay for each head against its definition in fp64:
prompts (whole, packed, in pieces) and single tokens, on both kernels."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from layer_reference import inside
from linattn_reference import linattn

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lead, H, G, dk, dv, dtype, seed=0, extra=0, fixed=False, rate=0.1):
    g = torch.Generator("cuda").manual_seed(seed)
    rows = 1
    for n in lead:
        rows *= n
    p = torch.randn(rows, extra + 2 * G * dk + H * dv, generator=g, device="cuda", dtype=DT[dtype])
    q, k, v = p[:, extra:].split((G * dk, G * dk, H * dv), 1)
    shape = lambda t, n, d: t.unflatten(1, (n, d)).unflatten(0, lead)  # noqa: E731
    e = torch.rand(*((H,) if fixed else tuple(lead) + (H,)), generator=g, device="cuda")
    return dict(q=shape(q, G, dk), k=shape(k, G, dk), v=shape(v, H, dv), log_decay=-rate * e)


def on_tensor_cores(x):
    q, v = x["q"], x["v"]
    lds = [t.stride(-3) for t in (q, x["k"], v)]
    return (v.dtype is torch.bfloat16 and q.shape[-1] % 8 == 0 and v.shape[-1] % 8 == 0 and all(n % 8 == 0 for n in lds)
            and all(x[n].data_ptr() % 16 == 0 for n in "qkv"))


def check(x, scale=0.25, state_in=None, slots=None, cu=None, segment=0, pieces=1, tol=1.0):
    o, S = gdn.gdn_linattn_fwd(**x, scale=scale, state_in=state_in, slots=slots, cu_seqlens=cu, segment=segment,
                               state_out=None if state_in is None else torch.full_like(state_in, 7.0))
    assert gdn.gdn_get_device_status() == 0
    ro, bo, rS, bS = linattn(**x, scale=scale, state_in=state_in, slots=slots, cu=cu, parts=on_tensor_cores(x), pieces=pieces)
    assert inside(o, ro, bo) <= tol
    where = range(len(rS)) if slots is None else slots.tolist()
    for i, e in enumerate(where):
        if e >= 0:
            assert inside(S[e], rS[i], bS[i] + 1e-37) <= tol, i
    if slots is not None and state_in is not None:      # entries of nobody stay
        rest = [i for i in range(len(S)) if i not in set(where)]
        assert bool((S[rest] == 7.0).all())
    return o, S


SHAPES = [(4, 4, 128, 128), (4, 2, 64, 64), (2, 1, 96, 192), (3, 3, 8, 8), (4, 1, 128, 72), (2, 2, 40, 24), (1, 1, 120, 256)]


@pytest.mark.parametrize("H,G,dk,dv", SHAPES)
@pytest.mark.parametrize("T", [1, 31, 128, 129, 300, 517])
def test_prompts_bf16(H, G, dk, dv, T):
    check(make((2, T), H, G, dk, dv, "bf16", seed=T))


@pytest.mark.parametrize("H,G,dk,dv", [(2, 2, 128, 128), (6, 3, 77, 45), (2, 1, 64, 65), (1, 1, 1, 1), (3, 1, 33, 130)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 32, 33, 200])
def test_prompts_any_rows(H, G, dk, dv, dtype, T):
    check(make((2, T), H, G, dk, dv, dtype, seed=T, extra=5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fixed", [True, False])
@pytest.mark.parametrize("segment", [0, 128, 256])
def test_packed_with_states_in_slots(dtype, fixed, segment):
    lengths = [200, 0, 1, 128, 333, 129, 257]
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")
    x = make((1, sum(lengths)), 4, 2, 64, 64, dtype, seed=3, fixed=fixed, extra=8)
    g = torch.Generator("cuda").manual_seed(1)
    pool = torch.randn(9, 4, 64, 64, generator=g, device="cuda")
    slots = torch.tensor([8, 2, 0, 5, -1, 3, 1], dtype=torch.int32, device="cuda")
    check(x, state_in=pool, slots=slots, cu=cu, segment=segment, pieces=1 + (segment > 0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_equal_whole_sequences(dtype):
    x = make((2, 1000), 2, 1, 128, 64, dtype, seed=5, rate=0.02)
    S0 = torch.randn(2, 2, 64, 128, device="cuda")
    a = check(x, state_in=S0)
    b = check(x, state_in=S0, segment=256, pieces=4)
    # two roundings of nearly the same values
    assert float((a[0].float() - b[0].float()).norm() / a[0].float().norm()) < (2e-3 if dtype == "bf16" else 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("segment", [0, 128])
def test_in_place_states_and_outputs_given(dtype, segment):
    x = make((2, 260), 2, 2, 64, 128, dtype, seed=7)
    S = torch.randn(2, 2, 128, 64, device="cuda")
    ro, bo, rS, bS = linattn(**x, scale=1.0, state_in=S, slots=None, cu=None, parts=dtype == "bf16", pieces=3)
    wide = torch.full((2, 260, 2 * 128 + 16), 3.0, device="cuda", dtype=DT[dtype])
    o = wide[..., 8:264].unflatten(-1, (2, 128))
    got, out = gdn.gdn_linattn_fwd(**x, state_in=S, state_out=S, o=o, segment=segment)
    assert got is o and out is S
    assert inside(o, ro, bo) <= 1 and all(inside(S[i], rS[i], bS[i]) <= 1 for i in range(2))
    assert bool((wide[..., :8] == 3).all()) and bool((wide[..., 264:] == 3).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [[0], [5, 6], [31, 32], [100, 127, 128], [299]])
def test_tokens_that_forget(dtype, at):
    x = make((1, 300), 2, 1, 64, 64, dtype, seed=9)
    x["log_decay"][:, at] = -float("inf")
    x["log_decay"][:, 50, 0] = -1e30
    x["log_decay"][:, 60, 1] = -90.0
    check(x, state_in=torch.randn(1, 2, 64, 64, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [0.0, 1e-4, 1.0, 20.0])
def test_decays_of_every_size(dtype, rate):
    check(make((1, 400), 2, 2, 64, 64, dtype, seed=11, rate=rate))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_that_fall_and_rise_within_a_block(dtype):
    """Sums that pass 2^-126 on the way, though the block's own does not; growth up to e^40."""
    x = make((1, 200), 2, 1, 64, 64, dtype, seed=17)
    for at, g in ((40, -60.0), (41, -60.0), (44, 20.0), (45, 20.0), (130, -70.0), (131, -20.0), (132, 9.0), (133, 8.0)):
        x["log_decay"][:, at, 0] = g
    check(x, state_in=torch.randn(1, 2, 64, 64, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fall", [-40.0, -62.0, -70.0, -82.0])
def test_tokens_behind_a_steep_decay_are_seen(dtype, fall):
    """A token that all but forgets, then tokens whose outputs come from those just behind it alone."""
    x = make((1, 200), 2, 1, 64, 64, dtype, seed=19)
    x = {n: t.clone() for n, t in x.items()}
    x["log_decay"][:, 1] = fall
    x["log_decay"][:, 32] = -5.7
    x["v"][:, 32:60] = 0
    check(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_decay"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_token_sees_nothing_of_those_behind_it(dtype, name, value):
    """What is infinite or NaN at a token leaves the outputs before it, and other sequences, as they were."""
    lengths = [150, 100]
    cu = torch.tensor([0, 150, 250], dtype=torch.int32, device="cuda")
    x = make((1, 250), 2, 1, 64, 64, dtype, seed=13)
    x = {n: t.clone() for n, t in x.items()}
    want, states = gdn.gdn_linattn_fwd(**x, cu_seqlens=cu)
    for t, first, last in ((140, 0, 140), (150, 0, 150)):
        y = {n: v.clone() for n, v in x.items()}
        y[name][0, t] = value
        o, S = gdn.gdn_linattn_fwd(**y, cu_seqlens=cu)
        assert torch.equal(o[0, first:last], want[0, first:last])
        if t == 140:
            assert torch.equal(o[0, 150:], want[0, 150:])
            assert torch.equal(S[1], states[1])
        else:
            assert torch.equal(S[0], states[0])
    assert gdn.gdn_get_device_status() == 0 and sum(lengths) == 250


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["k", "v", "log_decay"])
def test_a_piece_sees_nothing_of_those_behind_it(dtype, name):
    """The same where the sequence is cut: outputs ahead of the token, and the other sequences' outputs and states."""
    cu = torch.tensor([0, 300, 640], dtype=torch.int32, device="cuda")
    x = {n: t.clone() for n, t in make((1, 640), 2, 1, 64, 64, dtype, seed=23).items()}
    want, states = gdn.gdn_linattn_fwd(**x, cu_seqlens=cu, segment=128)
    for t, first, last, other in ((290, 0, 290, 1), (300, 0, 300, 0), (200, 0, 200, 1)):
        y = {n: v.clone() for n, v in x.items()}
        y[name][0, t] = float("inf")
        o, S = gdn.gdn_linattn_fwd(**y, cu_seqlens=cu, segment=128)
        assert torch.equal(o[0, first:last], want[0, first:last]) and torch.equal(S[other], states[other])
    assert gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_come_through(dtype):
    """v = inf at one token: o and S are infinite in that column from there on, where nothing is zero."""
    x = {n: t.clone() for n, t in make((1, 200), 1, 1, 64, 64, dtype, seed=15).items()}
    x["q"].abs_().add_(0.5)
    x["k"].abs_().add_(0.5)
    x["v"][0, 70, 0, 3] = float("inf")
    o, S = gdn.gdn_linattn_fwd(**x)
    assert bool((o[0, 70:, 0, 3] == float("inf")).all()) and bool((S[0, 0, 3] == float("inf")).all())
    rest = torch.arange(64) != 3
    assert bool(torch.isfinite(o[0, :, 0][:, rest]).all()) and bool(torch.isfinite(o[0, :70]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,dk,dv", [(4, 4, 128, 128), (4, 2, 64, 64), (6, 3, 77, 45), (2, 1, 96, 192), (1, 1, 1, 1), (2, 2, 34, 7)])
@pytest.mark.parametrize("N", [1, 5, 67])
def test_steps(dtype, H, G, dk, dv, N):
    x = make((N,), H, G, dk, dv, dtype, seed=N, extra=3 if N == 5 else 0)
    g = torch.Generator("cuda").manual_seed(2)
    pool = torch.randn(N + 3, H, dv, dk, generator=g, device="cuda")
    slots = torch.randperm(N + 3, generator=g, device="cuda")[:N].int()
    if N > 1:
        slots[1] = -1
    ro, bo, rS, bS = linattn(**x, scale=0.5, state_in=pool, slots=slots, cu=None, steps=True)
    before = pool.clone()
    o, S = gdn.gdn_linattn_step(**x, scale=0.5, state_in=pool, slots=slots)
    assert S is pool and gdn.gdn_get_device_status() == 0
    assert inside(o, ro, bo) <= 1
    used = set()
    for i, e in enumerate(slots.tolist()):
        if e >= 0:
            assert inside(S[e], rS[i], bS[i]) <= 1
            used.add(e)
    rest = [e for e in range(N + 3) if e not in used]
    assert torch.equal(S[rest], before[rest])


def test_step_of_fixed_decays_and_no_states():
    x = make((3,), 2, 2, 64, 64, "bf16", fixed=True)
    o, S = gdn.gdn_linattn_step(**x)
    ro, bo, rS, bS = linattn(**x, scale=1.0, state_in=None, slots=None, cu=None, steps=True)
    assert inside(o, ro, bo) <= 1 and all(inside(S[i], rS[i], bS[i] + 1e-37) <= 1 for i in range(3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps_is_one_longer_prompt(dtype):
    x = make((2, 150), 4, 2, 64, 64, dtype, seed=21)
    cut = lambda a, b: {n: t[:, a:b].contiguous() for n, t in x.items()}  # noqa: E731
    whole, final = gdn.gdn_linattn_fwd(**x)
    first, S = gdn.gdn_linattn_fwd(**cut(0, 140))
    parts = [first]
    for t in range(140, 150):
        o, S = gdn.gdn_linattn_step(**{n: v[:, t].contiguous() for n, v in x.items()}, state_in=S, state_out=S)
        parts.append(o[:, None])
    got = torch.cat(parts, 1)
    _, bound, rS, bS = linattn(**x, scale=1.0, state_in=None, slots=None, cu=None, parts=dtype == "bf16")
    assert inside(got, whole.double().cpu().numpy(), 2 * bound) <= 1
    assert all(inside(S[i], rS[i], 2 * bS[i]) <= 1 for i in range(2))


@pytest.mark.parametrize("T", [0, 1, 40])
def test_empty_sequences_hand_their_states_on(T):
    S0 = torch.randn(3, 2, 16, 16, device="cuda")
    cu = torch.tensor([0, 0, T, T], dtype=torch.int32, device="cuda")
    x = make((1, T), 2, 2, 16, 16, "bf16")
    o, S = gdn.gdn_linattn_fwd(**x, state_in=S0, cu_seqlens=cu)
    assert torch.equal(S[0], S0[0]) and torch.equal(S[2], S0[2]) and torch.equal(S[1], S0[1]) == (T == 0)


def test_bad_spans_and_slots_are_skipped():
    x = make((1, 200), 2, 2, 64, 64, "bf16")
    cu = torch.tensor([0, 100, 90, 200], dtype=torch.int32, device="cuda")
    S0 = torch.randn(3, 2, 64, 64, device="cuda")
    want, _ = gdn.gdn_linattn_fwd(**{n: t[:, :100].contiguous() for n, t in x.items()})
    o = torch.full_like(x["v"].contiguous(), 5.0)
    gdn.gdn_linattn_fwd(**x, cu_seqlens=torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda"), o=o)
    assert gdn.gdn_get_device_status() == 1                       # GDN_DEV_BAD_SEQLENS
    assert torch.equal(o[:, :100], want) and bool((o[:, 100:] == 5).all())
    del cu
    for segment in (0, 128):
        slots = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
        two = {n: t.view(2, 100, *t.shape[2:]) for n, t in ((n, t.contiguous()) for n, t in x.items())}
        pool = S0.clone()
        gdn.gdn_linattn_fwd(**two, state_in=pool, slots=slots, segment=segment)
        assert gdn.gdn_get_device_status() == 0x10                # GDN_DEV_BAD_SLOT
        assert torch.equal(pool[1:], S0[1:]) and not torch.equal(pool[0], S0[0])
