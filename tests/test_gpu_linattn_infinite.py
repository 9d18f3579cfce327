"""Infinities and NaN in linear attention: forgotten ones do not come back, whole or in
pieces, columns that fill up a tile, or lanes without one in a step, make none, and
states and values stay what they are under decays that forget nothing."""
import numpy as np
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from linattn_exact import agrees, walk
from test_gpu_linattn import make, on_tensor_cores

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def positive(T, H, G, dk, dv, dtype, seed=0, rate=0.05, extra=0, lead=1):
    """q and k above zero: an infinity meets no other of the other sign."""
    x = {n: t.clone() for n, t in make((lead, T), H, G, dk, dv, dtype, seed=seed, rate=rate).items()}
    for n in "qk":
        x[n].abs_().add_(0.5)
    if extra:                                     # rows that tensor copies cannot take
        for n in "qkv":
            t = x[n]
            wide = torch.zeros(*t.shape[:2], t[0, 0].numel() + extra, dtype=t.dtype, device="cuda")
            wide[..., extra:] = t.flatten(2)
            x[n] = wide[..., extra:].unflatten(-1, t.shape[2:])
    return x


def check(x, odd=(), state=None, segment=0, pieces=1):
    """``odd``: (name, index, value).  Bounds are those of the same call without the odd values, whose finite
    results are the same."""
    y = {n: t.clone() if t.is_contiguous() else t for n, t in x.items()}
    for name, at, value in odd:
        y[name] = y[name].clone() if y[name] is x[name] else y[name]
        y[name][at] = value
    plain = {n: t.clone() for n, t in x.items()}
    for name, at, _ in odd:
        plain[name][at] = 0
    tc = on_tensor_cores(y)
    S0 = None if state is None else torch.nan_to_num(state, nan=0, posinf=0, neginf=0)
    ro, _, rS, _ = walk(**y, state_in=state)
    so, bo, sS, bS = walk(**plain, state_in=S0, parts=tc, pieces=pieces)
    fin = np.isfinite(ro)
    assert np.allclose(ro[fin], so[fin], rtol=1e-9, atol=1e-30)
    # an infinite k meets the parts of what it multiplies, on tensor cores, which may have both signs
    kinds = not (tc and any(name == "k" for name, _, _ in odd))
    o, S = gdn.gdn_linattn_fwd(**y, state_in=state, segment=segment)
    assert gdn.gdn_get_device_status() == 0
    assert agrees(o, ro, bo, kinds) <= 1
    for i in range(len(rS)):
        assert agrees(S[i], rS[i], bS[i] + 1e-37, kinds) <= 1


FORMS = [("f32", 64, 64, 0), ("bf16", 64, 64, 3), ("f32", 128, 32, 0), ("bf16", 64, 64, 0), ("bf16", 128, 72, 0)]


@pytest.mark.parametrize("dtype,dk,dv,extra", FORMS)
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("t,forget", [(70, 73), (70, 100), (70, 130), (70, 200), (127, 128), (130, 131), (131, 160)])
@pytest.mark.parametrize("segment", [0, 128])
def test_what_is_forgotten_does_not_come_back(dtype, dk, dv, extra, name, value, t, forget, segment):
    """An odd value, then a token that forgets: in the same 32 tokens, the same chunk, the next, the next piece."""
    x = positive(300, 2, 1, dk, dv, dtype, seed=t, extra=extra)
    x["log_decay"][0, forget] = -INF if t % 2 else -100.0
    check(x, [(name, (0, t, 0, 3), value)], segment=segment, pieces=1 + segment // 128)


@pytest.mark.parametrize("dtype,dk,dv,extra", [("f32", 77, 45, 0), ("f32", 40, 64, 0), ("bf16", 40, 64, 0), ("bf16", 72, 72, 0),
                                               ("bf16", 8, 8, 0), ("bf16", 120, 64, 0), ("bf16", 77, 45, 3)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_columns_that_fill_up_a_tile_stay_out(dtype, dk, dv, extra, value):
    """d_k that is no whole tile: an infinite v makes its column infinite from there on, not NaN."""
    check(positive(300, 2, 2, dk, dv, dtype, seed=dk, extra=extra), [("v", (0, 70, 0, 3), value)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(96, 64), (40, 7), (64, 64), (128, 128), (33, 5), (1, 1)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_steps_of_an_infinite_value(dtype, dk, dv, value):
    """d_k that leaves lanes of a warp without a column."""
    x = {n: t[:, 0].contiguous() for n, t in positive(1, 2, 2, dk, dv, dtype, seed=dk, lead=3).items()}
    y = {n: t.clone() for n, t in x.items()}
    y["v"][1, 0, 0] = value
    S0 = torch.randn(3, 2, dv, dk, device="cuda")
    o, S = gdn.gdn_linattn_step(**y, state_in=S0)
    lay = lambda z: {n: t[:, None] for n, t in z.items()}  # noqa: E731
    ro, _, rS, _ = walk(**lay(y), state_in=S0)
    x["v"][1, 0, 0] = 0
    _, bo, _, bS = walk(**lay(x), state_in=S0)
    assert agrees(o[:, None], ro, bo) <= 1
    assert all(agrees(S[i], rS[i], bS[i]) <= 1 for i in range(3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [-0.2, -1.0, -3.0])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("segment", [0, 512])
def test_odd_states_stay_until_a_token_forgets(dtype, rate, value, segment):
    """Decays whose product over a chunk or a piece is below 2^-126, none of which is by itself."""
    x = positive(1200, 2, 1, 64, 64, dtype, seed=5)
    x["log_decay"][:] = rate
    S0 = torch.randn(1, 2, 64, 64, device="cuda")
    S0[0, 0, 3] = value
    S0[0, 1, 7] = value
    x["log_decay"][0, 900, 1] = -INF              # head 1 forgets, head 0 does not
    check(x, state=S0, segment=segment, pieces=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [-1.0, -3.0])
@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("t", [10, 100, 130])
def test_odd_values_stay_until_a_token_forgets(dtype, rate, value, t):
    x = positive(300, 2, 1, 64, 64, dtype, seed=t)
    x["log_decay"][:] = rate
    x["log_decay"][0, 280, 1] = -INF
    check(x, [("v", (0, t, 0, 3), value), ("v", (0, t, 1, 5), value)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [0.2, 0.6])
def test_growth_over_a_piece_leaves_zero_states_zero(dtype, rate):
    """Pieces that grow past the largest number, chunks of 128 that do not."""
    x = positive(1200, 2, 1, 64, 64, dtype, seed=7)
    x["log_decay"][:] = rate
    x["v"].zero_()
    o, S = gdn.gdn_linattn_fwd(**x, segment=512)
    assert bool((o == 0).all()) and bool((S == 0).all()) and gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces_that_grow_and_fall_again(dtype):
    """Half a piece up by e^60, the other half down again: states in between are finite, and so is the rest."""
    x = positive(1024, 2, 1, 64, 64, dtype, seed=9)
    x["log_decay"][:] = -60.0 / 256
    x["log_decay"][:, :256] = x["log_decay"][:, 512:768] = 60.0 / 256
    S0 = torch.randn(1, 2, 64, 64, device="cuda")
    for segment, pieces in ((0, 1), (512, 2)):
        check(x, state=S0, segment=segment, pieces=pieces)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.125, -2.0 ** -20, 2.0 ** 20])
@pytest.mark.parametrize("rate", [-0.2, -3.0])
def test_odd_states_under_a_scale(dtype, scale, rate):
    """A scale does not take a decay that no token forgets below what fp32 holds."""
    x = positive(300, 2, 1, 64, 64, dtype, seed=3)
    x["log_decay"][:] = rate
    x["v"][0, 40, 0, 5] = INF
    S0 = torch.zeros(1, 2, 64, 64, device="cuda")
    S0[0, 0, 3] = INF
    S0[0, 1, 7] = -INF
    o, S = gdn.gdn_linattn_fwd(**x, scale=scale, state_in=S0)
    ro, _, rS, _ = walk(**x, scale=scale, state_in=S0)
    odd = ~np.isfinite(ro)
    assert np.array_equal(o.double().cpu().numpy()[odd], ro[odd]) and bool(torch.isfinite(o.cpu()[torch.from_numpy(~odd)]).all())
    assert np.array_equal(np.isfinite(S[0].cpu().numpy()), np.isfinite(rS[0])) and gdn.gdn_get_device_status() == 0
