"""Infinite inputs, states that overflow and decays of -inf: scan and step give
what the recurrence gives, infinity where it has one and NaN only where it has NaN."""
import numpy as np
import pytest
import torch

import layer_reference as R
from test_gpu_ssm import draw, gdn, reference  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]
ROWS = ("x", "delta", "B", "C", "z")
SIZES = [1, 3, 13, 16, 20, 32, 50, 64, 100, 128]
inf = float("inf")


def same(got, ref, bound):
    """Equal NaN and infinities; the rest within the bound."""
    got = R.f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    wild = np.isinf(got) | np.isinf(ref)
    assert np.array_equal(got[wild], ref[wild])
    ok = ~(wild | np.isnan(ref))
    assert (np.abs(got[ok] - ref[ok]) <= bound[ok]).all()


def both(gdn, a, segment=0):  # noqa: F811
    """The scan, then the same tokens one by one, against the definition."""
    T = a["x"].shape[1]
    y0, bound, new, eb = reference(a, pieces=1 if segment == 0 else -(-T // 64))
    y, s = gdn.gdn_ssm_fwd(**a, segment=segment or T)
    same(y, y0, bound)
    same(s, np.stack(new), np.stack(eb))
    y0, bound, new, eb = reference(a)
    s, ys = a["state_in"], []
    for t in range(T):
        y, s = gdn.gdn_ssm_step(**dict({k: (v[:, t] if k in ROWS and v is not None else v) for k, v in a.items()}, state_in=s))
        ys.append(y)
    same(torch.stack(ys, 1), y0, bound)
    same(s, np.stack(new), np.stack(eb))
    assert gdn.gdn_get_device_status() == 0


def positive(a):
    """All terms of y positive, so that an infinite one makes y infinite."""
    a.update({k: a[k].abs() + 0.5 for k in ("x", "B", "C")}, z=None)
    if a["state_in"] is not None:
        a["state_in"] = a["state_in"].abs()
    return a


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", SIZES)
def test_infinite_state(gdn, S, dtype):  # noqa: F811
    a = positive(draw(S, (2, 37), 40, S, dtype=dtype, pool=2))
    a["state_in"][0, 3] = inf
    a["state_in"][1, 7, S - 1] = inf
    both(gdn, a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", SIZES)
def test_infinite_input(gdn, S, dtype):  # noqa: F811
    """x = inf; also one whose products with B are infinities of both signs."""
    a = positive(draw(S, (2, 37), 40, S, dtype=dtype, pool=2))
    a["x"][0, 5, 3] = inf
    a["x"][1, 18, 7] = -inf
    a["x"][1, 20, 8] = inf
    both(gdn, a)
    a["B"][1, 20] *= torch.where(torch.arange(S, device="cuda") % 2 == 0, 1, -1).to(a["B"].dtype)
    both(gdn, a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", SIZES)
def test_infinite_c(gdn, S, dtype):  # noqa: F811
    a = positive(draw(S, (2, 37), 40, S, dtype=dtype, pool=2))
    a["state_in"][0, 4] = 2                             # exact in few bits: nothing left of it after rounding
    a["C"][0, 0, 0, 0] = inf
    a["C"][0, 33, 0, S - 1] = inf
    a["C"][1, 9, 0, S // 2] = -inf
    both(gdn, a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [16, 33])
def test_overflowing_state(gdn, T, dtype):  # noqa: F811
    """States that grow by e^10 a token pass the largest number and stay infinite."""
    a = positive(draw(T, (1, T), 24, 16, dtype=dtype, pool=1))
    a.update(A=torch.ones_like(a["A"]), delta=torch.full_like(a["delta"], 10), delta_bias=None, delta_softplus=False, D=None)
    ref, _, new, _ = reference(a)
    y, s = gdn.gdn_ssm_fwd(**a)
    top = float(torch.finfo(torch.float32).max)
    assert (ref > 10 * top).any() and (ref < top / 10).any()
    assert (R.f64(y)[ref > 10 * top] == np.inf).all() and np.isfinite(R.f64(y)[ref < top / 10]).all()
    assert (s == inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 16, 17, 40, 250])
@pytest.mark.parametrize("S,ch", [(1, 40), (13, 40), (16, 64), (16, 43), (32, 40), (100, 40), (128, 64)])
def test_a_state_that_forgets_at_once(gdn, S, ch, T, dtype):  # noqa: F811
    """A = -inf: the state is the last token's d B x, whatever the length.  A decay
    below the smallest number is the same, which the reference can take."""
    a = draw(S + T, (2, T), ch, S, dtype=dtype, pool=2)
    a["A"][:, S // 2] = -1e30
    a["A"][5] = -1e30
    ref = reference(a)
    a["A"] = torch.where(a["A"] == -1e30, -inf, a["A"])
    for segment in (T, 64):
        y, s = gdn.gdn_ssm_fwd(**a, segment=segment)
        y0, bound, new, eb = ref if segment == T else reference(dict(a, A=a["A"].clamp(min=-1e30)), pieces=4)
        same(y, y0, bound)
        same(s, np.stack(new), np.stack(eb))
    b = {k: (v[:, 0] if k in ROWS else v) for k, v in a.items()}
    y, _ = gdn.gdn_ssm_step(**b)
    same(y, ref[0][:, 0], ref[1][:, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_step_with_infinite_rate(gdn, dtype):  # noqa: F811
    """A = -inf and a step size of zero: the state stays as it is, in scan and step."""
    a = draw(9, (1, 20), 40, 16, dtype=dtype, pool=1)
    a.update(delta_softplus=False, delta_bias=None, delta=torch.zeros_like(a["delta"]), A=torch.full_like(a["A"], -inf))
    _, s = gdn.gdn_ssm_fwd(**a)
    assert torch.equal(s, a["state_in"])
    _, s = gdn.gdn_ssm_step(**{k: (v[:, 0] if k in ROWS else v) for k, v in a.items()})
    assert torch.equal(s, a["state_in"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_input_without_skip(gdn, dtype):  # noqa: F811
    """Without D there is no skip term to make NaN of an infinite x."""
    a = positive(draw(3, (1, 20), 40, 4, dtype=dtype, pool=1))
    a.update(D=None)
    clean, _ = gdn.gdn_ssm_fwd(**a)
    a["x"][0, 5, 3] = inf
    clean[0, 5:, 3] = inf
    y, s = gdn.gdn_ssm_fwd(**a)
    assert torch.equal(y, clean) and (s[0, 3] == inf).all()
    one = {k: (v[:, 5] if k in ROWS and v is not None else v) for k, v in a.items()}
    y, _ = gdn.gdn_ssm_step(**one)
    assert y[0, 3] == inf and torch.isfinite(torch.cat([y[0, :3], y[0, 4:]])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 13, 16, 50, 128])
def test_infinite_state_over_pieces(gdn, S, dtype):  # noqa: F811
    """Infinite however far a piece's decay is below the smallest number."""
    a = positive(draw(S, (1, 300), 40, S, dtype=dtype, pool=1))
    a["delta_bias"] += 2                                # 64 tokens decay by e^-1000 and more
    a["state_in"][0, 3] = inf
    a["x"][0, 40, 5] = inf
    both(gdn, a, segment=64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growth_over_pieces(gdn, dtype):  # noqa: F811
    """Pieces that multiply by more than the largest number: zero stays zero, and a
    small state becomes what it becomes token by token."""
    a = draw(6, (1, 300), 40, 16, dtype=dtype, pool=1)
    a.update(A=torch.ones_like(a["A"]), delta=torch.zeros_like(a["delta"]), delta_bias=None, delta_softplus=False, D=None,
             z=None, x=torch.zeros_like(a["x"]))
    a["delta"][:, 64:128] = 1.5                         # e^96 over the second piece
    a["delta"][:, 200:210] = -1
    a["state_in"] *= 1e-30
    a["state_in"][:, 7] = 0
    y0, bound, new, eb = reference(a, pieces=5)
    y, s = gdn.gdn_ssm_fwd(**a, segment=64)
    same(y, y0, bound)
    same(s, np.stack(new), np.stack(eb))
    assert (s[0, 7] == 0).all() and torch.isfinite(s).all()
    a["delta"][:, 64:128] = 10                          # and by e^640
    a["state_in"].zero_()
    y, s = gdn.gdn_ssm_fwd(**a, segment=64)
    assert (y == 0).all() and (s == 0).all()
