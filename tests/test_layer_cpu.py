"""Refusals of the operators around the recurrence, on the host: through the C
ABI (nothing is enqueued, a message is set) and in the Python binding, plus the
scan's workspace size (CPU only)."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from gated_delta_rule_09_gb300 import layer


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_09_gb300 import _lib, build
    build.build()
    return _lib.load()


# far apart, 1 MiB each
P = {n: (i + 1) << 20 for i, n in enumerate(
    ["x", "y", "w", "b", "si", "so", "slots", "cu", "delta", "A", "B", "C", "D", "z", "gate", "ws"])}


def conv_fwd(lib, x=P["x"], w=P["w"], b=None, si=None, slots=None, y=P["y"], so=None, B=2, T=16, C=32, W=4, ldx=32,
             ldy=32, pool=2, cu=None, act=1, dtype=1):
    return lib.gdn_conv_fwd(x, w, b, si, slots, y, so, B, T, C, W, ldx, ldy, pool, cu, act, dtype, None)


def conv_step(lib, x=P["x"], w=P["w"], b=None, si=None, slots=None, y=P["y"], so=P["so"], N=2, C=32, W=4, ldx=32,
              ldy=32, pool=2, act=1, dtype=1):
    return lib.gdn_conv_step(x, w, b, si, slots, y, so, N, C, W, ldx, ldy, pool, act, dtype, None)


def ssm_fwd(lib, x=P["x"], delta=P["delta"], A=P["A"], Bm=P["B"], Cm=P["C"], D=None, z=None, db=None, si=None,
            slots=None, y=P["y"], so=None, B=2, T=16, C=32, S=16, G=1, ld=(32, 32, 16, 16, 32, 32), pool=2, cu=None,
            sp=1, dtype=1, segment=0, ws=None, wsb=0):
    return lib.gdn_ssm_fwd(x, delta, A, Bm, Cm, D, z, db, si, slots, y, so, B, T, C, S, G, *ld, pool, cu, sp, dtype,
                           segment, ws, wsb, None)


def ssm_step(lib, x=P["x"], delta=P["delta"], A=P["A"], Bm=P["B"], Cm=P["C"], D=None, z=None, db=None, si=None,
             slots=None, y=P["y"], so=P["so"], N=2, C=32, S=16, G=1, ld=(32, 32, 16, 16, 32, 32), pool=2, sp=1, dtype=1):
    return lib.gdn_ssm_step(x, delta, A, Bm, Cm, D, z, db, si, slots, y, so, N, C, S, G, *ld, pool, sp, dtype, None)


def norm(lib, x=P["x"], gate=None, w=None, b=None, y=P["y"], rows=8, C=64, G=4, ldx=64, ldg=64, ldy=64, eps=1e-5,
         rms=0, act=0, dtype=1):
    return lib.gdn_group_norm(x, gate, w, b, y, rows, C, G, ldx, ldg, ldy, eps, rms, act, dtype, None)


BOTH_CONV = [
    (dict(dtype=7), 2), (dict(act=5), 2), (dict(W=0), 2), (dict(W=9), 2), (dict(C=0), 1),
    (dict(x=None), 1), (dict(y=None), 1), (dict(w=None), 1),
    (dict(ldx=31), 1), (dict(ldy=8), 1),                       # rows that overlap themselves
    (dict(x=P["x"] + 1), 1), (dict(w=P["w"] + 2), 1), (dict(so=P["so"] + 1), 1), (dict(slots=P["slots"] + 2), 1),
    (dict(y=P["x"]), 1), (dict(y=P["x"] + 64), 1), (dict(y=P["w"]), 1),
    (dict(so=P["x"]), 1), (dict(so=P["y"]), 1),
    (dict(si=P["si"], so=P["si"] + 64), 1),                    # pools that overlap in part
    (dict(si=P["y"]), 1), (dict(si=P["si"], pool=1), 1), (dict(si=P["si"], pool=-1, slots=P["slots"]), 1),
]


@pytest.mark.parametrize("kw,code", BOTH_CONV + [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(cu=P["cu"], B=0), 1), (dict(cu=P["cu"] + 1), 1), (dict(y=P["cu"], cu=P["cu"]), 1)])
def test_conv_fwd_refusals(lib, kw, code):
    assert conv_fwd(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


@pytest.mark.parametrize("kw,code", BOTH_CONV + [(dict(N=-1), 1), (dict(so=None), 1)])
def test_conv_step_refusals(lib, kw, code):
    assert conv_step(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


BOTH_SSM = [
    (dict(dtype=7), 2), (dict(S=129), 2), (dict(S=0), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=3), 1),
    (dict(x=None), 1), (dict(delta=None), 1), (dict(A=None), 1), (dict(Bm=None), 1), (dict(Cm=None), 1), (dict(y=None), 1),
    (dict(ld=(31, 32, 16, 16, 32, 32)), 1), (dict(ld=(32, 31, 16, 16, 32, 32)), 1), (dict(ld=(32, 32, 15, 16, 32, 32)), 1),
    (dict(ld=(32, 32, 16, 15, 32, 32)), 1), (dict(ld=(32, 32, 16, 16, 31, 32), z=P["z"]), 1),
    (dict(ld=(32, 32, 16, 16, 32, 31)), 1),
    (dict(delta=P["delta"] + 1), 1), (dict(A=P["A"] + 2), 1), (dict(so=P["so"] + 2), 1), (dict(db=P["b"] + 1), 1),
    (dict(y=P["x"]), 1), (dict(y=P["delta"] + 32), 1), (dict(y=P["z"], z=P["z"]), 1), (dict(y=P["B"]), 1), (dict(y=P["A"]), 1),
    (dict(so=P["A"]), 1), (dict(so=P["y"]), 1), (dict(so=P["D"], D=P["D"]), 1), (dict(si=P["si"], so=P["si"] + 16), 1),
    (dict(si=P["y"]), 1), (dict(si=P["si"], pool=1), 1),
]


@pytest.mark.parametrize("kw,code", BOTH_SSM + [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(cu=P["cu"], B=0), 1),
    (dict(T=256, segment=64, so=None), 1),                                  # pieces without a workspace
    (dict(T=256, segment=64, ws=P["ws"], wsb=64), 1),                       # one too small
    (dict(T=256, segment=64, ws=P["ws"] + 8, wsb=1 << 20), 1),              # misaligned
    (dict(T=256, segment=64, ws=P["x"], wsb=1 << 20), 1),                   # over an argument
    (dict(T=256, segment=64, si=P["si"], so=P["so"], ws=P["so"], wsb=1 << 20), 1)])
def test_ssm_fwd_refusals(lib, kw, code):
    assert ssm_fwd(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


@pytest.mark.parametrize("kw,code", BOTH_SSM + [(dict(N=-1), 1), (dict(so=None), 1)])
def test_ssm_step_refusals(lib, kw, code):
    assert ssm_step(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(act=2), 2), (dict(rows=-1), 1), (dict(C=0), 1), (dict(G=0), 1), (dict(G=5), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(ldx=63), 1), (dict(ldy=63), 1), (dict(gate=P["gate"], ldg=63), 1), (dict(x=P["x"] + 1), 1), (dict(w=P["w"] + 2), 1),
    (dict(y=P["x"] + 16), 1), (dict(y=P["x"], ldx=80), 1),                  # in place needs one stride
    (dict(y=P["gate"] + 2, gate=P["gate"]), 1), (dict(w=P["y"]), 1), (dict(b=P["y"] + 4), 1)])
def test_group_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


def test_nothing_to_do_is_a_no_op(lib):
    """No rows and no state to hand on: no CUDA call (this host has no GPU)."""
    assert conv_fwd(lib, B=0) == 0 and conv_fwd(lib, T=0, x=None, y=None) == 0 and conv_step(lib, N=0) == 0
    assert ssm_fwd(lib, B=0) == 0 and ssm_fwd(lib, T=0) == 0 and ssm_step(lib, N=0) == 0
    assert norm(lib, rows=0) == 0
    assert lib.gdn_last_launch_count(None) == 0


def test_workspace_size(lib):
    """Per piece a state and a sum of step sizes, each part rounded up to 16
    bytes; nothing when a sequence fits in one piece."""
    size = lib.gdn_ssm_fwd_workspace_size
    a16 = lambda v: (v + 15) // 16 * 16  # noqa: E731
    need = lambda slots, C, S: a16(slots * C * S * 4) + a16(slots * C * 4)  # noqa: E731
    assert size(2, 300, 40, 13, None, 64) == need(2 * 5, 40, 13)
    assert size(2, 300, 40, 13, None, 100) == need(2 * 3, 40, 13)      # 100 rounds up to 128
    assert size(3, 300, 40, 13, P["cu"], 64) == need(300 // 64 + 3, 40, 13)
    assert size(2, 300, 40, 13, None, 300) == 0 and size(2, 64, 40, 13, None, 64) == 0
    assert size(0, 300, 40, 13, None, 64) == 0 and size(2, 0, 40, 13, None, 64) == 0
    assert gdn.gdn_ssm_fwd_workspace_size(2, 300, 40, 13, segment=64) == need(10, 40, 13)
    assert gdn.gdn_ssm_fwd_workspace_size(3, 300, 40, 13, packed=True, segment=64) == need(7, 40, 13)


# ---- the Python binding

@pytest.fixture
def host_only(monkeypatch):
    """CPU tensors let through, no library and no streams."""
    monkeypatch.setattr(layer, "_cuda", lambda *a: None)
    monkeypatch.setattr(layer, "_handle", lambda *a: 0)
    monkeypatch.setattr(layer, "_call", lambda fn, index, *a: fn(*a))

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                if name.endswith("workspace_size"):
                    return 0
                raise RuntimeError("reached the library")
            return call

    monkeypatch.setattr(layer._lib, "load", lambda: Lib())


z = torch.zeros
bf = torch.bfloat16


def conv_args(**kw):
    return dict(dict(x=z(2, 8, 16, dtype=bf), weight=z(16, 4), bias=z(16), state_in=z(2, 3, 16, dtype=bf)), **kw)


def ssm_args(**kw):
    return dict(dict(x=z(2, 8, 16), delta=z(2, 8, 16), A=z(16, 4), B=z(2, 8, 2, 4), C=z(2, 8, 2, 4), D=z(16),
                     z=z(2, 8, 16), delta_bias=z(16), state_in=z(2, 16, 4)), **kw)


def first(v):
    return v[:, 0] if v.dim() > 2 and v.shape[:2] == (2, 8) else v


CONV_BAD = [dict(weight=z(15, 4)), dict(weight=z(16)), dict(bias=z(15)), dict(state_in=z(2, 4, 16, dtype=bf)),
            dict(state_out=z(3, 3, 16, dtype=bf)), dict(slots=z(3, dtype=torch.int32)), dict(act="gelu"),
            dict(weight=z(4, 16).t())]


@pytest.mark.parametrize("bad", CONV_BAD + [
    dict(x=z(2, 8, 32, dtype=bf)[..., ::2]), dict(x=z(2, 16, 16, dtype=bf)[:, ::3][:, :5], y=z(2, 4, 16, dtype=bf)),
    dict(y=z(2, 8, 17, dtype=bf)), dict(cu_seqlens=torch.tensor([0, 16], dtype=torch.int32)),
    dict(state_in=None, slots=z(2, dtype=torch.int32))])
def test_conv_binding_refuses(host_only, bad):
    with pytest.raises(ValueError):
        gdn.gdn_conv_fwd(**conv_args(**bad))


@pytest.mark.parametrize("bad", CONV_BAD)
def test_conv_step_binding_refuses(host_only, bad):
    a = conv_args(**bad)
    with pytest.raises(ValueError):
        gdn.gdn_conv_step(**dict(a, x=first(a["x"])))


SSM_BAD = [dict(delta=z(2, 8, 17)), dict(A=z(15, 4)), dict(A=z(16)), dict(B=z(2, 8, 2, 5)), dict(C=z(2, 8, 1, 4)),
           dict(D=z(15)), dict(delta_bias=z(17)), dict(z=z(2, 8, 15)), dict(state_in=z(2, 4, 16)),
           dict(state_out=z(1, 16, 4)), dict(slots=z(1, dtype=torch.int32)), dict(B=z(2, 8, 4, 4)[:, :, ::2])]


@pytest.mark.parametrize("bad", SSM_BAD + [dict(B=z(2, 8, 4)), dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)),
                                           dict(y=z(2, 8, 15))])
def test_ssm_binding_refuses(host_only, bad):
    with pytest.raises(ValueError):
        gdn.gdn_ssm_fwd(**ssm_args(**bad))


@pytest.mark.parametrize("bad", SSM_BAD)
def test_ssm_step_binding_refuses(host_only, bad):
    a = ssm_args(**bad)
    with pytest.raises(ValueError):
        gdn.gdn_ssm_step(**{k: first(v) if k != "state_in" and k != "state_out" else v for k, v in a.items()})


@pytest.mark.parametrize("bad", [dict(weight=z(31)), dict(bias=z(33)), dict(gate=z(3, 31)), dict(y=z(2, 32)), dict(act="relu"),
                                 dict(x=z(3, 64)[:, ::2])])
def test_group_norm_binding_refuses(host_only, bad):
    with pytest.raises(ValueError):
        gdn.gdn_group_norm(**dict(dict(x=z(3, 32), groups=4), **bad))


@pytest.mark.parametrize("bad", [dict(x=z(2, 8, 16, dtype=torch.float16)), dict(bias=z(16, dtype=bf)),
                                 dict(state_in=z(2, 3, 16))])
def test_types_are_refused(host_only, bad):
    with pytest.raises(TypeError):
        gdn.gdn_conv_fwd(**conv_args(**bad))


def test_right_arguments_reach_the_library(host_only):
    a, s = conv_args(), ssm_args()
    calls = [(gdn.gdn_conv_fwd, a), (gdn.gdn_conv_fwd, dict(a, x=z(2, 8, 40, dtype=bf)[..., 5:21])),
             (gdn.gdn_conv_step, dict(a, x=first(a["x"]))), (gdn.gdn_ssm_fwd, s),
             (gdn.gdn_ssm_step, {k: first(v) if k != "state_in" else v for k, v in s.items()}),
             (gdn.gdn_group_norm, dict(x=z(3, 5, 32), groups=4, gate=z(3, 5, 64)[..., 32:]))]
    for fn, kw in calls:
        with pytest.raises(RuntimeError, match="reached the library"):
            fn(**kw)


def test_cpu_tensors_are_refused():
    with pytest.raises(TypeError):
        gdn.gdn_conv_fwd(**conv_args())
    with pytest.raises(TypeError):
        gdn.gdn_ssm_fwd(**ssm_args())
    with pytest.raises(TypeError):
        gdn.gdn_group_norm(z(3, 32), 4)
