"""Refusals of linear attention and of the norms around a block, on the host:
through the C ABI (nothing is enqueued, a message is set) and in the Python
binding, plus the workspace size (CPU only)."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from test_layer_cpu import host_only, lib  # noqa: F401

# far apart, 16 MiB each
P = {n: (i + 1) << 24 for i, n in enumerate(
    ["q", "k", "v", "g", "o", "si", "so", "slots", "cu", "ws", "y", "r", "ro", "h", "gate", "w", "b", "s"])}
LD = (64, 64, 128, 4, 128)


def fwd(lib, q=P["q"], k=P["k"], v=P["v"], g=P["g"], si=None, slots=None, o=P["o"], so=None, B=2, T=16, H=4, G=2, dk=32,
        dv=32, ld=LD, pool=2, cu=None, scale=1.0, dtype=1, segment=0, ws=None, wsb=0):
    return lib.gdn_linattn_fwd(q, k, v, g, si, slots, o, so, B, T, H, G, dk, dv, *ld, pool, cu, scale, dtype, segment, ws,
                               wsb, None)


def step(lib, q=P["q"], k=P["k"], v=P["v"], g=P["g"], si=None, slots=None, o=P["o"], so=P["so"], N=2, H=4, G=2, dk=32,
         dv=32, ld=LD, pool=2, scale=1.0, dtype=1):
    return lib.gdn_linattn_step(q, k, v, g, si, slots, o, so, N, H, G, dk, dv, *ld, pool, scale, dtype, None)


def norm(lib, y=P["y"], r=P["r"], gate=None, pw=None, pb=None, s=None, qw=None, qb=None, ro=P["ro"], h=P["h"], rows=8, C=64,
         ld=(64, 64, 64, 64, 64), rs=1.0, eps=1e-5, rms=1, post=1, act=2, dtype=1, rtype=1):
    return lib.gdn_block_norm(y, r, gate, pw, pb, s, qw, qb, ro, h, rows, C, *ld, rs, eps, rms, post, act, dtype, rtype, None)


def with_ld(i, v):
    return LD[:i] + (v,) + LD[i + 1:]


BOTH = [
    (dict(dtype=7), 2), (dict(dk=129), 2), (dict(dk=0), 1), (dict(dv=0), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(G=3), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(o=None), 1),
    (dict(ld=with_ld(0, 63)), 1), (dict(ld=with_ld(1, 63)), 1), (dict(ld=with_ld(2, 127)), 1), (dict(ld=with_ld(3, 3)), 1),
    (dict(ld=with_ld(4, 127)), 1), (dict(ld=with_ld(0, -64)), 1),
    (dict(q=P["q"] + 1), 1), (dict(g=P["g"] + 2), 1), (dict(si=P["si"] + 2, so=P["so"]), 1), (dict(slots=P["slots"] + 1), 1),
    (dict(o=P["q"]), 1), (dict(o=P["v"] + 64), 1), (dict(o=P["g"]), 1), (dict(so=P["v"]), 1), (dict(so=P["o"]), 1),
    (dict(si=P["si"], so=P["si"] + 64), 1), (dict(si=P["o"], so=P["so"]), 1), (dict(si=P["si"], so=P["so"], pool=1), 1),
    (dict(si=P["si"], so=P["so"], pool=-1, slots=P["slots"]), 1),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(B=-1), 1), (dict(T=-1), 1), (dict(cu=P["cu"], B=0), 1), (dict(cu=P["cu"] + 1), 1), (dict(o=P["cu"], cu=P["cu"]), 1),
    (dict(T=512, segment=128), 1),                                          # pieces without a workspace
    (dict(T=512, segment=128, ws=P["ws"], wsb=64), 1),                      # one too small
    (dict(T=512, segment=128, ws=P["ws"] + 8, wsb=1 << 24), 1),             # misaligned
    (dict(T=512, segment=128, ws=P["k"], wsb=1 << 24), 1),                  # over an argument
    (dict(T=512, segment=128, si=P["si"], so=P["so"], ws=P["si"], wsb=1 << 24), 1),
    (dict(T=512, segment=128, o=P["ws"] + 4096, ws=P["ws"], wsb=1 << 24), 1)])
def test_prompt_refusals(lib, kw, code):  # noqa: F811
    assert fwd(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


@pytest.mark.parametrize("kw,code", BOTH + [(dict(N=-1), 1), (dict(so=None), 1)])
def test_step_refusals(lib, kw, code):  # noqa: F811
    assert step(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


TOP = 2 ** 31 - 2 ** 16


def test_sizes_past_32_bits_are_refused(lib):  # noqa: F811
    far = dict(q=1 << 50, k=1 << 51, v=1 << 52, g=1 << 53, o=1 << 54, H=1, G=1, dk=1, dv=1, ld=(1, 1, 1, 1, 1))
    for cu in (None, P["cu"]):
        assert fwd(lib, B=1, T=TOP + 1, cu=cu, **far) == 2
    assert fwd(lib, B=TOP + 1, T=0) == 2 and step(lib, N=TOP + 1, so=1 << 55, **far) == 2
    wide = dict(far, H=1 << 16, dv=1 << 16, ld=(1, 1, 1 << 33, 1 << 16, 1 << 33))
    assert fwd(lib, B=1, T=1, **wide) == 2 and step(lib, N=1, so=1 << 55, **wide) == 2
    many = dict(far, H=1 << 10, dv=1 << 10, ld=(1, 1, 1 << 20, 1 << 10, 1 << 20))
    assert fwd(lib, B=1 << 20, T=1, **many) == 2                 # more than 2^31 blocks


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(dtype=0, rtype=1), 2), (dict(rtype=5), 2), (dict(act=3), 2), (dict(act=-1), 2), (dict(rows=-1), 1),
    (dict(C=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(y=None), 1), (dict(ro=None), 1),
    (dict(ld=(63, 64, 64, 64, 64)), 1), (dict(ld=(64, 63, 64, 64, 64)), 1), (dict(ld=(64, 64, 63, 64, 64), gate=P["gate"]), 1),
    (dict(ld=(64, 64, 64, 63, 64)), 1), (dict(ld=(64, 64, 64, 64, 63)), 1),
    (dict(y=P["y"] + 1), 1), (dict(rtype=0, r=P["r"] + 2), 1), (dict(pw=P["w"] + 2), 1), (dict(s=P["s"] + 1), 1),
    (dict(post=0, pw=P["w"]), 1), (dict(post=0, pb=P["b"]), 1), (dict(h=None, qw=P["w"]), 1), (dict(h=None, qb=P["b"]), 1),
    (dict(h=P["ro"]), 1), (dict(ro=P["y"] + 16), 1), (dict(h=P["r"] + 2), 1), (dict(pw=P["ro"]), 1), (dict(qb=P["h"]), 1),
    (dict(ro=P["r"], ld=(64, 64, 64, 80, 64)), 1),                          # in place needs one stride
    (dict(ro=P["y"], rtype=0), 1), (dict(h=P["r"], rtype=0), 1)])           # and one type
def test_block_norm_refusals(lib, kw, code):  # noqa: F811
    assert norm(lib, **kw) == code, lib.gdn_get_last_error()
    assert lib.gdn_get_last_error()


def test_nothing_to_do_is_a_no_op(lib):  # noqa: F811
    """No rows and no state to hand on: no CUDA call (this host has no GPU)."""
    assert fwd(lib, B=0) == 0 and fwd(lib, T=0, q=None, v=None) == 0 and step(lib, N=0) == 0 and norm(lib, rows=0) == 0
    assert lib.gdn_last_launch_count(None) == 0


def test_workspace_size(lib):  # noqa: F811
    """Per piece a state and a decay for each head, each part rounded up to 16
    bytes; nothing when a sequence fits in one piece."""
    size = lib.gdn_linattn_fwd_workspace_size
    a16 = lambda v: (v + 15) // 16 * 16  # noqa: E731
    need = lambda slots, H, dk, dv: a16(slots * H * dk * dv * 4) + a16(slots * H * 4)  # noqa: E731
    for tc in (-1, 0, 1):
        assert size(2, 300, 3, 13, 5, None, 128, tc) == need(2 * 3, 3, 13, 5)
        assert size(2, 300, 3, 13, 5, None, 100, tc) == need(2 * 3, 3, 13, 5)     # 100 rounds up to 128
        assert size(3, 300, 3, 13, 5, P["cu"], 128, tc) == need(300 // 128 + 3, 3, 13, 5)
        assert size(2, 300, 3, 13, 5, None, 300, tc) == 0 and size(2, 128, 3, 13, 5, None, 128, tc) == 0
        assert size(0, 300, 3, 13, 5, None, 128, tc) == 0 and size(2, 0, 3, 13, 5, None, 128, tc) == 0
    for args in ((1, 131072, 8, 128, 128), (4, 4096, 16, 128, 128), (3, 517, 6, 77, 45), (1, 1, 1, 1, 1)):
        for cu in (None, P["cu"]):
            both = [size(*args, cu, 0, tc) for tc in (0, 1)]
            assert size(*args, cu, 0, -1) == max(both)
    assert size(1, 131072, 8, 128, 128, None, 0, 1) > 0 and size(4, 4096, 16, 128, 128, None, 0, 1) == 0
    assert gdn.gdn_linattn_fwd_workspace_size(2, 300, 3, 13, 5, segment=128) == need(6, 3, 13, 5)


# ---- the Python binding
z = torch.zeros
bf = torch.bfloat16


def lin_args(**kw):
    return dict(dict(q=z(2, 8, 2, 16), k=z(2, 8, 2, 16), v=z(2, 8, 4, 12), log_decay=z(2, 8, 4), state_in=z(2, 4, 12, 16)), **kw)


def first(v):
    return v[:, 0] if v.dim() > 2 and v.shape[:2] == (2, 8) else v


BAD = [dict(q=z(2, 8, 2, 15)), dict(k=z(2, 8, 2, 17)), dict(k=z(2, 8, 1, 16)), dict(q=z(2, 8, 4)), dict(log_decay=z(3)),
       dict(log_decay=z(2, 8, 3)), dict(state_in=z(2, 4, 16, 12)), dict(state_out=z(1, 4, 12, 16)),
       dict(slots=z(1, dtype=torch.int32)), dict(o=z(2, 8, 4, 13)), dict(q=z(2, 8, 2, 32)[..., ::2]),
       dict(k=z(2, 8, 4, 16)[:, :, ::2]), dict(v=z(2, 8, 4, 24)[..., ::2])]


@pytest.mark.parametrize("bad", BAD + [dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)), dict(q=z(2, 7, 2, 16)),
                                       dict(state_in=None, slots=z(2, dtype=torch.int32)), dict(v=z(8, 4, 12))])
def test_prompt_binding_refuses(host_only, bad):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.gdn_linattn_fwd(**lin_args(**bad))


@pytest.mark.parametrize("bad", BAD)
def test_step_binding_refuses(host_only, bad):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.gdn_linattn_step(**{k: v if k.startswith("state") else first(v) for k, v in lin_args(**bad).items()})


NORM = dict(y=z(3, 32), residual=z(3, 32))


@pytest.mark.parametrize("bad", [
    dict(residual=z(3, 31)), dict(gate=z(2, 32)), dict(post_weight=z(31)), dict(pre_bias=z(33)), dict(scale=z(1, 32)),
    dict(gate_act="tanh"), dict(post=False, post_weight=z(32)), dict(pre=False, pre_bias=z(32)), dict(pre=False, h=z(3, 32)),
    dict(residual_out=z(2, 32)), dict(h=z(3, 33)), dict(y=z(3, 64)[:, ::2]), dict(residual=z(3, 64)[:, ::2]),
    dict(scale=z(64)[::2])])
def test_block_norm_binding_refuses(host_only, bad):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.gdn_block_norm(**dict(NORM, **bad))


@pytest.mark.parametrize("fn,kw", [
    (gdn.gdn_linattn_fwd, lin_args(v=z(2, 8, 4, 12, dtype=torch.float16))), (gdn.gdn_linattn_fwd, lin_args(q=z(2, 8, 2, 16, dtype=bf))),
    (gdn.gdn_linattn_fwd, lin_args(log_decay=z(4, dtype=bf))), (gdn.gdn_linattn_fwd, lin_args(log_decay=0.5)),
    (gdn.gdn_linattn_fwd, lin_args(state_in=z(2, 4, 12, 16, dtype=bf))),
    (gdn.gdn_linattn_fwd, lin_args(segment=128, workspace=z(64))),
    (gdn.gdn_block_norm, dict(NORM, y=z(3, 32, dtype=torch.float16))), (gdn.gdn_block_norm, dict(NORM, residual=z(3, 32, dtype=bf))),
    (gdn.gdn_block_norm, dict(NORM, gate=z(3, 32, dtype=bf))), (gdn.gdn_block_norm, dict(NORM, scale=z(32, dtype=bf))),
    (gdn.gdn_block_norm, dict(NORM, residual_out=z(3, 32, dtype=bf)))])
def test_types_are_refused(host_only, fn, kw):  # noqa: F811
    with pytest.raises(TypeError):
        fn(**kw)


@pytest.mark.parametrize("workspace", [torch.zeros(1 << 16, 2, dtype=torch.uint8)[:, 0],
                                       torch.zeros(1, dtype=torch.uint8).expand(1 << 16)])
def test_strided_workspace_is_refused(host_only, workspace):  # noqa: F811
    with pytest.raises(ValueError):
        gdn.gdn_linattn_fwd(**lin_args(), segment=128, workspace=workspace)


def test_right_arguments_reach_the_library(host_only):  # noqa: F811
    a = lin_args()
    p = z(2, 8, 2 * 32 + 48 + 5)[..., 5:]
    sliced = dict(a, q=p[..., :32].unflatten(-1, (2, 16)), k=p[..., 32:64].unflatten(-1, (2, 16)), v=p[..., 64:].unflatten(-1, (4, 12)))
    calls = [(gdn.gdn_linattn_fwd, a), (gdn.gdn_linattn_fwd, sliced), (gdn.gdn_linattn_fwd, dict(a, log_decay=z(4))),
             (gdn.gdn_linattn_fwd, dict(a, log_decay=z(2, 8, 9)[..., 3:7])),
             (gdn.gdn_linattn_step, {k: v if k == "state_in" else first(v) for k, v in sliced.items()}),
             (gdn.gdn_block_norm, NORM), (gdn.gdn_block_norm, dict(y=z(2, 3, 32, dtype=bf), residual=z(2, 3, 32))),
             (gdn.gdn_block_norm, dict(y=z(3, 32), gate=z(3, 64)[:, 32:], scale=z(32), pre=False))]
    for fn, kw in calls:
        with pytest.raises(RuntimeError, match="reached the library"):
            fn(**kw)


def test_cpu_tensors_are_refused():
    with pytest.raises(TypeError):
        gdn.gdn_linattn_fwd(**lin_args())
    with pytest.raises(TypeError):
        gdn.gdn_block_norm(**NORM)
