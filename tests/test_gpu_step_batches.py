"""Single tokens of batches large enough that a thread takes several sequences
(``gdn_conv_step`` from 384 blocks on, 1024 for single elements; ``gdn_ssm_step``
from 512), against the definition in fp64 and the same rows in small batches."""
import numpy as np
import pytest
import torch

import layer_reference as R
import test_gpu_conv as conv
import test_gpu_ssm as ssm
from test_gpu_ssm import gdn  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = ("x", "delta", "B", "C", "z")


def some_slots(n, seed):
    """Permuted entries of a pool five larger; every seventh sequence has none."""
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(n + 5, generator=g)[:n].int()
    slots[3::7] = -1
    return slots.cuda()


def off_alignment(t):
    """The same values one element further than an aligned start."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    return flat.copy_(t.flatten()).view(t.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,ch,S,G,extra", [(513, 128, 16, 1, 0), (514, 128, 13, 2, 5), (515, 128, 6, 1, 0), (1025, 130, 8, 1, 64),
                                            (131, 127, 40, 1, 3), (131, 128, 32, 4, 0), (130, 100, 128, 1, 0), (601, 513, 3, 9, 0)])
def test_ssm_step(gdn, N, ch, S, G, extra, dtype):  # noqa: F811
    a = ssm.draw(N + S, (N, 1), ch, S, G, dtype, pool=N + 5, extra=extra)
    slots = some_slots(N, S)
    y0, bound, new, eb = ssm.reference(a, slots)
    b = {k: (v[:, 0] if k in ROWS else v) for k, v in a.items()}
    keep = a["state_in"].clone()
    for state in (a["state_in"], off_alignment(keep)):
        out = torch.full_like(keep, 7)
        y, _ = gdn.gdn_ssm_step(**dict(b, state_in=state), state_out=out, slots=slots)
        assert gdn.gdn_last_launch_count() == (1, 7) and gdn.gdn_get_device_status() == 0
        assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1
        used = set()
        for i, e in enumerate(slots.tolist()):
            if e >= 0:
                assert R.inside(out[e], new[i], eb[i]) <= 1, i
                used.add(e)
        rest = sorted(set(range(N + 5)) - used)
        assert (out[rest] == 7).all() and torch.equal(state, keep)
        pool = state.clone() if state is a["state_in"] else off_alignment(keep)
        y2, same = gdn.gdn_ssm_step(**dict(b, state_in=pool), slots=slots)      # in place
        assert same is pool and torch.equal(y2, y)
        assert torch.equal(pool[sorted(used)], out[sorted(used)]) and torch.equal(pool[rest], keep[rest])
    some = torch.full_like(keep, 7)
    for lo in range(0, N, 25):
        part = {k: (v[lo:lo + 25] if k in ROWS else v) for k, v in b.items()}
        y, _ = gdn.gdn_ssm_step(**part, state_out=some, slots=slots[lo:lo + 25].contiguous())
        assert R.inside(y, y0[lo:lo + 25, 0], bound[lo:lo + 25, 0]) <= 1
    assert torch.equal(some, out)
    y, s = gdn.gdn_ssm_step(**dict(b, state_in=None, z=None, D=None))           # no slots, no states yet
    y0, bound, new, eb = ssm.reference(dict(a, state_in=None, z=None, D=None))
    assert R.inside(y, y0[:, 0], bound[:, 0]) <= 1 and R.inside(s, np.stack(new), np.stack(eb)) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,C,W,extra", [(387, 64, 4, 0), (389, 512, 4, 64), (390, 40, 8, 0), (386, 66, 3, 2), (1027, 63, 4, 0),
                                         (1029, 7, 2, 1), (515, 261, 5, 0), (1025, 24, 1, 0)])
def test_conv_step(gdn, N, C, W, extra, dtype):  # noqa: F811
    x, w, b, s = conv.draw(N + C, (N,), C, W, dtype, extra=extra, pool=N + 5)
    slots = some_slots(N, C)
    ref, bound, new = R.conv(x[:, None], w, b, s, slots, None, "silu")
    y, out = gdn.gdn_conv_step(x, w, b, state_in=s, state_out=torch.full_like(s, 7), slots=slots)
    assert gdn.gdn_last_launch_count() == (1, 6) and gdn.gdn_get_device_status() == 0
    assert R.inside(y, ref[:, 0], bound[:, 0]) <= 1
    used = sorted(e for e in slots.tolist() if e >= 0)
    rest = sorted(set(range(N + 5)) - set(used))
    if W > 1:
        want = torch.full_like(s, 7)
        for i, e in enumerate(slots.tolist()):
            if e >= 0:
                want[e] = torch.as_tensor(new[i])
        assert torch.equal(out, want)
        pool = s.clone()
        y2, same = gdn.gdn_conv_step(x, w, b, state_in=pool, slots=slots)       # in place
        assert same is pool and torch.equal(y2, y)
        assert torch.equal(pool[used], want[used]) and torch.equal(pool[rest], s[rest])
        pool = off_alignment(s)
        y2, _ = gdn.gdn_conv_step(x, w, b, state_in=pool, slots=slots)
        assert R.inside(y2, ref[:, 0], bound[:, 0]) <= 1 and torch.equal(pool[used], want[used])
    some = torch.full_like(s, 7)
    for lo in range(0, N, 25):
        part, _ = gdn.gdn_conv_step(x[lo:lo + 25], w, b, state_in=s, state_out=some, slots=slots[lo:lo + 25].contiguous())
        assert torch.equal(part, y[lo:lo + 25])
    assert torch.equal(some, out)
    y, out = gdn.gdn_conv_step(x, w, None, act="none")                          # no slots, no states yet
    ref, bound, new = R.conv(x[:, None], w, None, None, None, None, "none")
    assert R.inside(y, ref[:, 0], bound[:, 0]) <= 1 and np.array_equal(R.f64(out), np.stack(new))


def test_a_slot_past_the_pool_leaves_its_neighbours(gdn):  # noqa: F811
    """One bad slot among the sequences of a thread: that sequence runs without a state."""
    N = 515
    a = ssm.draw(4, (N, 1), 128, 16, pool=N)
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(4)).int().cuda()
    bad, none = slots.clone(), slots.clone()
    bad[::6] = N
    none[::6] = -1
    b = {k: (v[:, 0] if k in ROWS else v) for k, v in a.items()}
    pools = [a["state_in"].clone() for _ in range(2)]
    got = [gdn.gdn_ssm_step(**dict(b, state_in=p), slots=s)[0] for p, s in zip(pools, (bad, none))]
    assert gdn.gdn_get_device_status() == 0x10
    assert torch.equal(got[0], got[1]) and torch.equal(pools[0], pools[1])
    x, w, bias, s = conv.draw(5, (N,), 96, 4, "bf16", pool=N)
    pools = [s.clone() for _ in range(2)]
    got = [gdn.gdn_conv_step(x, w, bias, state_in=p, slots=t)[0] for p, t in zip(pools, (bad, none))]
    assert gdn.gdn_get_device_status() == 0x10
    assert torch.equal(got[0], got[1]) and torch.equal(pools[0], pools[1])
