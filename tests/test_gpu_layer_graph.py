"""A decoding step of the operators around the recurrence as a CUDA graph: given
outputs and pools, captured once, replayed on new inputs and slots."""
import pytest
import torch

import test_gpu_conv as conv
import test_gpu_ssm as ssm
from test_gpu_ssm import gdn  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = ("x", "delta", "B", "C", "z")


@pytest.mark.parametrize("N", [1, 7, 300])
def test_replayed_step(gdn, N):  # noqa: F811
    C, W, pool = 256, 4, N + 3
    tokens, x, w, b, taps = [], None, None, None, None
    for t in range(3):                                # three tokens of every sequence
        x, w, b, taps = conv.draw(t, (N,), C, W, "bf16", pool=pool)
        a = ssm.draw(t, (N, 1), C, 16, pool=pool)
        slots = torch.randperm(pool, generator=torch.Generator().manual_seed(t))[:N].int().cuda()
        tokens.append(dict({k: a[k][:, 0].contiguous() for k in ROWS}, u=x, slots=slots))
    params = {k: a[k] for k in ("A", "D", "delta_bias", "delta_softplus")}

    def step(i, taps, states, ys):
        gdn.gdn_conv_step(i["u"], w, b, state_in=taps, state_out=taps, slots=i["slots"], y=ys[0])
        gdn.gdn_ssm_step(**dict({k: i[k] for k in ROWS}, x=ys[0]), **params, state_in=states, state_out=states,
                         slots=i["slots"], y=ys[1])
        gdn.gdn_group_norm(ys[1], 4, gate=i["z"], rms=True, y=ys[2])

    new = lambda: [torch.empty(N, C, dtype=torch.bfloat16, device="cuda") for _ in range(3)]  # noqa: E731
    want, pools = [], (taps.clone(), a["state_in"].clone())
    for i in tokens:
        ys = new()
        step(i, *pools, ys)
        want.append(ys)
    static, mine, out = {k: v.clone() for k, v in tokens[0].items()}, (taps.clone(), a["state_in"].clone()), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(static, *mine, out)
    assert torch.equal(mine[0], taps) and torch.equal(mine[1], a["state_in"])     # captured, not run
    for i, ys in zip(tokens, want):
        for k, v in i.items():
            static[k].copy_(v)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, ys))
    assert torch.equal(mine[0], pools[0]) and torch.equal(mine[1], pools[1])
    assert gdn.gdn_get_device_status() == 0


def test_replayed_prompt(gdn):  # noqa: F811
    """A scan in pieces and a convolution, in place, with the workspace given."""
    a = ssm.draw(5, (2, 200), 64, 16, pool=2)
    x, w, b, taps = conv.draw(5, (2, 200), 64, 4, "bf16", pool=2)
    ws = torch.empty(gdn.gdn_ssm_fwd_workspace_size(2, 200, 64, 16, segment=64), dtype=torch.uint8, device="cuda")
    ys = [torch.empty_like(x) for _ in range(2)]

    def run(taps, states):
        gdn.gdn_conv_fwd(x, w, b, state_in=taps, state_out=taps, y=ys[0])
        gdn.gdn_ssm_fwd(**dict(a, x=ys[0], state_in=states), state_out=states, y=ys[1], segment=64, workspace=ws)

    eager = (taps.clone(), a["state_in"].clone())
    run(*eager)
    want = [y.clone() for y in ys]
    mine = (taps.clone(), a["state_in"].clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*mine)
    for y in ys:
        y.zero_()
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(ys, want))
    assert torch.equal(mine[0], eager[0]) and torch.equal(mine[1], eager[1])
    assert gdn.gdn_get_device_status() == 0
