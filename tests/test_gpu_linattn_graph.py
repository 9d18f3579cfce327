"""Linear attention and the norms around a block as a serving loop runs them:
captured once and replayed on new inputs, on another stream, two calls at once,
and states far into a large pool."""
import pytest
import torch

import gated_delta_rule_09_gb300 as gdn
from layer_reference import inside
from linattn_reference import linattn
from test_gpu_linattn import make

pytestmark = pytest.mark.gpu


def test_replayed_step():
    """Three tokens of every sequence: norm before, attention, residual sum and norm, in given buffers."""
    N, H, D, pool = 6, 4, 64, 9
    g = torch.Generator("cuda").manual_seed(0)
    w = 1 + 0.1 * torch.randn(H * D, generator=g, device="cuda")
    tokens = [dict(make((N,), H, 2, D, D, "bf16", seed=t),
                   slots=torch.randperm(pool, generator=torch.Generator().manual_seed(t))[:N].int().cuda(),
                   stream=torch.randn(N, H * D, generator=g, device="cuda").bfloat16()) for t in range(3)]
    start = torch.randn(pool, H, D, D, generator=g, device="cuda")

    def run(i, states, out):
        gdn.gdn_linattn_step(i["q"], i["k"], i["v"], i["log_decay"], state_in=states, state_out=states, slots=i["slots"],
                             o=out[0])
        gdn.gdn_block_norm(out[0].flatten(1), i["stream"], post_weight=w, pre_weight=w, residual_out=out[1], h=out[2])

    new = lambda: [torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")] + [  # noqa: E731
        torch.empty(N, H * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    states, want = start.clone(), []
    for i in tokens:
        out = new()
        run(i, states, out)
        want.append(out)
    static, mine, out = {k: v.clone() for k, v in tokens[0].items()}, start.clone(), new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(static, mine, out)
    assert torch.equal(mine, start)                                        # captured, not run
    for i, expect in zip(tokens, want):
        for k, v in i.items():
            static[k].copy_(v)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, expect))
    assert torch.equal(mine, states) and gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("segment", [0, 128])
def test_replayed_prompt(dtype, segment):
    x = make((2, 400), 2, 1, 64, 64, dtype, seed=1)
    S = torch.randn(2, 2, 64, 64, device="cuda")
    need = gdn.gdn_linattn_fwd_workspace_size(2, 400, 2, 64, 64, segment=segment)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    o, mine = torch.empty_like(x["v"].contiguous()), S.clone()
    want, final = gdn.gdn_linattn_fwd(**x, state_in=S, segment=segment)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_linattn_fwd(**x, state_in=mine, state_out=mine, o=o, segment=segment, workspace=ws)
    graph.replay()
    assert torch.equal(o, want) and torch.equal(mine, final)
    graph.replay()                                                         # goes on from the states it left
    again, last = gdn.gdn_linattn_fwd(**x, state_in=final, segment=segment)
    assert torch.equal(o, again) and torch.equal(mine, last) and gdn.gdn_get_device_status() == 0


def test_two_calls_at_once():
    """On two streams, each with its own workspace; then the same inputs one after the other."""
    xs = [make((1, 3000), 4, 4, 128, 64, "bf16", seed=s) for s in range(2)]
    want = [gdn.gdn_linattn_fwd(**x, segment=512) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(3):
        got = [gdn.gdn_linattn_fwd(**x, segment=512, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for (o, S), (p, R) in zip(got, want):
        assert torch.equal(o, p) and torch.equal(S, R)
    assert gdn.gdn_get_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_call_gives_the_same_bits(dtype):
    x = make((3, 700), 2, 2, 128, 128, dtype, seed=4)
    first = gdn.gdn_linattn_fwd(**x)
    for _ in range(5):
        o, S = gdn.gdn_linattn_fwd(**x)
        assert torch.equal(o, first[0]) and torch.equal(S, first[1])


def test_states_past_32_bits():
    """A pool of more than 2^31 numbers, its last entries in use."""
    H, D, pool = 16, 128, 8200                        # 2.15e9 numbers, 8.6 GB
    S = torch.empty(pool, H, D, D, device="cuda")
    slots = torch.tensor([pool - 1, 0], dtype=torch.int32, device="cuda")
    S[[pool - 1, 0]] = torch.randn(2, H, D, D, device="cuda")
    small = S[[pool - 1, 0]].clone()
    x = make((2, 130), H, 2, D, D, "bf16", seed=6)
    for segment in (0, 128):
        a, _ = gdn.gdn_linattn_fwd(**x, state_in=S, slots=slots, segment=segment)
        b, small = gdn.gdn_linattn_fwd(**x, state_in=small, segment=segment)
        assert torch.equal(a, b) and torch.equal(S[[pool - 1, 0]], small)
    one = {n: t[:, 0].contiguous() for n, t in x.items()}
    a, _ = gdn.gdn_linattn_step(**one, state_in=S, slots=slots)
    b, small = gdn.gdn_linattn_step(**one, state_in=small)
    assert torch.equal(a, b) and torch.equal(S[[pool - 1, 0]], small)
    assert gdn.gdn_get_device_status() == 0


def test_many_chunks_at_full_load():
    """More blocks than multiprocessors, 32 chunks each, again and again."""
    x = make((5, 4096), 16, 16, 128, 128, "bf16", seed=8, rate=1.0)
    o, S = gdn.gdn_linattn_fwd(**x)
    for _ in range(20):
        p, R = gdn.gdn_linattn_fwd(**x)
        assert torch.equal(o, p) and torch.equal(S, R)
    for n, h in ((0, 0), (3, 7), (4, 15)):
        one = {k: t[n:n + 1, :600, h:h + 1].contiguous() for k, t in x.items()}
        ro, bo, _, _ = linattn(**one, scale=1.0, state_in=None, slots=None, cu=None, parts=True)
        assert inside(o[n:n + 1, :600, h:h + 1], ro, bo) <= 1
    assert gdn.gdn_get_device_status() == 0
