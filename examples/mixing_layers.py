"""Two sequence-mixing layers on the package's entry points, as a server runs
them: a packed prompt of several sequences first, then token by token with the
states kept in pools, and the same tokens as one longer prompt to compare with.

  gated delta rule   convolution of q | k | v -> gdn_chunk_fwd / gdn_decode_step
                     -> group norm of the heads, gated
  selective scan     convolution -> gdn_ssm_fwd / gdn_ssm_step (gated)
                     -> group norm of the heads

    python examples/mixing_layers.py [--tokens 200] [--steps 8]
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_09_gb300 as gdn  # noqa: E402

WIDTH, HEADS, DIM, TAPS, STATES = 256, 4, 64, 4, 16
INNER = HEADS * DIM


class Weights:
    """Random parameters: projections in bf16, the small ones in fp32."""

    def __init__(self, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self._g = g
        self.delta_in = self._proj(WIDTH, 4 * INNER + 2 * HEADS)        # q | k | v | gate | alpha | beta
        self.delta_conv = self._normal(3 * INNER, TAPS) / TAPS ** 0.5
        self.delta_norm = 1 + 0.1 * self._normal(INNER)
        self.scan_in = self._proj(WIDTH, 2 * INNER)                     # x | z
        self.scan_conv = self._normal(INNER, TAPS) / TAPS ** 0.5
        self.scan_bias = 0.1 * self._normal(INNER)
        self.scan_bcd = self._proj(INNER, INNER + 2 * STATES)           # delta | B | C
        self.A = -torch.arange(1, STATES + 1, device="cuda").float().repeat(INNER, 1)
        self.D = torch.ones(INNER, device="cuda")
        step = torch.exp(torch.empty(INNER, device="cuda").uniform_(-6.9, -2.3, generator=g))
        self.delta_bias = step + torch.log(-torch.expm1(-step))
        self.scan_norm = 1 + 0.1 * self._normal(INNER)

    def _normal(self, *shape):
        return torch.randn(*shape, generator=self._g, device="cuda")

    def _proj(self, n, m):
        return (self._normal(n, m) / n ** 0.5).bfloat16()


class Pools:
    """What is kept between calls: one entry per request slot."""

    def __init__(self, slots):
        z = lambda *s, dt=torch.float32: torch.zeros(*s, device="cuda", dtype=dt)  # noqa: E731
        self.delta_conv = z(slots, TAPS - 1, 3 * INNER, dt=torch.bfloat16)
        self.delta = z(slots, HEADS, DIM, DIM)
        self.scan_conv = z(slots, TAPS - 1, INNER, dt=torch.bfloat16)
        self.scan = z(slots, INNER, STATES)


def _delta_inputs(p, conv):
    """q, k, v per head (unit keys and queries), decay and write strength."""
    q, k, v = (t.unflatten(-1, (HEADS, DIM)) for t in conv.split(INNER, -1))
    unit = lambda t: F.normalize(t.float(), dim=-1).to(t.dtype)  # noqa: E731
    alpha, beta = p[..., 4 * INNER:].float().split(HEADS, -1)
    return unit(q), unit(k), v.contiguous(), (-0.1 * F.softplus(alpha)).contiguous(), torch.sigmoid(beta)


def delta_prompt(w, pools, u, slots, cu):
    p = u @ w.delta_in
    conv, _ = gdn.gdn_conv_fwd(p[..., :3 * INNER], w.delta_conv, state_in=pools.delta_conv, slots=slots, cu_seqlens=cu)
    q, k, v, la, be = _delta_inputs(p, conv)
    o, S = gdn.gdn_chunk_fwd(q, k, v, la, be, S0=pools.delta[slots.long()], cu_seqlens=cu)
    pools.delta[slots.long()] = S
    return gdn.gdn_group_norm(o.flatten(-2), HEADS, w.delta_norm, gate=p[..., 3 * INNER:4 * INNER], rms=True)


def delta_step(w, pools, u, slots):
    p = u @ w.delta_in
    conv, _ = gdn.gdn_conv_step(p[:, :3 * INNER], w.delta_conv, state_in=pools.delta_conv, slots=slots)
    q, k, v, la, be = _delta_inputs(p, conv)
    o, S = gdn.gdn_decode_step(q, k, v, la, be.contiguous(), S_in=pools.delta[slots.long()])
    pools.delta[slots.long()] = S
    return gdn.gdn_group_norm(o.flatten(-2), HEADS, w.delta_norm, gate=p[:, 3 * INNER:4 * INNER], rms=True)


def _scan_inputs(w, x):
    p = x @ w.scan_bcd
    delta, B, C = p.split((INNER, STATES, STATES), -1)
    return dict(x=x, delta=delta, A=w.A, B=B.unsqueeze(-2), C=C.unsqueeze(-2), D=w.D, delta_bias=w.delta_bias,
                delta_softplus=True)


def scan_prompt(w, pools, u, slots, cu):
    p = u @ w.scan_in
    x, _ = gdn.gdn_conv_fwd(p[..., :INNER], w.scan_conv, w.scan_bias, state_in=pools.scan_conv, slots=slots,
                            cu_seqlens=cu)
    y, _ = gdn.gdn_ssm_fwd(**_scan_inputs(w, x), z=p[..., INNER:], state_in=pools.scan, slots=slots, cu_seqlens=cu)
    return gdn.gdn_group_norm(y, HEADS, w.scan_norm, y=y)


def scan_step(w, pools, u, slots):
    p = u @ w.scan_in
    x, _ = gdn.gdn_conv_step(p[:, :INNER], w.scan_conv, w.scan_bias, state_in=pools.scan_conv, slots=slots)
    y, _ = gdn.gdn_ssm_step(**_scan_inputs(w, x), z=p[:, INNER:], state_in=pools.scan, slots=slots)
    return gdn.gdn_group_norm(y, HEADS, w.scan_norm, y=y)


LAYERS = {"gated delta rule": (delta_prompt, delta_step), "selective scan": (scan_prompt, scan_step)}


def _pack(seqs):
    lengths = [len(s) for s in seqs]
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")
    return torch.cat(seqs)[None], cu


def run(tokens=200, steps=8, seed=0):
    """{layer: (outputs of prompt then steps, outputs of the whole as prompts)}, per sequence."""
    g = torch.Generator("cuda").manual_seed(seed)
    w = Weights(seed)
    lengths = [tokens, max(1, tokens // 3), 1]
    seqs = [torch.randn(n + steps, WIDTH, generator=g, device="cuda").bfloat16() for n in lengths]
    slots = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
    got = {}
    for name, (prompt, step) in LAYERS.items():
        pools = Pools(5)
        u, cu = _pack([s[:n] for s, n in zip(seqs, lengths)])
        parts = [[t] for t in prompt(w, pools, u, slots, cu)[0].split(lengths)]
        for t in range(steps):
            y = step(w, pools, torch.stack([s[n + t] for s, n in zip(seqs, lengths)]), slots)
            for i, p in enumerate(parts):
                p.append(y[i:i + 1])
        u, cu = _pack(seqs)
        whole = prompt(w, Pools(5), u, slots, cu)[0].split([n + steps for n in lengths])
        got[name] = ([torch.cat(p) for p in parts], list(whole))
    return got


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    for name, (steps, whole) in run(a.tokens, a.steps).items():
        worst = max(float((s - t).float().norm() / t.float().norm()) for s, t in zip(steps, whole))
        print("%-16s prompt then %d steps against one prompt: relative difference %.1e (bf16 keeps 4e-3)"
              % (name, a.steps, worst))
    flags = gdn.gdn_get_device_status()
    print("device status %#x" % flags)
    return int(flags != 0)


if __name__ == "__main__":
    sys.exit(main())
