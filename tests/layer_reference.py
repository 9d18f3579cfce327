"""The operators around the recurrence from their definitions, in fp64 on the
CPU, with a running bound on what fp32 arithmetic may be off.

Every function takes the tensors a test passed to the library (any device) and
returns (results, bounds).  The bounds are first-order rounding analysis, not
fitted: U is fp32's unit roundoff, EX the relative error of 2^x as the hardware
computes it (2 ulp), and a bf16 output adds half an ulp of the stored value.
"""
import numpy as np
import torch

from parity_util import half_ulp_bf16

U = 2.0 ** -24
EX = 2.0 ** -22


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def silu(v):
    return v * sigmoid(v)


def silu_error(v):
    """fp32 v / (1 + e^-v): the exponent's rounding grows with |v|."""
    return np.abs(silu(v)) * (8 * U + EX + 2 * U * np.abs(v))


def stored(ref, bound, dtype):
    """The bound after one rounding to the output type."""
    half_ulp = half_ulp_bf16(np.abs(ref) + bound) if dtype == torch.bfloat16 else U * (np.abs(ref) + bound)
    return bound + half_ulp + 1e-37


def offsets(x, cu):
    if cu is None:
        B, T = x.shape[:2]
        return [i * T for i in range(B + 1)]
    return [int(c) for c in cu.cpu()]


def entries(slots, n):
    return list(range(n)) if slots is None else [int(s) for s in slots.cpu()]


def conv(x, weight, bias, state_in, slots, cu, act):
    """x [B,T,C]; returns y, its bound, and the new state per sequence (exact)."""
    W = weight.shape[1]
    cu = offsets(x, cu)
    X, w, b = f64(x).reshape(-1, x.shape[-1]), f64(weight), f64(bias)
    y, bound, new = np.zeros_like(X), np.zeros_like(X), []
    S = f64(state_in)
    ent = entries(slots, len(cu) - 1)
    for i, e in enumerate(ent):
        keep = np.zeros((W - 1, X.shape[1])) if S is None or not 0 <= e < len(S) else S[e]
        seq = np.concatenate([keep, X[cu[i]:cu[i + 1]]])
        for t in range(cu[i + 1] - cu[i]):
            terms = seq[t:t + W].T * w
            v, m = terms.sum(1), np.abs(terms).sum(1)
            if b is not None:
                v, m = v + b, m + np.abs(b)
            off = (W + 1) * U * m
            y[cu[i] + t] = silu(v) if act == "silu" else v
            bound[cu[i] + t] = 1.1 * off + silu_error(v) if act == "silu" else off
        new.append(seq[len(seq) - (W - 1):])
    return y.reshape(x.shape), stored(y, bound, x.dtype).reshape(x.shape), new


def ssm(x, delta, A, B, C, D, z, delta_bias, softplus, state_in, slots, cu, pieces=1):
    """x [b,T,ch]; returns y, its bound, new states and their bounds."""
    ch, S = A.shape
    G = B.shape[-2]
    cu = offsets(x, cu)
    X, Z = f64(x).reshape(-1, ch), None if z is None else f64(z).reshape(-1, ch)
    raw, A = f64(delta).reshape(-1, ch), f64(A)
    Bm, Cm = f64(B).reshape(-1, G, S), f64(C).reshape(-1, G, S)
    if delta_bias is not None:
        raw = raw + f64(delta_bias)
    d = np.logaddexp(raw, 0) if softplus else raw
    ed = (8 * U + EX + 4 * U * np.abs(raw)) if softplus else np.full_like(raw, 2 * U)   # relative, of d
    skip = np.zeros(ch) if D is None else f64(D)
    rep = lambda m: np.repeat(m, ch // G, axis=0)  # noqa: E731
    # h enters C h with 11 significant bits in bf16 calls; in fp32 calls h and C in two such
    # parts each, which leaves less than 2^-22 of either
    cut = 2.0 ** -10 if x.dtype == torch.bfloat16 else 2.0 ** -21
    y, bound, new, eb = np.zeros_like(X), np.zeros_like(X), [], []
    P = f64(state_in)
    for i, e in enumerate(entries(slots, len(cu) - 1)):
        h = np.zeros((ch, S)) if P is None or not 0 <= e < len(P) else P[e].copy()
        m, err = np.abs(h), np.zeros((ch, S))       # sum of magnitudes, error so far
        for t in range(cu[i], cu[i + 1]):
            ex = d[t][:, None] * A
            a = np.exp(ex)
            w = (d[t] * X[t])[:, None] * rep(Bm[t])
            ea = EX + np.abs(ex) * (ed[t][:, None] + 4 * U)
            err = a * err + a * m * (ea + 2 * U) + np.abs(w) * (ed[t][:, None] + 4 * U)
            h, m = a * h + w, a * m + np.abs(w)
            c = rep(Cm[t])
            # a piece's start state is decayed by exp(A sum d): the rounding of sums of up
            # to 64 + 64 terms, times |v| e^-|v| <= 0.37, for each earlier piece
            extra = (0.37 * 128 + 8) * U * m * (pieces - 1)
            v = (c * h).sum(1) + skip * X[t]
            # C h on the tensor cores: operands cut to what tf32 keeps, sums in fp32 that need
            # not round to nearest
            ev = (np.abs(c) * (err + extra + cut * np.abs(h) + (S + 8) * 2 * U * m)).sum(1)
            ev = ev + 2 * U * np.abs(skip * X[t])
            if Z is not None:
                g = silu(Z[t])
                ev = (ev + 2 * U * np.abs(v)) * np.abs(g) + np.abs(v) * silu_error(Z[t])
                v = v * g
            y[t], bound[t] = v, ev + U * np.abs(v)
        new.append(h)
        eb.append(err + (0.37 * 128 + 8) * U * m * (pieces - 1) + 2 * U * m)
    return y.reshape(x.shape), stored(y, bound, x.dtype).reshape(x.shape), new, eb


def norm(x, groups, weight, bias, gate, eps, rms, act):
    X = f64(x)
    rows = X.reshape(-1, groups, X.shape[-1] // groups)
    n = rows.shape[-1]
    mean = 0 if rms else rows.mean(-1, keepdims=True)
    c = rows - mean
    var = (c * c).mean(-1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    # a sum over n elements in chains of at most n / 32 + 8 additions, 32 lanes wide or wider
    k = (n / 32 + 8) * U
    emean = 0 if rms else k * np.abs(rows).mean(-1, keepdims=True) + U * np.abs(rows)
    u = c * r
    # relative error of r: half that of var + eps, whose own error is 2 k var + the mean's square and cross terms
    er = 0.5 * (2 * k * var + (2 * emean * np.abs(c)).mean(-1, keepdims=True)
                + (emean ** 2 * np.ones_like(c)).mean(-1, keepdims=True)) * r * r + 4 * U
    off = emean * r + np.abs(u) * (er + 2 * U)
    u, off = u.reshape(X.shape), off.reshape(X.shape)
    if weight is not None:
        off = off * np.abs(f64(weight)) + U * np.abs(u * f64(weight))
        u = u * f64(weight)
    if bias is not None:
        u = u + f64(bias)
        off = off + U * np.abs(u)
    if act == "silu":
        off = 1.1 * off + silu_error(u)
        u = silu(u)
    if gate is not None:
        g = silu(f64(gate))
        off = (off + 2 * U * np.abs(u)) * np.abs(g) + np.abs(u) * silu_error(f64(gate))
        u = u * g
    return u, stored(u, off, x.dtype)


def inside(got, ref, bound):
    """Largest error as a share of its bound (<= 1 passes); NaNs must agree."""
    got = f64(got)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    if not ok.any():
        return 0.0
    d = np.abs(got[ok] - ref[ok])
    return float(np.max(d / np.maximum(bound[ok], 1e-300)))
