"""Linear attention with a decay for each head, and the norms around a block,
from their definitions in fp64 on the CPU, with a bound on what the library's
arithmetic may be off (first-order rounding analysis, not fitted).

U is fp32's unit roundoff, EX the relative error of 2^x as the hardware
computes it (2 ulp).
"""
import numpy as np
import torch

from layer_reference import EX, U, entries, f64, offsets, sigmoid, silu_error, stored

CHUNK = 32           # tokens that one decay factor covers at least, but for a sequence's tail
FORGET = -126 * np.log(2)


def linattn(q, k, v, log_decay, scale, state_in, slots, cu, parts=False, steps=False, pieces=1):
    """q, k [B,T,G,dk], v [B,T,H,dv] (steps: [N,...]); returns o, its bound, the
    new states and their bounds.  ``parts``: the tensor-core kernel, where the
    decayed v enters products as three bf16 parts, P and S rounded to bf16 once."""
    H, dv = v.shape[-2:]
    G, dk = q.shape[-2:]
    cu = list(range(v.shape[0] + 1)) if steps else offsets(v, cu)
    Q, K = (np.repeat(f64(x).reshape(-1, G, dk), H // G, axis=1) for x in (q, k))
    V = f64(v).reshape(-1, H, dv)
    g = f64(log_decay)
    g = np.broadcast_to(g, (len(V), H)) if g.ndim == 1 else g.reshape(-1, H)
    o, bound, new, eb = np.zeros_like(V), np.zeros_like(V), [], []
    S0 = f64(state_in)
    # a rounding to bf16 (8 bits) is off by at most half a step, 2^-8 of the value (eps = 2^-7): three parts,
    # each the rounding of what those before it leave, leave 2^-24; P and S are rounded once, one of the two a term
    cut, half_step = (2.0 ** -24, 2.0 ** -8) if parts else (0.0, 0.0)
    for i, e in enumerate(entries(slots, len(cu) - 1)):
        S = np.zeros((H, dv, dk)) if S0 is None or not 0 <= e < len(S0) else S0[e].copy()
        m, err = np.abs(S), np.zeros_like(S)       # sum of magnitudes; error of the decays' chain so far
        reach = np.zeros(H)                        # sum of |g| over the last tokens, at most a block of 32
        for t in range(cu[i], cu[i + 1]):
            gt = g[t]
            a = np.where(gt <= FORGET, 0.0, np.exp(np.maximum(gt, FORGET)))
            fin = np.where(gt <= FORGET, 0.0, np.abs(gt))
            reach = np.abs(np.where(g[max(cu[i], t - 31):t + 1] <= FORGET, 0, g[max(cu[i], t - 31):t + 1])).sum(0)
            a3 = a[:, None, None]
            # a factor 2^x over 32 tokens and its product: EX + 4 U; the sums in its exponent 12 roundings
            rel = ((EX + 4 * U) / CHUNK + 12 * U * fin)[:, None, None]
            w, wa = V[t][:, :, None] * K[t][:, None, :], np.abs(V[t])[:, :, None] * np.abs(K[t])[:, None, :]
            err = a3 * (err + rel * m)
            S, m = (a3 * S + w, a3 * m + wa)
            # within a chunk: factors over part of a block, one rounding for each term of a sum of 128 (twice
            # where the sum need not round to nearest), the parts' cut, and the join of pieces
            inside = (2 * EX + 12 * U * reach)[:, None, None] + (2 if parts else 1) * 130 * U + cut + (pieces > 1) * 4 * U
            es = err + inside * m
            qa = np.abs(Q[t])[:, None, :]
            y = (S * Q[t][:, None, :]).sum(-1)
            ya = (m * qa).sum(-1)
            ey = (es * qa).sum(-1) + ((2 if parts else 1) * (dk + 4) * U + 1.01 * half_step) * ya
            o[t] = scale * y
            bound[t] = abs(scale) * ey + 2 * U * np.abs(o[t])
        new.append(S)
        eb.append(err + (inside if cu[i + 1] > cu[i] else 0) * m + 2 * U * m)
    return o.reshape(v.shape), stored(o, bound, v.dtype).reshape(v.shape), new, eb


def _norm(x, ex, weight, bias, eps, rms):
    """Norm of rows and its error, from the rows' error ``ex``."""
    n = x.shape[-1]
    k = (n / 32 + 8) * U    # a sum over n elements in chains of at most n / 32 + 8 additions
    mean = 0 if rms else x.mean(-1, keepdims=True)
    em = 0 if rms else k * np.abs(x).mean(-1, keepdims=True) + ex.mean(-1, keepdims=True)
    c = x - mean
    ec = ex + em + U * np.abs(c)
    var = (c * c).mean(-1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    er = 0.5 * (2 * k * var + (2 * ec * np.abs(c) + ec * ec).mean(-1, keepdims=True)) * r * r + 4 * U
    u = c * r
    eu = ec * r + np.abs(u) * (er + 2 * U)
    if weight is not None:
        u, eu = u * f64(weight), eu * np.abs(f64(weight)) + U * np.abs(u * f64(weight))
    if bias is not None:
        u = u + f64(bias)
        eu = eu + U * np.abs(u)
    return u, eu


def block_norm(y, residual, post_weight, post_bias, pre_weight, pre_bias, gate, gate_act, scale, residual_scale, eps, rms,
               post, pre):
    """Returns r, its bound, h, its bound (None without a norm before)."""
    u = f64(y)
    eu = np.zeros_like(u)
    if post:
        u, eu = _norm(u, eu, post_weight, post_bias, eps, rms)
    if scale is not None:
        u, eu = u * f64(scale), eu * np.abs(f64(scale)) + U * np.abs(u * f64(scale))
    if gate is not None:
        G = f64(gate)
        f = {"none": G, "sigmoid": sigmoid(G), "silu": G * sigmoid(G)}[gate_act]
        ef = 0 if gate_act == "none" else (8 * U + EX + 2 * U * np.abs(G)) * np.abs(f)
        u, eu = u * f, eu * np.abs(f) + np.abs(u) * ef + U * np.abs(u * f)
    rtype = y.dtype
    if residual is not None:
        res = f64(residual) * residual_scale
        rtype = residual.dtype
        u = u + res
        eu = eu + U * np.abs(res) + U * np.abs(u)
    h = eh = None
    if pre:
        h, eh = _norm(u, eu, pre_weight, pre_bias, eps, rms)
        eh = stored(h, eh, y.dtype)
    return u, stored(u, eu, rtype), h, eh
