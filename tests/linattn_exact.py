"""Linear attention token by token in fp64 on the CPU, with bounds that grow only
with what lies between two tokens, and with infinities as the definition has them.

A token whose decay is below 2^-126 forgets: what was before it does not count,
infinite or not.  Every other decay keeps an infinity or a NaN as it is.
"""
import numpy as np

from layer_reference import EX, U, entries, f64, offsets, stored
from linattn_reference import CHUNK, FORGET


def walk(q, k, v, log_decay, scale=1.0, state_in=None, slots=None, cu=None, parts=False, pieces=1):
    """Returns o, its bound, the new states and their bounds.

    ``parts``: the tensor-core kernel.  The decayed v enters as three bf16 parts (2^-24 is
    left, a half step 2^-8 each), P and the state as two (2^-16 is left); sums there need
    not round to nearest; P's factors are products of two powers whose exponents are
    rounded sums over a block of 32 (``reach``, at most 90 log 2 where they are used).
    Else fp32: a factor between two tokens is off by its exponential and by roundings of
    the sum of decays between them, which ``err`` gathers token by token.
    """
    H, dv = v.shape[-2:]
    G, dk = q.shape[-2:]
    cu = offsets(v, cu)
    Q, K = (np.repeat(f64(x).reshape(-1, G, dk), H // G, axis=1) for x in (q, k))
    V = f64(v).reshape(-1, H, dv)
    g = f64(log_decay)
    g = np.broadcast_to(g, (len(V), H)) if g.ndim == 1 else g.reshape(-1, H)
    o, bound, new, eb = np.zeros_like(V), np.zeros_like(V), [], []
    S0 = f64(state_in)
    cut, part = (2.0 ** -24, 2.0 ** -16) if parts else (0.0, 0.0)
    more = 2 if parts else 1
    with np.errstate(invalid="ignore", over="ignore"):
        for i, e in enumerate(entries(slots, len(cu) - 1)):
            S = np.zeros((H, dv, dk)) if S0 is None or not 0 <= e < len(S0) else S0[e].copy()
            m, err = np.abs(S), np.zeros_like(S)
            inside = np.zeros((H, 1, 1))
            for t in range(cu[i], cu[i + 1]):
                gone = (g[t] <= FORGET)[:, None, None]
                a = np.exp(np.where(gone[:, 0, 0], 0.0, g[t]))[:, None, None]
                fin = np.where(gone[:, 0, 0], 0.0, np.abs(g[t]))
                rel = ((EX + 4 * U) / CHUNK + 12 * U * fin)[:, None, None]
                reach = 0.0
                if parts:
                    last = g[max(cu[i], t - 31):t + 1]
                    reach = np.minimum(np.where(last <= FORGET, 0, np.abs(last)).sum(0), 90 * np.log(2))
                w = V[t][:, :, None] * K[t][:, None, :]
                wa = np.abs(V[t])[:, :, None] * np.abs(K[t])[:, None, :]
                err = np.where(gone, 0.0, a * (err + rel * m))
                S, m = np.where(gone, 0.0, a * S) + w, np.where(gone, 0.0, a * m) + wa
                inside = (2 * EX + 12 * U * reach) * np.ones((H, 1, 1)).reshape(H) if parts else np.full(H, 2 * EX)
                inside = inside[:, None, None] + more * 130 * U + cut + (pieces > 1) * 8 * U
                qa = np.abs(Q[t])[:, None, :]
                ya = (m * qa).sum(-1)
                ey = ((err + inside * m) * qa).sum(-1) + (more * (dk + 4) * U + 1.01 * part) * ya
                o[t] = scale * (S * Q[t][:, None, :]).sum(-1)
                bound[t] = abs(scale) * ey + 2 * U * np.abs(o[t])
            new.append(S)
            eb.append(err + (inside if cu[i + 1] > cu[i] else 0) * m + 2 * U * m)
        return o.reshape(v.shape), stored(o, bound, v.dtype).reshape(v.shape), new, eb


def agrees(got, ref, bound, kinds=True):
    """Where the reference is finite the error as a share of its bound; elsewhere the same
    infinity or NaN (``kinds``), or at least nothing finite.  At most 1 passes."""
    got = f64(got)
    assert got.shape == ref.shape
    fin = np.isfinite(ref)
    if kinds:
        same = (np.isnan(got) & np.isnan(ref)) | (got == ref)
        assert same[~fin].all(), "%d of %d" % ((~same[~fin]).sum(), (~fin).sum())
    else:
        assert not np.isfinite(got[~fin]).any()
    assert np.isfinite(got[fin]).all(), "%d of %d" % ((~np.isfinite(got[fin])).sum(), fin.sum())
    return float(np.max(np.abs(got[fin] - ref[fin]) / np.maximum(bound[fin], 1e-300))) if fin.any() else 0.0
