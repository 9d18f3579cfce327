"""Work of the sequence-mixing layer around the recurrence, as timed passes.

Five operators, each in its plain form (elementary torch operations in 32 bits)
and through the package's entry points:

  conv       short causal depthwise convolution over a prompt (gdn_conv_fwd)
  conv_step  the same for one new token per sequence (gdn_conv_step)
  ssm        selective state space scan over a prompt (gdn_ssm_fwd)
  ssm_step   the same for one new token per sequence (gdn_ssm_step)
  norm       group norm of a token's heads, channels last, with an
             activation or a gate (gdn_group_norm)

A case holds sizes only; prepare() draws everything else from the seed.  Rows
of x, z, B, C are slices of wider rows, as a projection writes them.  States
live in pools addressed by slot numbers where a case has "slots".  A step reads
its state from one pool and writes it to a second one, so that a pass can be
repeated on the same inputs; a decoding loop passes one pool for both.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STATE_UPDATES = 27610 * 4096 * 16       # largest scan: tokens x channels x states
CONV_ELEMENTS = 4 * 4096 * 6144         # largest convolution: tokens x channels


def listed():
    return [
        # q, k and v of 16 heads of 128 ahead of the chunked pass, four training-length prompts
        dict(name="conv_prompt", op="conv", seqs=4, tokens=16384, packed=False, channels=6144, width=4,
             bias=False, state=False, slots=False, extra=2048, dtype="bf16"),
        # ragged pack in fp32 with an odd channel count, continued from kept states
        dict(name="conv_ragged", op="conv", seqs=8, tokens=27610, packed=True, channels=1023, width=3,
             bias=True, state=True, slots=True, extra=0, dtype="f32"),
        # one token of each of 256 sequences being decoded
        dict(name="conv_step_batch", op="conv_step", seqs=256, channels=6144, width=4, bias=False, slots=True,
             extra=2048, dtype="bf16"),
        # one sequence being decoded: latency
        dict(name="conv_step_one", op="conv_step", seqs=1, channels=2048, width=4, bias=True, slots=False,
             extra=0, dtype="bf16"),
        # four training-length prompts
        dict(name="ssm_prompt", op="ssm", seqs=4, tokens=16384, packed=False, channels=2048, states=16, groups=1,
             state=False, slots=False, gate=True, dtype="bf16"),
        # eight prompts of unequal length in one pack, continued from kept states
        dict(name="ssm_packed", op="ssm", seqs=8, tokens=27610, packed=True, channels=4096, states=16, groups=1,
             state=True, slots=True, gate=True, dtype="bf16"),
        # one very long document
        dict(name="ssm_long", op="ssm", seqs=1, tokens=131072, packed=False, channels=1024, states=16, groups=1,
             state=False, slots=False, gate=True, dtype="bf16"),
        # short fp32 prompts with nothing a multiple of anything
        dict(name="ssm_odd", op="ssm", seqs=3, tokens=3 * 517, packed=False, channels=203, states=13, groups=7,
             state=True, slots=False, gate=False, dtype="f32"),
        # one token of each of 256 sequences being decoded
        dict(name="ssm_step_batch", op="ssm_step", seqs=256, channels=4096, states=16, groups=1, slots=True,
             gate=True, dtype="bf16"),
        # one sequence being decoded: latency
        dict(name="ssm_step_one", op="ssm_step", seqs=1, channels=2048, states=16, groups=1, slots=False,
             gate=True, dtype="bf16"),
        # heads of 128 normed and gated after a prompt's scan
        dict(name="norm_prompt", op="norm", rows=16384, channels=2048, groups=16, rms=False, affine=True,
             gate=True, act="none", dtype="bf16"),
        # a decoding batch with heads of an odd width
        dict(name="norm_odd", op="norm", rows=256, channels=1925, groups=7, rms=True, affine=True, gate=False,
             act="silu", dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("conv", "conv_step", "ssm", "ssm", "ssm_step", "norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    even = flag()                      # half of the channel counts are multiples of 64, as heads are

    def channels(lo, hi):
        c = _log(rng, lo, hi)
        return max(64, c // 64 * 64) if even else c

    if op == "conv":
        C = channels(1, 8192)
        seqs = _log(rng, 1, 64)
        packed = flag()
        tokens = max(1, min(_log(rng, 1, 65536), CONV_ELEMENTS // C))
        tokens = tokens if packed else max(1, tokens // seqs) * seqs
        return dict(op=op, seqs=seqs, tokens=tokens, packed=packed, channels=C, width=rng.choice((2, 3, 4, 4)),
                    bias=flag(), state=flag(), slots=flag(), extra=rng.choice((0, 0, 64, 5)), dtype=dtype)
    if op == "conv_step":
        return dict(op=op, seqs=_log(rng, 1, 1024), channels=channels(1, 8192), width=rng.choice((2, 3, 4, 4)),
                    bias=flag(), slots=flag(), extra=rng.choice((0, 0, 64, 5)), dtype=dtype)
    if op == "ssm":
        C = channels(1, 8192)
        states = rng.choice((16, 16, 16, _log(rng, 1, 128)))
        seqs = _log(rng, 1, 32)
        packed = flag()
        tokens = max(1, min(_log(rng, 1, 131072), STATE_UPDATES // (C * states)))
        tokens = tokens if packed else max(1, tokens // seqs) * seqs
        return dict(op=op, seqs=seqs, tokens=tokens, packed=packed, channels=C, states=states,
                    groups=rng.choice([g for g in (1, 1, 2, 4, 7) if C % g == 0]), state=flag(), slots=flag(),
                    gate=flag(), dtype=dtype)
    if op == "ssm_step":
        C = channels(1, 8192)
        states = rng.choice((16, 16, 16, _log(rng, 1, 128)))
        seqs = max(1, min(_log(rng, 1, 1024), (1 << 26) // (C * states)))
        return dict(op=op, seqs=seqs, channels=C, states=states,
                    groups=rng.choice([g for g in (1, 1, 2, 4, 7) if C % g == 0]), slots=flag(), gate=flag(),
                    dtype=dtype)
    groups = rng.choice((1, 2, 7, 16, 32))
    width = rng.choice((64, 128, 256, _log(rng, 1, 8192 // groups)))
    rows = max(1, min(_log(rng, 1, 65536), CONV_ELEMENTS // (groups * width)))
    return dict(op=op, rows=rows, channels=groups * width, groups=groups, rms=flag(), affine=flag(), gate=flag(),
                act=rng.choice(("none", "silu")), dtype=dtype)


def _offsets(case, seed):
    """Where each sequence begins and ends; a pack of four or more has an empty sequence and one of one token."""
    n, tokens = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [i * (tokens // n) for i in range(n + 1)]
    r = random.Random(seed * 7919 + 13)
    cuts = sorted(r.randint(0, tokens) for _ in range(n - 1))
    cu = [0] + cuts + [tokens]
    if n >= 4:
        cu[1] = cu[0]
        cu[2] = min(cu[1] + 1, cu[3])
    return cu


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    st = dict(case=case)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev) * scale

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def wide(rows, width, extra, scale=1.0):
        """A [rows, width] slice of rows that are `extra` wider, from their end."""
        full = torch.randn(rows, width + extra, generator=g, device=dev, dtype=dt)
        return (full.mul_(scale) if scale != 1.0 else full)[:, extra:]

    if op == "norm":
        R, C = case["rows"], case["channels"]
        st["x"] = wide(R, C, 0) + normal(R, 1).to(dt)
        st["gate"] = wide(R, C, 0) if case["gate"] else None
        st["weight"] = 1 + normal(C, scale=0.1) if case["affine"] else None
        st["bias"] = normal(C, scale=0.1) if case["affine"] and not case["rms"] else None
        return st

    n, C = case["seqs"], case["channels"]
    if op in ("conv", "ssm"):
        cu = _offsets(case, seed)
        st["longest"] = max(b - a for a, b in zip(cu, cu[1:]))
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        rows = case["tokens"]
        lead = (1, rows) if case["packed"] else (n, rows // n)
    else:
        rows, lead = n, (n,)
    st["lead"] = lead
    pool = n + n // 8 + 1 if case["slots"] else n
    st["slots"] = torch.randperm(pool, generator=g, device=dev)[:n].int() if case["slots"] else None

    if op in ("conv", "conv_step"):
        W = case["width"]
        st["x"] = wide(rows, C, case["extra"]).unflatten(0, lead)
        st["weight"] = (uniform(C, W) * 2 - 1) / math.sqrt(W)
        st["bias"] = normal(C, scale=0.1) if case["bias"] else None
        has = op == "conv_step" or case["state"]
        st["state_in"] = torch.randn(pool, W - 1, C, generator=g, device=dev, dtype=dt) if has else None
        st["state_out"] = torch.zeros(pool, W - 1, C, device=dev, dtype=dt)
        return st

    S, G = case["states"], case["groups"]
    x = wide(rows, C, 0)
    st["x"] = (x * torch.sigmoid(x)).unflatten(0, lead)          # what the convolution hands on
    st["delta"] = wide(rows, C, 0, 0.5).unflatten(0, lead)       # raw step sizes; softplus(delta + bias) ~ 1e-3 .. 1e-1
    step = torch.exp(uniform(C) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    st["delta_bias"] = step + torch.log(-torch.expm1(-step))
    st["A"] = -torch.arange(1, S + 1, device=dev, dtype=torch.float32) * torch.exp(normal(C, S, scale=0.1))
    bc = wide(rows, 2 * G * S, 64)
    st["B"] = bc[:, :G * S].unflatten(1, (G, S)).unflatten(0, lead)
    st["C"] = bc[:, G * S:].unflatten(1, (G, S)).unflatten(0, lead)
    st["D"] = 1 + normal(C, scale=0.1)
    st["z"] = wide(rows, C, C).unflatten(0, lead) if case["gate"] else None
    has = op == "ssm_step" or case["state"]
    st["state_in"] = normal(pool, C, S) if has else None
    st["state_out"] = torch.zeros(pool, C, S, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return OWN[op](st)
    return PLAIN[op](st)


def _own_conv(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_conv_fwd(st["x"], st["weight"], st["bias"], state_in=st["state_in"], state_out=st["state_out"],
                            slots=st["slots"], cu_seqlens=st["cu"] if st["case"]["packed"] else None, act="silu")


def _own_conv_step(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_conv_step(st["x"], st["weight"], st["bias"], state_in=st["state_in"], state_out=st["state_out"],
                             slots=st["slots"], act="silu")


def _own_ssm(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_ssm_fwd(st["x"], st["delta"], st["A"], st["B"], st["C"], D=st["D"], z=st["z"],
                           delta_bias=st["delta_bias"], delta_softplus=True, state_in=st["state_in"],
                           state_out=st["state_out"], slots=st["slots"],
                           cu_seqlens=st["cu"] if st["case"]["packed"] else None)


def _own_ssm_step(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_ssm_step(st["x"], st["delta"], st["A"], st["B"], st["C"], D=st["D"], z=st["z"],
                            delta_bias=st["delta_bias"], delta_softplus=True, state_in=st["state_in"],
                            state_out=st["state_out"], slots=st["slots"])


def _own_norm(st):
    import gated_delta_rule_09_gb300 as gdn
    c = st["case"]
    return gdn.gdn_group_norm(st["x"], c["groups"], weight=st["weight"], bias=st["bias"], gate=st["gate"],
                              eps=1e-5, rms=c["rms"], act=c["act"])


def _keep(st, new):
    """Write the sequences' new states to their places in the output pool."""
    if st["slots"] is None:
        st["state_out"].copy_(new)
    else:
        st["state_out"].index_copy_(0, st["slots"].long(), new.to(st["state_out"].dtype))
    return st["state_out"]


def _kept(st):
    """The sequences' states before the call, in 32 bits."""
    if st["state_in"] is None:
        n = st["case"]["seqs"]
        return torch.zeros(n, *st["state_out"].shape[1:], device=st["state_out"].device)
    return (st["state_in"] if st["slots"] is None else st["state_in"][st["slots"].long()]).float()


def _silu(v):
    return v * torch.sigmoid(v)


def _plain_conv(st):
    W = st["case"]["width"]
    x = st["x"].flatten(0, 1)
    R, C = x.shape
    cu = st["cu"].long()
    n = cu.numel() - 1
    # the sequences one after another, each with its W - 1 kept inputs ahead of it
    row = torch.arange(R, device=x.device)
    at = row + torch.searchsorted(cu[1:], row, right=True) * (W - 1)
    ahead = (cu[:-1] + torch.arange(n, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    ext = torch.empty(R + n * (W - 1), C, device=x.device)
    ext[at + W - 1] = x.float()
    ext[ahead.flatten()] = _kept(st).flatten(0, 1)
    y = sum(ext[at + j] * st["weight"][:, j] for j in range(W))
    if st["bias"] is not None:
        y = y + st["bias"]
    y = _silu(y)
    last = (cu[1:] + torch.arange(n, device=x.device) * (W - 1))[:, None] + torch.arange(W - 1, device=x.device)
    return y.to(x.dtype).unflatten(0, st["lead"]), _keep(st, ext[last])


def _plain_conv_step(st):
    x, kept = st["x"].float(), _kept(st)
    ext = torch.cat([kept, x[:, None]], 1)
    y = (ext * st["weight"].t()).sum(1)
    if st["bias"] is not None:
        y = y + st["bias"]
    return _silu(y).to(st["x"].dtype), _keep(st, ext[:, 1:])


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _ssm_out(st, h, x, Cm, z):
    """C h + D x, gated: h [R, C, S], x [R, C], Cm [R, G, S]."""
    G = Cm.shape[1]
    y = (h.unflatten(1, (G, -1)) * Cm.float()[:, :, None]).sum(-1).flatten(1) + st["D"] * x
    return y if z is None else y * _silu(z.float())


def _plain_ssm(st):
    x = st["x"].flatten(0, 1).float()
    Bm, Cm = st["B"].flatten(0, 1).float(), st["C"].flatten(0, 1)
    G = Bm.shape[1]
    d = _softplus(st["delta"].flatten(0, 1).float() + st["delta_bias"])
    a = torch.exp(d[:, :, None] * st["A"])
    b = ((d * x).unflatten(1, (G, -1))[..., None] * Bm[:, :, None]).flatten(1, 2)
    R = x.shape[0]
    cu = st["cu"].long()
    some = (cu[1:] > cu[:-1]).float()
    start = cu[:-1].clamp(max=R - 1)
    h0 = _kept(st)
    b.index_add_(0, start, a[start] * h0 * some[:, None, None])   # the kept state enters at the first token
    is_start = torch.zeros(R, device=x.device).index_add_(0, start, some)
    a.mul_((1 - is_start)[:, None, None])
    off = 1                                                       # h = a h + b, spans doubled until they cover a sequence
    while off < st["longest"]:
        b = torch.cat([b[:off], torch.addcmul(b[off:], a[off:], b[:-off])])
        if 2 * off < st["longest"]:
            a = torch.cat([a[:off], a[off:] * a[:-off]])
        off *= 2
    del a
    y = _ssm_out(st, b, x, Cm, None if st["z"] is None else st["z"].flatten(0, 1))
    final = torch.where(some[:, None, None] > 0, b[(cu[1:] - 1).clamp(min=0)], h0)
    return y.to(st["x"].dtype).unflatten(0, st["lead"]), _keep(st, final)


def _plain_ssm_step(st):
    x = st["x"].float()
    G = st["B"].shape[1]
    d = _softplus(st["delta"].float() + st["delta_bias"])
    b = ((d * x).unflatten(1, (G, -1))[..., None] * st["B"].float()[:, :, None]).flatten(1, 2)
    h = torch.exp(d[:, :, None] * st["A"]) * _kept(st) + b
    return _ssm_out(st, h, x, st["C"], st["z"]).to(st["x"].dtype), _keep(st, h)


def _plain_norm(st):
    c = st["case"]
    x = st["x"].float().unflatten(1, (c["groups"], -1))
    if not c["rms"]:
        x = x - x.mean(-1, keepdim=True)
    y = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)).flatten(1)
    if st["weight"] is not None:
        y = y * st["weight"]
    if st["bias"] is not None:
        y = y + st["bias"]
    if c["act"] == "silu":
        y = _silu(y)
    if st["gate"] is not None:
        y = y * _silu(st["gate"].float())
    return y.to(st["x"].dtype)


OWN = dict(conv=_own_conv, conv_step=_own_conv_step, ssm=_own_ssm, ssm_step=_own_ssm_step, norm=_own_norm)
PLAIN = dict(conv=_plain_conv, conv_step=_plain_conv_step, ssm=_plain_ssm, ssm_step=_plain_ssm_step,
             norm=_plain_norm)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, C = case["op"], case["channels"]
    if op == "norm":
        n = case["rows"] * C
        return {"bytes": n * e * (3 if case["gate"] else 2) + 8 * C * case["affine"],
                "flops": n * (8 + 4 * case["gate"])}
    seqs = case["seqs"]
    if op in ("conv", "conv_step"):
        W = case["width"]
        rows = case["tokens"] if op == "conv" else seqs
        states = 2 if op == "conv_step" or case["state"] else 1
        return {"bytes": 2 * rows * C * e + 4 * C * (W + case["bias"]) + states * seqs * (W - 1) * C * e,
                "flops": rows * C * (2 * W + 4)}
    S, G = case["states"], case["groups"]
    rows = case["tokens"] if op == "ssm" else seqs
    states = 2 if op == "ssm_step" or case["state"] else 1
    return {"bytes": rows * e * ((3 + case["gate"]) * C + 2 * G * S) + states * seqs * C * S * 4 + 4 * C * (S + 2),
            "flops": rows * C * (7 * S + 12)}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _place(st, new, keep_dtype):
    """The output pool after the call, with the sequences' new states in place."""
    pool = torch.zeros_like(st["state_out"], dtype=torch.float64)
    slots = range(len(new)) if st["slots"] is None else st["slots"].tolist()
    for i, s in enumerate(slots):
        pool[s] = new[i].to(keep_dtype).double() if keep_dtype is not None else new[i]
    return pool


def _before(st, i, shape):
    if st["state_in"] is None:
        return torch.zeros(shape, dtype=torch.float64, device=st["x"].device)
    return st["state_in"][i if st["slots"] is None else int(st["slots"][i])].double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    sigmoid = lambda v: 1 / (1 + torch.exp(-v))  # noqa: E731
    if op == "norm":
        x = st["x"].double().reshape(case["rows"], case["groups"], -1)
        if case["rms"]:
            y = x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / x.shape[-1] + 1e-5)
        else:
            var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
            y = (x - mean) / torch.sqrt(var + 1e-5)
        y = y.reshape(case["rows"], -1)
        y = y * st["weight"].double() if st["weight"] is not None else y
        y = y + st["bias"].double() if st["bias"] is not None else y
        y = y * sigmoid(y) if case["act"] == "silu" else y
        if st["gate"] is not None:
            gate = st["gate"].double()
            y = y * gate * sigmoid(gate)
        return y
    n, C = case["seqs"], case["channels"]
    steps = op.endswith("_step")
    x = st["x"] if steps else st["x"].flatten(0, 1)
    cu = list(range(n + 1)) if steps else st["cu"].tolist()
    if op.startswith("conv"):
        W = case["width"]
        w = st["weight"].double()
        ys, new = [], []
        for i in range(n):
            seq = torch.cat([_before(st, i, (W - 1, C)), x[cu[i]:cu[i + 1]].double()])
            if cu[i + 1] > cu[i]:
                y = torch.einsum("tcw,cw->tc", seq.unfold(0, W, 1), w)
                y = y + st["bias"].double() if st["bias"] is not None else y
                ys.append(y * sigmoid(y))
            new.append(seq[seq.shape[0] - (W - 1):])
        return torch.cat(ys).reshape(st["x"].shape), _place(st, new, st["state_out"].dtype)
    S, G = case["states"], case["groups"]
    A, D = st["A"].double(), st["D"].double()
    B, Cm, raw = (st[k] if steps else st[k].flatten(0, 1) for k in ("B", "C", "delta"))
    z = None if st["z"] is None else (st["z"] if steps else st["z"].flatten(0, 1))
    lengths = [b - a for a, b in zip(cu, cu[1:])]
    if max(lengths) > 200000:
        return None
    h = torch.stack([_before(st, i, (C, S)) for i in range(n)])
    y = torch.empty(x.shape[0], C, dtype=torch.float64, device=x.device)
    order = sorted(range(n), key=lambda i: -lengths[i])            # longest first: the live ones are a prefix
    h = h[order]
    first = torch.tensor([cu[i] for i in order], device=x.device)
    live = n
    for t in range(max(lengths)):                                  # token by token, all sequences at once
        while lengths[order[live - 1]] <= t:
            live -= 1
        r = first[:live] + t
        d = raw[r].double() + st["delta_bias"].double()
        d = torch.logaddexp(d, torch.zeros_like(d))
        xt = x[r].double()
        hb = h[:live].view(live, G, C // G, S)
        hb.mul_(torch.exp(d.unsqueeze(-1) * A).view_as(hb))
        hb.add_((d * xt).view(live, G, C // G, 1) * B[r].double().unsqueeze(2))
        y[r] = torch.einsum("lgcs,lgs->lgc", hb, Cm[r].double()).reshape(live, C) + D * xt
    if z is not None:
        zz = z.double()
        y = y * zz * sigmoid(zz)
    back = [h[order.index(i)] for i in range(n)]
    return y.reshape(st["x"].shape), _place(st, back, None)
