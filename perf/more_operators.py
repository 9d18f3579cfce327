"""Work of a linear attention layer and of the norms around a block, as timed passes.

Three operators, each in its plain form (elementary torch operations in 32
bits, decays summed in 64) and through the package's entry points:

  linattn       linear attention with a decay for each head over prompts
                (gdn_linattn_fwd): S <- e^g S + v k^T, o = scale S q
  linattn_step  the same for one new token per sequence (gdn_linattn_step)
  block_norm    norm after a block, its gate and scale, the residual sum and
                the norm before the next block in one pass (gdn_block_norm)

A case holds sizes only; prepare() draws everything else from the seed.  q, k
and v are slices of one projection's rows.  States live in pools addressed by
slot numbers where a case has "slots"; a pass reads them from one pool and
writes them to a second one, so that it can be repeated on the same inputs (a
decoding loop passes one pool for both).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROW_ELEMENTS = 131072 * 8 * 256         # largest prompt: tokens x heads x (d_k + d_v)
STATE_ELEMENTS = 256 * 16 * 128 * 128   # largest step: sequences x heads x d_k x d_v
NORM_ELEMENTS = 16384 * 4096            # largest norm: rows x channels
CHUNK = 64                              # tokens per chunk of the plain form


def listed():
    return [
        # four training-length prompts, a data-dependent decay per token and head
        dict(name="lin_prompt", op="linattn", seqs=4, tokens=16384, packed=False, heads=16, groups=16, dk=128, dv=128,
             fixed=False, state=False, slots=False, extra=0, dtype="bf16"),
        # eight prompts of unequal length in one pack, continued from kept states, q and k shared by 4 heads each
        dict(name="lin_packed", op="linattn", seqs=8, tokens=27610, packed=True, heads=32, groups=8, dk=128, dv=128,
             fixed=False, state=True, slots=True, extra=64, dtype="bf16"),
        # one very long document, a fixed decay per head
        dict(name="lin_long", op="linattn", seqs=1, tokens=131072, packed=False, heads=8, groups=8, dk=128, dv=128,
             fixed=True, state=False, slots=False, extra=0, dtype="bf16"),
        # many small heads that share one q and k, two prompts
        dict(name="lin_shared", op="linattn", seqs=2, tokens=8192, packed=False, heads=64, groups=1, dk=128, dv=64,
             fixed=False, state=False, slots=False, extra=0, dtype="bf16"),
        # one short prompt: latency
        dict(name="lin_short", op="linattn", seqs=1, tokens=300, packed=False, heads=16, groups=16, dk=96, dv=192,
             fixed=True, state=True, slots=False, extra=0, dtype="bf16"),
        # short fp32 prompts with nothing a multiple of anything
        dict(name="lin_odd", op="linattn", seqs=3, tokens=3 * 517, packed=True, heads=6, groups=3, dk=77, dv=45,
             fixed=False, state=True, slots=True, extra=5, dtype="f32"),
        # one token of each of 256 sequences being decoded
        dict(name="lin_step_batch", op="linattn_step", seqs=256, heads=16, groups=16, dk=128, dv=128, fixed=False,
             slots=True, extra=0, dtype="bf16"),
        # one sequence being decoded: latency
        dict(name="lin_step_one", op="linattn_step", seqs=1, heads=16, groups=4, dk=128, dv=128, fixed=True,
             slots=False, extra=0, dtype="bf16"),
        # between two blocks of a prompt: norm after, gate, residual sum, norm before
        dict(name="norm_prompt", op="block_norm", rows=16384, channels=4096, rms=True, post=True, pre=True, affine=True,
             gate="silu", scale=True, residual_scale=1.0, stream="same", dtype="bf16"),
        # the same sum with a stream kept in 32 bits, mean and variance norms, no gate
        dict(name="norm_stream", op="block_norm", rows=8192, channels=2048, rms=False, post=True, pre=True, affine=True,
             gate="none", scale=False, residual_scale=0.5, stream="f32", dtype="bf16"),
        # a decoding batch of an odd width in fp32
        dict(name="norm_odd", op="block_norm", rows=256, channels=1925, rms=False, post=True, pre=True, affine=True,
             gate="sigmoid", scale=True, residual_scale=1.0, stream="same", dtype="f32"),
        # one sequence being decoded: latency
        dict(name="norm_one", op="block_norm", rows=1, channels=4096, rms=True, post=False, pre=True, affine=True,
             gate="none", scale=False, residual_scale=1.0, stream="same", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("linattn", "linattn", "linattn", "linattn_step", "block_norm", "block_norm"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "block_norm":
        channels = rng.choice((1024, 2048, 4096, 8192, _log(rng, 1, 12288), _log(rng, 1, 12288)))
        rows = max(1, min(_log(rng, 1, 65536), NORM_ELEMENTS // channels))
        post, pre = rng.choice(((True, True), (True, True), (False, True), (True, False)))
        return dict(op=op, rows=rows, channels=channels, rms=flag(), post=post, pre=pre, affine=flag(),
                    gate=rng.choice(("none", "sigmoid", "silu")), scale=flag(), residual_scale=rng.choice((1.0, 0.5)),
                    stream=rng.choice(("same", "f32")), dtype=dtype)
    heads = _log(rng, 1, 64)
    groups = rng.choice([g for g in range(1, heads + 1) if heads % g == 0])
    dk, dv = rng.choice(((128, 128), (128, 128), (64, 64), (128, 64), (96, 192), (128, 256),
                         (_log(rng, 1, 128), _log(rng, 1, 256))))
    extra = rng.choice((0, 0, 64, 5))
    if op == "linattn":
        seqs = _log(rng, 1, 32)
        packed = flag()
        tokens = max(1, min(_log(rng, 1, 131072), ROW_ELEMENTS // (heads * (dk + dv))))
        tokens = tokens if packed else max(1, tokens // seqs) * seqs
        return dict(op=op, seqs=seqs, tokens=tokens, packed=packed, heads=heads, groups=groups, dk=dk, dv=dv,
                    fixed=flag(), state=flag(), slots=flag(), extra=extra, dtype=dtype)
    seqs = max(1, min(_log(rng, 1, 1024), STATE_ELEMENTS // (heads * dk * dv)))
    return dict(op=op, seqs=seqs, heads=heads, groups=groups, dk=dk, dv=dv, fixed=flag(), slots=flag(), extra=extra,
                dtype=dtype)


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

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype) * scale

    if op == "block_norm":
        R, C = case["rows"], case["channels"]
        st["y"] = normal(R, C, dtype=dt) + normal(R, 1, dtype=dt)
        st["residual"] = normal(R, C, scale=3.0, dtype=torch.float32 if case["stream"] == "f32" else dt)
        st["gate"] = normal(R, C, dtype=dt) if case["gate"] != "none" else None
        st["scale"] = normal(C, scale=0.1) if case["scale"] else None
        for side in ("post", "pre"):
            has = case["affine"] and case[side]
            st[side + "_weight"] = 1 + normal(C, scale=0.1) if has else None
            st[side + "_bias"] = normal(C, scale=0.1) if has and not case["rms"] else None
        return st

    n, H, G, dk, dv = (case[k] for k in ("seqs", "heads", "groups", "dk", "dv"))
    if op == "linattn":
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
    # one projection's rows: something else | q | k | v
    p = normal(rows, case["extra"] + 2 * G * dk + H * dv, dtype=dt)
    q, k, v = p[:, case["extra"]:].split((G * dk, G * dk, H * dv), 1)
    st["q"] = q.unflatten(1, (G, dk)).unflatten(0, lead)
    st["k"] = k.unflatten(1, (G, dk)).unflatten(0, lead)
    st["v"] = v.unflatten(1, (H, dv)).unflatten(0, lead)
    st["scale"] = dk ** -0.5
    if case["fixed"]:      # heads that keep 32 to 8192 tokens
        st["decay"] = torch.log1p(-torch.exp2(-5 - 8 * torch.rand(H, generator=g, device=dev)))
    else:                  # a step size of 1e-3 to 1e-1 around each head's own, times a rate of 1 to 16
        rate = 1 + 15 * torch.rand(H, generator=g, device=dev)
        step = torch.exp(torch.rand(H, generator=g, device=dev) * math.log(100.0) + math.log(0.001))
        st["decay"] = (-rate * step * torch.exp(normal(rows, H, scale=0.5))).unflatten(0, lead)
    has = op == "linattn_step" or case["state"]
    st["state_in"] = normal(pool, H, dv, dk) if has else None
    st["state_out"] = torch.zeros(pool, H, dv, dk, device=dev)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return OWN[op](st)
    return PLAIN[op](st)


def _own_linattn(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_linattn_fwd(st["q"], st["k"], st["v"], st["decay"], scale=st["scale"], state_in=st["state_in"],
                               state_out=st["state_out"], slots=st["slots"],
                               cu_seqlens=st["cu"] if st["case"]["packed"] else None)


def _own_linattn_step(st):
    import gated_delta_rule_09_gb300 as gdn
    return gdn.gdn_linattn_step(st["q"], st["k"], st["v"], st["decay"], scale=st["scale"], state_in=st["state_in"],
                                state_out=st["state_out"], slots=st["slots"])


def _own_block_norm(st):
    import gated_delta_rule_09_gb300 as gdn
    c = st["case"]
    out, h = gdn.gdn_block_norm(st["y"], st["residual"], post_weight=st["post_weight"], post_bias=st["post_bias"],
                                pre_weight=st["pre_weight"], pre_bias=st["pre_bias"], gate=st["gate"],
                                gate_act=c["gate"], scale=st["scale"], residual_scale=c["residual_scale"], eps=1e-5,
                                rms=c["rms"], post=c["post"], pre=c["pre"])
    return (out, h) if c["pre"] else out


def _keep(st, new):
    """Write the sequences' new states to their places in the output pool."""
    if st["slots"] is None:
        st["state_out"].copy_(new)
    else:
        st["state_out"].index_copy_(0, st["slots"].long(), new)
    return st["state_out"]


def _kept(st):
    """The sequences' states before the call."""
    if st["state_in"] is None:
        return torch.zeros(st["case"]["seqs"], *st["state_out"].shape[1:], device=st["state_out"].device)
    return st["state_in"] if st["slots"] is None else st["state_in"][st["slots"].long()]


def _plain_linattn(st):
    H, G = st["case"]["heads"], st["case"]["groups"]
    q, k, v = (st[n].flatten(0, 1) for n in ("q", "k", "v"))
    R, dev = v.shape[0], v.device
    decay = st["decay"].expand(R, H) if st["case"]["fixed"] else st["decay"].flatten(0, 1)
    cu = st["cu"].long()
    n = cu.numel() - 1
    # the sequences one after another in whole chunks; rows past a sequence's end carry nothing
    length = cu[1:] - cu[:-1]
    chunks = (length + CHUNK - 1) // CHUNK
    last = chunks.cumsum(0)
    first = last - chunks
    M = R // CHUNK + n                                            # at most so many
    c = torch.arange(M, device=dev)
    s = torch.searchsorted(last, c, right=True)
    used = s < n
    s = s.clamp(max=n - 1)
    token = (c - first[s])[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    real = (token < length[s][:, None]) & used[:, None]
    row = torch.where(real, cu[:-1][s][:, None] + token, R)
    at = row.clamp(max=R - 1)
    live = real[:, None, :, None]
    lay = lambda t: torch.where(live, t[at].float().transpose(1, 2), 0.0)  # noqa: E731
    qc, kc = (lay(t).repeat_interleave(H // G, 1) for t in (q, k))
    vc = lay(v)
    g = torch.where(real[:, None], decay[at].double().transpose(1, 2), 0.0).cumsum(-1)     # [M, H, CHUNK]
    seen = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    between = torch.where(seen, torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~seen, 0.0)), 0.0).float()
    o = (qc @ kc.transpose(-1, -2) * between) @ vc
    del between
    b = (vc * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(-1, -2) @ kc        # [M, H, dv, dk]
    a = torch.exp(g[..., -1]).float()
    # a sequence's kept state enters at its first chunk; then spans are doubled until they cover a sequence
    some = (length > 0).float()
    start = first.clamp(max=M - 1)
    h0 = _kept(st)
    b.index_add_(0, start, a[start][:, :, None, None] * h0 * some[:, None, None, None])
    is_start = torch.zeros(M, device=dev).index_add_(0, start, some)
    a = a * (1 - is_start)[:, None]
    off = 1
    while off * CHUNK < st["longest"]:
        b = torch.cat([b[:off], torch.addcmul(b[off:], a[off:][:, :, None, None], b[:-off])])
        a = torch.cat([a[:off], a[off:] * a[:-off]])
        off *= 2
    before = torch.cat([torch.zeros_like(b[:1]), b[:-1]]) * (1 - is_start)[:, None, None, None]
    before.index_add_(0, start, h0 * some[:, None, None, None])
    o = (o + torch.exp(g).float()[..., None] * (qc @ before.transpose(-1, -2))) * st["scale"]
    out = torch.empty(R + 1, H, o.shape[-1], device=dev)
    out[row] = o.transpose(1, 2)
    final = torch.where(some[:, None, None, None] > 0, b[(last - 1).clamp(min=0)], h0)
    return out[:R].to(v.dtype).unflatten(0, st["lead"]), _keep(st, final)


def _plain_linattn_step(st):
    r = st["case"]["heads"] // st["case"]["groups"]
    q, k = (st[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    decay = torch.exp(st["decay"])
    h = decay[..., None, None] * _kept(st) + st["v"].float()[..., None] * k[:, :, None]
    o = (h * q[:, :, None]).sum(-1) * st["scale"]
    return o.to(st["v"].dtype), _keep(st, h)


def _normed(x, weight, bias, rms):
    if not rms:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    if weight is not None:
        x = x * weight
    return x if bias is None else x + bias


def _plain_block_norm(st):
    c = st["case"]
    u = st["y"].float()
    if c["post"]:
        u = _normed(u, st["post_weight"], st["post_bias"], c["rms"])
    if st["gate"] is not None:
        gate = st["gate"].float()
        u = u * torch.sigmoid(gate) * (gate if c["gate"] == "silu" else 1.0)
    if st["scale"] is not None:
        u = u * st["scale"]
    r = st["residual"].float() * c["residual_scale"] + u
    out = r.to(st["residual"].dtype)
    if not c["pre"]:
        return out
    return out, _normed(r, st["pre_weight"], st["pre_bias"], c["rms"]).to(st["y"].dtype)


OWN = dict(linattn=_own_linattn, linattn_step=_own_linattn_step, block_norm=_own_block_norm)
PLAIN = dict(linattn=_plain_linattn, linattn_step=_plain_linattn_step, block_norm=_plain_block_norm)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "block_norm":
        C, n = case["channels"], case["rows"] * case["channels"]
        stream = 4 if case["stream"] == "f32" else e
        parts = case["post"] + case["pre"]
        params = case["scale"] + case["affine"] * parts * (1 if case["rms"] else 2)
        return {"bytes": n * (e * (1 + (case["gate"] != "none") + case["pre"]) + 2 * stream) + 4 * C * params,
                "flops": n * (3 + 5 * parts + 4 * (case["gate"] != "none"))}
    seqs, H, G, dk, dv = (case[k] for k in ("seqs", "heads", "groups", "dk", "dv"))
    rows = case["tokens"] if op == "linattn" else seqs
    states = 2 if op == "linattn_step" or case["state"] else 1
    return {"bytes": rows * (2 * G * dk + 2 * H * dv) * e + 4 * H * (1 if case["fixed"] else rows)
            + states * seqs * H * dk * dv * 4,
            "flops": rows * H * dk * dv * 4}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _place(st, new):
    """The output pool after the call, with the sequences' new states in place."""
    pool = torch.zeros_like(st["state_out"], dtype=torch.float64)
    for i, s in enumerate(range(len(new)) if st["slots"] is None else st["slots"].tolist()):
        pool[s] = new[i]
    return pool


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    sigmoid = lambda t: 1 / (1 + torch.exp(-t))  # noqa: E731
    if op == "block_norm":
        def norm(x, weight, bias):
            if case["rms"]:
                x = x / torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / x.shape[1] + 1e-5)
            else:
                var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
                x = (x - mean) / torch.sqrt(var + 1e-5)
            x = x if weight is None else x * weight.double()
            return x if bias is None else x + bias.double()

        u = st["y"].double()
        u = norm(u, st["post_weight"], st["post_bias"]) if case["post"] else u
        if st["gate"] is not None:
            gate = st["gate"].double()
            u = u * (sigmoid(gate) * gate if case["gate"] == "silu" else sigmoid(gate))
        u = u if st["scale"] is None else u * st["scale"].double()
        r = st["residual"].double() * case["residual_scale"] + u
        return (r, norm(r, st["pre_weight"], st["pre_bias"])) if case["pre"] else r
    n, H, G, dk, dv = (case[k] for k in ("seqs", "heads", "groups", "dk", "dv"))
    steps = op == "linattn_step"
    cu = list(range(n + 1)) if steps else st["cu"].tolist()
    lengths = [b - a for a, b in zip(cu, cu[1:])]
    if max(lengths) * max(1.0, n * H * dk * dv / 2e7) > 400000:
        return None
    q, k, v = (st[name] if steps else st[name].flatten(0, 1) for name in ("q", "k", "v"))
    if case["fixed"]:
        decay = torch.exp(st["decay"].double()).expand(v.shape[0], H)
    else:
        decay = torch.exp((st["decay"] if steps else st["decay"].flatten(0, 1)).double())
    order = sorted(range(n), key=lambda i: -lengths[i])            # longest first: the live ones are a prefix
    S = torch.zeros(n, H, dv, dk, dtype=torch.float64, device=v.device)
    if st["state_in"] is not None:
        where = list(range(n)) if st["slots"] is None else st["slots"].tolist()
        S = st["state_in"][[where[i] for i in order]].double()
    first = torch.tensor([cu[i] for i in order], device=v.device)
    o = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    live = n
    for t in range(max(lengths)):                                  # token by token, all sequences at once
        while lengths[order[live - 1]] <= t:
            live -= 1
        r = first[:live] + t
        Sl = S[:live].view(live, G, H // G, dv, dk)
        Sl.mul_(decay[r].view(live, G, H // G, 1, 1))
        Sl.addcmul_(v[r].double().view(live, G, H // G, dv, 1), k[r].double().view(live, G, 1, 1, dk))
        o[r] = torch.einsum("lghvk,lgk->lghv", Sl, q[r].double()).reshape(live, H, dv)
    back = [S[order.index(i)] for i in range(n)]
    return o.reshape(st["v"].shape) * st["scale"], _place(st, back)
