"""Cases of the operators of the tensor-parallel region between g and g*.

After g each rank holds the whole sequence and a slice of the channels, so a
tensor here is a list of t rank buffers.  Three operators work on them: rotary
positions (`sp_rope_*`), the gated linear recurrence along the sequence
(`sp_gated_scan_*`) and group norm with an activation (`sp_group_norm_*`).

`run` computes a case in plain torch operations, or with the library's entry
points where `own` is true; `exact` computes it from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 64 requests, 64 query and 8 key heads of 128 over 8 ranks,
        # each request at its own far position
        dict(name="rope_step", op="rope", t=8, b=64, s=1, heads=9, d=128, rot=128,
             layout="half", dtype="bf16", where="positions", scaling="parts", back=False),
        # queries and keys of one packed training batch of 16,384 tokens, h = 8192 over 8 ranks
        dict(name="rope_packed", op="rope", t=8, b=1, s=16384, heads=9, d=128, rot=128,
             layout="half", dtype="bf16", where="packed", scaling="none", back=False),
        # gradient of a partly rotated head of odd width, rows cut from a wider projection
        dict(name="rope_odd_back", op="rope", t=2, b=3, s=1999, heads=5, d=80, rot=20,
             layout="interleaved", dtype="fp16", where="dense", scaling="linear", back=True),
        # one decoding step of 64 requests, 8192 channels over 8 ranks
        dict(name="scan_step", op="scan", t=8, b=64, s=1, c=1024, tied=True, dtype="bf16",
             seqs=0, state=True, back=False),
        # prompts of one batch packed without padding, states in and out
        dict(name="scan_packed", op="scan", t=8, b=1, s=16384, c=1024, tied=True, dtype="bf16",
             seqs=12, state=True, back=False),
        # a training step (output and gradients) at the same size, the whole sequence one document
        dict(name="scan_train", op="scan", t=8, b=1, s=16384, c=1024, tied=True, dtype="bf16",
             seqs=0, state=False, back=True),
        # one rank's channels alone over a long sequence: little to run side by side
        dict(name="scan_long_rank", op="scan", t=1, b=1, s=65537, c=512, tied=True,
             dtype="bf16", seqs=0, state=True, back=True),
        # float32 with odd sizes, the input not tied to the gate
        dict(name="scan_odd_fp32", op="scan", t=2, b=3, s=1501, c=264, tied=False, dtype="fp32",
             seqs=0, state=True, back=True),
        # per-token norm of the heads of 64 decoded tokens
        dict(name="norm_step", op="norm", t=8, n=64, l=1, c=1024, groups=8, norm="layernorm",
             act="silu", dtype="bf16", back=False),
        # per-token norm of the heads of 16,384 tokens, output and gradients
        dict(name="norm_heads_train", op="norm", t=8, n=16384, l=1, c=1024, groups=8,
             norm="rmsnorm", act="silu", dtype="bf16", back=True),
        # groups over whole samples of 4096 positions, channels last, output and gradients
        dict(name="norm_samples_train", op="norm", t=1, n=8, l=4096, c=1280, groups=32,
             norm="layernorm", act="silu", dtype="bf16", back=True),
        # few and long samples of an odd length
        dict(name="norm_long_odd", op="norm", t=2, n=1, l=32771, c=640, groups=5,
             norm="layernorm", act="none", dtype="fp16", back=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes spread over their logarithm; tokens and channels cut so that no
    case is larger than the largest listed one."""
    op = rng.choice(("rope", "scan", "norm"))
    t = rng.choice((1, 2, 4, 8))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    wide = 2 if dtype == "fp32" else 1
    most = (1 << 27) // wide            # elements of one tensor over all ranks
    if op == "rope":
        d = rng.choice((32, 64, 80, 96, 128, 128, 192, 256))
        rot = rng.choice((d, d, d // 2, 4 * rng.randint(1, d // 4)))
        heads = rng.randint(1, 24)
        where = rng.choice(("dense", "packed", "positions"))
        s = max(1, min(_log(rng, 1, 16384), most // (t * heads * d)))
        b = 1 if where == "packed" else max(1, min(_log(rng, 1, 64), most // (t * heads * d * s)))
        return dict(op=op, t=t, b=b, s=s, heads=heads, d=d, rot=rot,
                    layout=rng.choice(("half", "interleaved")), dtype=dtype, where=where,
                    scaling=rng.choice(("none", "linear", "base", "parts")) if rot > 2 else "none",
                    back=rng.random() < 0.5)
    if op == "scan":
        c = 8 * _log(rng, 4, 256)
        packed = rng.random() < 0.5
        s = max(1, min(_log(rng, 1, 65536), most // (t * c)))
        b = 1 if packed else max(1, min(_log(rng, 1, 64), most // (t * c * s)))
        return dict(op=op, t=t, b=b, s=s, c=c, tied=rng.random() < 0.7, dtype=dtype,
                    seqs=_log(rng, 1, 64) if packed else 0, state=rng.random() < 0.5,
                    back=rng.random() < 0.5)
    c_group = 8 * rng.choice((1, 2, 3, 4, 5, 8, 10, 16, 16, 32))
    groups = rng.choice((1, 2, 4, 5, 8, 16, 32))
    c = c_group * groups
    l = rng.choice((1, 1, _log(rng, 2, 128), _log(rng, 128, 32768)))
    l = max(1, min(l, most // (t * c)))
    n = max(1, min(_log(rng, 1, 16384 if l == 1 else 64), most // (t * c * l)))
    return dict(op=op, t=t, n=n, l=l, c=c, groups=groups,
                norm=rng.choice(("layernorm", "layernorm", "rmsnorm")),
                act=rng.choice(("none", "silu")), dtype=dtype, back=rng.random() < 0.5)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        tokens = case["b"] * case["s"]
        n = case["t"] * tokens * case["heads"] * case["d"]
        # x read, y written; 6 operations a pair
        return {"bytes": 2 * n * size + (8 * tokens if case["where"] == "positions" else 0),
                "flops": 3 * n * case["rot"] // case["d"]}
    if case["op"] == "scan":
        n = case["t"] * case["b"] * case["s"] * case["c"]
        seqs = case["seqs"] or case["b"]
        states = 4 * case["t"] * seqs * case["c"] if case["state"] else 0
        # forward: gate and value read, y written, states in and out; backward: gate,
        # value and dy read, two gradients written, the states' gradients in and out
        units = 3 + (5 if case["back"] else 0)
        return {"bytes": units * n * size + states * (5 if case["back"] else 2),
                "flops": (40 if case["back"] else 12) * n}
    n = case["t"] * case["n"] * case["l"] * case["c"]
    stats = case["t"] * case["n"] * case["groups"] * 4 * (2 if case["norm"] == "layernorm" else 1)
    params = case["t"] * case["c"] * (2 if case["norm"] == "layernorm" else 1)
    units = 2 + (3 if case["back"] else 0)
    return {"bytes": units * n * size + stats * (2 if case["back"] else 1)
            + params * (size * 2 + 4 if case["back"] else size),
            "flops": (40 if case["back"] else 15) * n}


# ------------------------------------------------------------------- inputs

def _rand(shape, gen, dtype, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return x.mul_(scale).add_(shift).to(dtype)


def _lengths(total, seqs, rng):
    """Lengths of `seqs` packed sequences, lognormal around their mean; with four
    or more of them one is empty and one has a single token."""
    w = [math.exp(rng.gauss(0.0, 0.6)) for _ in range(seqs)]
    if seqs >= 4:
        w[1], w[2] = 0.0, 0.0
    cut, acc, ends = sum(w), 0.0, []
    for x in w:
        acc += x
        ends.append(int(round(total * acc / cut)))
    ends[-1] = total
    lens = [e - (ends[i - 1] if i else 0) for i, e in enumerate(ends)]
    if seqs >= 4 and lens[0] > 0:
        lens[0] -= 1
        lens[2] += 1
    return lens


def _offsets(total, seqs, rng):
    cu = [0]
    for n in _lengths(total, seqs, rng):
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


ROPE = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=4.0),
        "parts": dict(factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0, mscale=1.2)}


def _inv_freq(rot, base, scaling):
    """Radians per position of each pair, and the factor on cos and sin."""
    o = ROPE[scaling]
    f = o.get("factor", 1.0)
    if scaling == "base":
        base = base * f ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    w = torch.pow(torch.tensor(base, dtype=torch.float64), -2 * i / rot)
    if scaling == "linear":
        w = w / f
    if scaling == "parts":
        turns = o["original_len"] * w / (2 * math.pi)
        g = ((turns - o["low_turns"]) / (o["high_turns"] - o["low_turns"])).clamp(0, 1)
        w = w * (g + (1 - g) / f)
    return w, o.get("mscale", 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    t = case["t"]
    st = dict(case)
    if case["op"] == "rope":
        b, s, heads, d = case["b"], case["s"], case["heads"], case["d"]
        # the heads of one rank's fused projection: what follows them in a row is not read
        rows = [_rand((b, s, heads + 1, d), gen, dt) for _ in range(t)]
        st["x"] = [r[:, :, :heads] for r in rows]
        st["y"] = [torch.empty((b, s, heads, d), dtype=dt, device=DEV) for _ in range(t)]
        st["cu"] = _offsets(s, max(1, min(8, s)), rng) if case["where"] == "packed" else None
        st["positions"] = (torch.randint(0, 1 << 20, (b, s), generator=gen, device=DEV)
                           if case["where"] == "positions" else None)
        st["first"] = 100000 if case["where"] == "dense" else 0
        w, st["mscale"] = _inv_freq(case["rot"], 500000.0, case["scaling"])
        st["inv_freq"] = w.to(DEV)
        if own:
            from sp_boundary_norm_gb300 import binding as sp
            st["table"] = sp.sp_rope_table(case["rot"], base=500000.0, scaling=case["scaling"],
                                           **ROPE[case["scaling"]])
    elif case["op"] == "scan":
        b, s, c = case["b"], case["s"], case["c"]
        # half of the channels remember a few tokens, half up to thousands
        shift = torch.rand((c,), generator=gen, device=DEV) * 8
        st["gate"] = [(_rand((b, s, c), gen, torch.float32, 1.5) + shift).to(dt) for _ in range(t)]
        st["value"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
        st["cu"] = _offsets(s, case["seqs"], rng) if case["seqs"] else None
        n_states = case["seqs"] or b
        st["h0"] = ([_rand((n_states, c), gen, torch.float32) for _ in range(t)]
                    if case["state"] else None)
        st["y"] = [torch.empty_like(v) for v in st["value"]]
        st["hT"] = [torch.empty_like(h) for h in st["h0"]] if case["state"] else None
        if case["back"]:
            st["dy"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
            st["dhT"] = ([_rand((n_states, c), gen, torch.float32) for _ in range(t)]
                         if case["state"] else None)
            st["dgate"] = [torch.empty_like(v) for v in st["value"]]
            st["dvalue"] = [torch.empty_like(v) for v in st["value"]]
            st["dh0"] = [torch.empty_like(h) for h in st["h0"]] if case["state"] else None
            if own:
                from sp_boundary_norm_gb300 import binding as sp
                shape = sp.sp_gated_scan_states_shape(b, s, c)
                st["states"] = [torch.empty(shape, dtype=torch.float32, device=DEV)
                                for _ in range(t)]
    else:
        n, l, c, groups = case["n"], case["l"], case["c"], case["groups"]
        # activations with a mean per channel, as a trained layer's have
        shift = torch.randn((c,), generator=gen, device=DEV)
        st["x"] = [(_rand((n, l, c), gen, torch.float32) + shift).to(dt) for _ in range(t)]
        st["gamma"] = _rand((t * c,), gen, dt, 0.1, 1.0)
        st["beta"] = _rand((t * c,), gen, dt, 0.1) if case["norm"] == "layernorm" else None
        st["y"] = [torch.empty_like(x) for x in st["x"]]
        stat = lambda: [torch.empty((n, groups), dtype=torch.float32, device=DEV)  # noqa: E731
                        for _ in range(t)]
        st["mean"] = stat() if case["norm"] == "layernorm" else None
        st["rstd"] = stat()
        st["eps"] = 1e-5 if case["norm"] == "layernorm" else 1e-6
        if case["back"]:
            st["dy"] = [_rand((n, l, c), gen, dt) for _ in range(t)]
            st["dx"] = [torch.empty_like(x) for x in st["x"]]
            st["dgamma"] = torch.empty((t * c,), dtype=torch.float32, device=DEV)
            st["dbeta"] = torch.empty_like(st["dgamma"]) if case["norm"] == "layernorm" else None
            if own:
                from sp_boundary_norm_gb300 import binding as sp
                st["workspace"] = torch.empty(
                    sp.sp_group_norm_bwd_workspace_bytes(n, l, c, groups, t, dtype=dt),
                    dtype=torch.uint8, device=DEV)
    return st


# -------------------------------------------------------------------- passes

def run(st):
    if own:
        return {"rope": _own_rope, "scan": _own_scan, "norm": _own_norm}[st["op"]](st)
    return {"rope": _plain_rope, "scan": _plain_scan, "norm": _plain_norm}[st["op"]](st)


def _own_rope(st):
    from sp_boundary_norm_gb300 import binding as sp
    where = dict(layout=st["layout"], positions=st["positions"], first_position=st["first"],
                 cu_seqlens=st["cu"])
    if st["back"]:
        sp.sp_rope_bwd(st["x"], st["table"], dx=st["y"], **where)
    else:
        sp.sp_rope_fwd(st["x"], st["table"], y=st["y"], **where)
    return st["y"]


def _own_scan(st):
    from sp_boundary_norm_gb300 import binding as sp
    how = dict(tied=st["tied"], cu_seqlens=st["cu"], h0=st["h0"])
    sp.sp_gated_scan_fwd(st["gate"], st["value"], y=st["y"], hT=st["hT"],
                         states=st.get("states"), **how)
    out = {"y": st["y"], "hT": st["hT"]}
    if st["back"]:
        sp.sp_gated_scan_bwd(st["gate"], st["value"], st["states"], st["dy"], dhT=st["dhT"],
                             dgate=st["dgate"], dvalue=st["dvalue"], dh0=st["dh0"], **how)
        out.update(dgate=st["dgate"], dvalue=st["dvalue"], dh0=st["dh0"])
    return out


def _own_norm(st):
    from sp_boundary_norm_gb300 import binding as sp
    how = dict(groups=st["groups"], norm=st["norm"], act=st["act"])
    sp.sp_group_norm_fwd(st["x"], st["gamma"], st["beta"], eps=st["eps"], y=st["y"],
                         mean=st["mean"], rstd=st["rstd"], **how)
    out = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if st["back"]:
        sp.sp_group_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"], st["beta"],
                             dx=st["dx"], dgamma=st["dgamma"], dbeta=st["dbeta"],
                             workspace=st["workspace"], **how)
        out.update(dx=st["dx"], dgamma=st["dgamma"], dbeta=st["dbeta"])
    return out


def _starts(cu, s):
    """Of each token of a packed batch its sequence, and whether it begins one."""
    tok = torch.arange(s, device=DEV)
    seq = torch.searchsorted(cu[1:].long(), tok, right=True)
    return seq, tok == cu.long()[seq]


def _plain_rope(st):
    x = torch.stack(st["x"]).float()
    s, rot = st["s"], st["rot"]
    if st["positions"] is not None:
        pos = st["positions"].double()
    else:
        pos = torch.arange(st["first"], st["first"] + s, device=DEV, dtype=torch.float64)
        if st["cu"] is not None:
            seq, _ = _starts(st["cu"], s)
            pos = pos - st["cu"].long()[seq]
    ang = pos[..., None] * st["inv_freq"]             # 32 bits would lose far positions' angles
    cos = (torch.cos(ang) * st["mscale"]).float()[..., None, :]
    sin = (torch.sin(ang) * st["mscale"]).float()[..., None, :]
    if st["back"]:
        sin = -sin
    if st["layout"] == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    y = torch.cat((turned, x[..., rot:]), -1).to(st["x"][0].dtype)
    return list(y)


def _scan(a, u):
    """h[i] = a[i] h[i-1] + u[i] along dim 2, h[-1] = 0, by doubling steps."""
    step, n = 1, a.shape[2]
    while step < n:
        u = torch.cat((u[:, :, :step], u[:, :, step:] + a[:, :, step:] * u[:, :, :-step]), 2)
        if 2 * step < n:
            a = torch.cat((a[:, :, :step], a[:, :, step:] * a[:, :, :-step]), 2)
        step *= 2
    return u


def _plain_scan(st):
    g, v = torch.stack(st["gate"]).float(), torch.stack(st["value"]).float()
    dt = st["value"][0].dtype
    t, b, s, c = g.shape
    a, k = torch.sigmoid(g), torch.sigmoid(-g)        # k = 1 - a without its cancellation
    first = torch.zeros((b, s), dtype=torch.bool, device=DEV)
    last = first.clone()
    if st["cu"] is None:
        first[:, 0], last[:, -1] = True, True
        rows = torch.arange(b, device=DEV)
        full = torch.ones(b, dtype=torch.bool, device=DEV)
    else:
        cu = st["cu"].long()
        full = cu[1:] > cu[:-1]                        # the sequences that have a token
        first[0, cu[:-1][full]] = True
        last[0, cu[1:][full] - 1] = True
        rows = torch.nonzero(full)[:, 0]
    h0 = torch.zeros((t, full.numel(), c), device=DEV)
    if st["h0"] is not None:
        h0 = torch.stack(st["h0"])
    keep = torch.where(first[None, :, :, None], 0.0, a)
    u = k * v if st["tied"] else v
    start = torch.zeros_like(u)
    start[:, first] = a[:, first] * h0[:, rows]
    h = _scan(keep, u + start)
    out = {"y": list(h.to(dt)), "hT": None}
    if st["state"]:
        hT = h0.clone()
        hT[:, rows] = h[:, last]
        out["hT"] = list(hT)
    if not st["back"]:
        return out
    d = torch.stack(st["dy"]).float()
    dhT = torch.zeros_like(h0) if st["dhT"] is None else torch.stack(st["dhT"])
    d[:, last] += dhT[:, rows]
    # dh[i] = d[i] + a[i+1] dh[i+1] inside a sequence: the same scan from the end
    nxt = torch.cat((keep[:, :, 1:], torch.zeros_like(keep[:, :, :1])), 2)
    dh = _scan(nxt.flip(2), d.flip(2)).flip(2)
    before = torch.cat((torch.zeros_like(h[:, :, :1]), h[:, :, :-1]), 2)
    before[:, first] = h0[:, rows]
    da = dh * (before - v if st["tied"] else before)
    dh0 = dhT.clone()
    dh0[:, rows] = (a * dh)[:, first]
    out.update(dgate=list((da * a * k).to(dt)), dvalue=list((dh * k if st["tied"] else dh).to(dt)),
               dh0=list(dh0) if st["state"] else None)
    return out


def _plain_norm(st):
    x = torch.stack(st["x"]).float()
    dt = st["x"][0].dtype
    t, n, l, c = x.shape
    x = x.view(t, n, l, st["groups"], -1)
    ln = st["norm"] == "layernorm"
    gamma = st["gamma"].float().view(t, 1, 1, st["groups"], -1)
    beta = st["beta"].float().view(t, 1, 1, st["groups"], -1) if ln else 0.0
    mean = x.mean((2, 4), keepdim=True) if ln else None
    z = x - mean if ln else x
    rstd = torch.rsqrt((z * z).mean((2, 4), keepdim=True) + st["eps"])
    z = z * rstd
    q = z * gamma + beta
    sig = torch.sigmoid(q) if st["act"] == "silu" else None
    y = q * sig if st["act"] == "silu" else q
    out = {"y": list(y.view(t, n, l, c).to(dt)),
           "mean": list(mean.view(t, n, -1)) if ln else None, "rstd": list(rstd.view(t, n, -1))}
    if not st["back"]:
        return out
    dq = torch.stack(st["dy"]).float().view_as(x)
    if st["act"] == "silu":
        dq = dq * (sig * (1 + q * (1 - sig)))
    dz = dq * gamma
    dx = dz - z * (dz * z).mean((2, 4), keepdim=True)
    if ln:
        dx = dx - dz.mean((2, 4), keepdim=True)
    out.update(dx=list((dx * rstd).view(t, n, l, c).to(dt)),
               dgamma=(dq * z).sum((1, 2)).view(-1),
               dbeta=dq.sum((1, 2)).view(-1) if ln else None)
    return out


# --------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](st)


def _exact_rope(st):
    """Each pair as a complex number, times mscale exp(i position frequency)."""
    s, rot, half = st["s"], st["rot"], st["rot"] // 2
    o = ROPE[st["scaling"]]
    freq = []
    for i in range(half):
        base = 500000.0
        if st["scaling"] == "base":
            base *= math.exp(math.log(o["factor"]) * rot / (rot - 2))
        w = math.exp(-math.log(base) * 2 * i / rot)
        if st["scaling"] == "linear":
            w /= o["factor"]
        if st["scaling"] == "parts":
            g = (o["original_len"] * w / math.tau - o["low_turns"]) / (o["high_turns"] - o["low_turns"])
            g = min(1.0, max(0.0, g))
            w = g * w + (1 - g) * w / o["factor"]
        freq.append(w)
    if st["positions"] is not None:
        pos = st["positions"]
    elif st["cu"] is not None:
        cu = st["cu"].tolist()
        pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])])[None].to(DEV)
    else:
        pos = (torch.arange(s, device=DEV) + st["first"])[None]
    ang = pos.double()[..., None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(ang, o.get("mscale", 1.0)), -ang if st["back"] else ang)
    out = []
    for x in st["x"]:
        y = x.double()
        part = y[..., :rot]
        pairs = part.unflatten(-1, (2, half)).transpose(-1, -2) if st["layout"] == "half" \
            else part.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, :, None])
        y[..., :rot] = (z.transpose(-1, -2) if st["layout"] == "half" else z).flatten(-2)
        out.append(y)
    return out


def _exact_scan(st):
    """Token by token; the gradients by the chain rule backwards through the tokens."""
    def tokens_first(xs):
        return torch.stack(xs, 1).permute(2, 0, 1, 3).double()       # (s, b, t, c)

    def ranks(x):
        return [r.permute(1, 0, 2) for r in x.unbind(2)]

    g, v = tokens_first(st["gate"]), tokens_first(st["value"])
    s, b, t, c = g.shape
    cu = st["cu"].tolist() if st["cu"] is not None else None
    spans = [(0, s)] if cu is None else list(zip(cu, cu[1:]))
    begins = {p: i for i, (p, q) in enumerate(spans) if q > p}
    ends = {q - 1: i for i, (p, q) in enumerate(spans) if q > p}
    # states: all batch rows of a dense call, one row of a packed call at a time
    states = (1, b, t, c) if cu is None else (len(spans), 1, t, c)
    zero = torch.zeros(states, dtype=torch.float64, device=DEV)
    h0 = zero if st["h0"] is None else torch.stack(st["h0"], 1).double().view(states)
    a = 1 / (1 + torch.exp(-g))
    w = v / (1 + torch.exp(g)) if st["tied"] else v
    hT, y, h = h0.clone(), torch.empty_like(g), None
    for i in range(s):
        if i in begins:
            h = h0[begins[i]]
        h = torch.addcmul(w[i], a[i], h, out=y[i])
        if i in ends:
            hT[ends[i]] = h
    out = {"y": ranks(y), "hT": list(hT.view(-1, t, c).unbind(1)) if st["state"] else None}
    if not st["back"]:
        return out
    dy = tokens_first(st["dy"])
    dhT = zero if st["dhT"] is None else torch.stack(st["dhT"], 1).double().view(states)
    dh, dh0 = torch.empty_like(y), dhT.clone()
    for i in reversed(range(s)):
        if i in ends:
            torch.add(dy[i], dhT[ends[i]], out=dh[i])
        else:
            torch.addcmul(dy[i], a[i + 1], dh[i + 1], out=dh[i])
        if i in begins:
            dh0[begins[i]] = a[i] * dh[i]
    y = y.roll(1, 0)                                   # the state before each token
    for i, k in begins.items():
        y[i] = h0[k]
    dg = dh * torch.exp(-g) * a * a * (y - v if st["tied"] else y)
    out.update(dgate=ranks(dg), dvalue=ranks(dh / (1 + torch.exp(g)) if st["tied"] else dh),
               dh0=list(dh0.view(-1, t, c).unbind(1)) if st["state"] else None)
    return out


def _exact_norm(st):
    """The formula rank by rank; the gradients by differentiating it."""
    ln, c, groups = st["norm"] == "layernorm", st["c"], st["groups"]
    out = {"y": [], "mean": [] if ln else None, "rstd": []}
    back = {"dx": [], "dgamma": [], "dbeta": [] if ln else None}
    for r, x in enumerate(st["x"]):
        x = x.double().requires_grad_(st["back"])
        gamma = st["gamma"][r * c:(r + 1) * c].double().requires_grad_(st["back"])
        beta = st["beta"][r * c:(r + 1) * c].double().requires_grad_(st["back"]) if ln else None
        # group by group: rows of the l * c / groups values that share their statistics
        xg = x.unflatten(2, (groups, -1)).transpose(1, 2).flatten(2)
        mean = xg.sum(-1) / xg.shape[-1] if ln else torch.zeros_like(xg[..., 0])
        var = ((xg - mean[..., None]) ** 2).sum(-1) / xg.shape[-1]
        rstd = 1 / torch.sqrt(var + st["eps"])
        z = ((xg - mean[..., None]) * rstd[..., None]).unflatten(2, (st["l"], -1))
        q = z.transpose(1, 2).flatten(2) * gamma
        q = q + beta if ln else q
        y = q / (1 + torch.exp(-q)) if st["act"] == "silu" else q
        if st["back"]:
            want = (x, gamma, beta) if ln else (x, gamma)
            got = torch.autograd.grad(y, want, st["dy"][r].double())
            back["dx"].append(got[0])
            back["dgamma"].append(got[1])
            if ln:
                back["dbeta"].append(got[2])
        out["y"].append(y.detach())
        if ln:
            out["mean"].append(mean.detach())
        out["rstd"].append(rstd.detach())
    if st["back"]:
        out.update(dx=back["dx"], dgamma=torch.cat(back["dgamma"]),
                   dbeta=torch.cat(back["dbeta"]) if ln else None)
    return out
