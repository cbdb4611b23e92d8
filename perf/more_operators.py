"""Cases of a state space layer and of rotary positions with several axes.

They run between g and the next g*, on lists of t rank buffers like the operators
that `perf/operators.py` measures: rotary positions whose pairs follow several
coordinates of a token (`sp_rope_axes_*`), the short causal convolution along the
tokens (`sp_causal_conv_*`) and the selective state space scan behind it
(`sp_selective_scan_*`).

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
        # one decoding step of 64 requests that hold images and video: 64 query and 8 key
        # heads of 128 over 8 ranks, pairs shared out to time, height and width
        dict(name="axes_step", op="axes", t=8, b=64, s=1, heads=9, d=128, sections="16,24,24",
             order="blocks", freq="shared", layout="half", dtype="bf16", back=False),
        # queries and keys of one batch of 16,384 video patches, h = 8192 over 8 ranks
        dict(name="axes_video", op="axes", t=8, b=1, s=16384, heads=9, d=128,
             sections="16,24,24", order="cyclic", freq="shared", layout="half", dtype="bf16",
             back=False),
        # gradient of an image encoder's heads of odd width: height and width, each with
        # its own frequencies
        dict(name="axes_image_back", op="axes", t=2, b=3, s=1999, heads=5, d=80,
             sections="20,20", order="blocks", freq="own", layout="interleaved", dtype="fp16",
             back=True),
        # one decoding step of 64 requests, 8192 channels over 8 ranks
        dict(name="conv_step", op="conv", t=8, b=64, s=1, c=1024, width=4, act="silu",
             dtype="bf16", seqs=0, state=True, back=False),
        # prompts of one batch packed without padding, states in and out
        dict(name="conv_packed", op="conv", t=8, b=1, s=16384, c=1024, width=4, act="silu",
             dtype="bf16", seqs=12, state=True, back=False),
        # a training step (output and gradients) at the same size, one document
        dict(name="conv_train", op="conv", t=8, b=1, s=16384, c=1024, width=4, act="silu",
             dtype="bf16", seqs=0, state=False, back=True),
        # float32 with odd sizes and three taps
        dict(name="conv_odd_fp32", op="conv", t=2, b=3, s=1501, c=264, width=3, act="none",
             dtype="fp32", seqs=0, state=True, back=True),
        # one decoding step of 64 requests, 8192 channels of 16 states over 8 ranks
        dict(name="ssm_step", op="ssm", t=8, b=64, s=1, c=1024, n=16, groups=1, gated=True,
             dtype="bf16", seqs=0, state=True, back=False),
        # prompts of one batch packed without padding, states in and out
        dict(name="ssm_packed", op="ssm", t=8, b=1, s=8192, c=1024, n=16, groups=1, gated=True,
             dtype="bf16", seqs=12, state=True, back=False),
        # a training step (output and gradients), one document
        dict(name="ssm_train", op="ssm", t=8, b=1, s=8192, c=1024, n=16, groups=1, gated=True,
             dtype="bf16", seqs=0, state=False, back=True),
        # one rank's channels alone over a long sequence: little to run side by side
        dict(name="ssm_long_rank", op="ssm", t=1, b=1, s=32769, c=512, n=16, groups=1,
             gated=False, dtype="bf16", seqs=0, state=True, back=True),
        # float32 with odd sizes, more states, two groups of channels
        dict(name="ssm_odd_fp32", op="ssm", t=2, b=3, s=701, c=272, n=32, groups=2, gated=True,
             dtype="fp32", seqs=0, state=True, back=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Sizes spread over their logarithm; tokens and channels cut so that no
    case is larger than the largest listed one."""
    op = rng.choice(("axes", "conv", "ssm"))
    t = rng.choice((1, 2, 4, 8))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    wide = 2 if dtype == "fp32" else 1
    most = (1 << 27) // wide            # elements of one tensor over all ranks
    if op == "axes":
        axes = rng.choice((2, 2, 3, 3, 4))
        d = rng.choice((32, 64, 80, 96, 128, 128, 192, 256))
        pairs = rng.choice((d // 2, d // 2, d // 4, rng.randint(axes, d // 2)))
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        heads = rng.randint(1, 24)
        s = max(1, min(_log(rng, 1, 16384), most // (t * heads * d)))
        b = max(1, min(_log(rng, 1, 64), most // (t * heads * d * s)))
        return dict(op=op, t=t, b=b, s=s, heads=heads, d=d,
                    sections=",".join(str(n) for n in sections),
                    order=rng.choice(("blocks", "cyclic")), freq=rng.choice(("shared", "own")),
                    layout=rng.choice(("half", "interleaved")), dtype=dtype,
                    back=rng.random() < 0.5)
    c = 8 * _log(rng, 4, 256)
    packed = rng.random() < 0.5
    if op == "conv":
        s = max(1, min(_log(rng, 1, 65536), most // (t * c)))
        b = 1 if packed else max(1, min(_log(rng, 1, 64), most // (t * c * s)))
        return dict(op=op, t=t, b=b, s=s, c=c, width=rng.choice((2, 3, 4, 4)),
                    act=rng.choice(("none", "silu", "silu")), dtype=dtype,
                    seqs=_log(rng, 1, 64) if packed else 0, state=rng.random() < 0.5,
                    back=rng.random() < 0.5)
    n = rng.choice((8, 16, 16, 32, 64))
    most = (1 << 29) // n               # channels of tokens: half the largest's states
    s = max(1, min(_log(rng, 1, 32768), most // (t * c)))
    b = 1 if packed else max(1, min(_log(rng, 1, 64), most // (t * c * s)))
    groups = rng.choice([g for g in (1, 1, 1, 2, 4) if c % (8 * g) == 0])
    return dict(op=op, t=t, b=b, s=s, c=c, n=n, groups=groups, gated=rng.random() < 0.6,
                dtype=dtype, seqs=_log(rng, 1, 64) if packed else 0, state=rng.random() < 0.5,
                back=rng.random() < 0.5)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    t, tokens = case["t"], case["b"] * case["s"]
    if case["op"] == "axes":
        sections = [int(v) for v in case["sections"].split(",")]
        n = t * tokens * case["heads"]
        # x read, y written, the coordinates; 6 operations a pair
        return {"bytes": 2 * n * case["d"] * size + 8 * tokens * len(sections),
                "flops": 6 * n * sum(sections)}
    n = t * tokens * case["c"]
    seqs = case["seqs"] or case["b"]
    if case["op"] == "conv":
        w = case["width"]
        params = t * case["c"] * (w + 1)
        states = t * seqs * (w - 1) * case["c"] * size if case["state"] else 0
        # forward: x read, y written, states in and out; backward: x and dy read, dx
        # written, the state and its gradients
        return {"bytes": (2 + (3 if case["back"] else 0)) * n * size
                + states * (5 if case["back"] else 2)
                + params * ((2 * size + 4) if case["back"] else size),
                "flops": n * ((6 * w + 20) if case["back"] else (2 * w + 5))}
    states = t * seqs * case["c"] * case["n"] * 4 if case["state"] else 0
    shared = 2 * t * tokens * case["groups"] * case["n"] * size      # B and C
    params = t * case["c"] * (case["n"] + 2) * 4
    units = 3 + case["gated"] + ((5 + 2 * case["gated"]) if case["back"] else 0)
    # forward: u, dt, z, B, C read, y written; backward: those and dy read, the gradients
    # of each written
    return {"bytes": units * n * size + states * (5 if case["back"] else 2)
            + shared * (3 if case["back"] else 1) + params * (3 if case["back"] else 1),
            "flops": n * case["n"] * (28 if case["back"] else 7)}


# ------------------------------------------------------------------- inputs

def _rand(shape, gen, dtype, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return x.mul_(scale).add_(shift).to(dtype)


def _offsets(total, seqs, rng):
    """Prefix sums of `seqs` packed sequences, lognormal around their mean; with four
    or more of them one is empty and one has a single token."""
    w = [math.exp(rng.gauss(0.0, 0.6)) for _ in range(seqs)]
    if seqs >= 4:
        w[1], w[2] = 0.0, 0.0
    whole, acc, cu = sum(w), 0.0, [0]
    for x in w:
        acc += x
        cu.append(int(round(total * acc / whole)))
    cu[-1] = total
    if seqs >= 4 and cu[1] > 0:
        cu[1] -= 1
        cu[2] -= 1
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _axes_table(sections, order, freq):
    """Axis and radians per position of each pair; the first axis counts frames, two
    to a second."""
    pairs = sum(sections)
    if order == "blocks":
        axis = [k for k, n in enumerate(sections) for _ in range(n)]
    else:
        axis = [k for i in range(max(sections)) for k, n in enumerate(sections) if i < n]
    place = [axis[:i].count(k) for i, k in enumerate(axis)]
    rate = [i / pairs if freq == "shared" else place[i] / sections[k] for i, k in enumerate(axis)]
    w = torch.pow(torch.tensor(10000.0, dtype=torch.float64),
                  -torch.tensor(rate, dtype=torch.float64))
    axis = torch.tensor(axis)
    return axis.to(DEV), torch.where(axis == 0, w / 2, w).to(DEV)


def _coordinates(axes, b, s, gen):
    """Patches of one video a row, frame by frame and line by line behind a text of a
    random length; a single token is at a far position."""
    if s == 1:
        return torch.randint(0, 1 << 20, (axes, b, s), generator=gen, device=DEV)
    side = max(1, int(round(math.sqrt(s / 8))))
    i = torch.arange(s, device=DEV)
    first = torch.randint(0, 100000, (1, b, 1), generator=gen, device=DEV)
    grid = torch.stack((i // (side * side), i // side % side, i % side, i % 7))
    return (grid[4 - axes if axes == 2 else 0:][:axes, None] + first).contiguous()


def _buffers(st, name, shape, dtype):
    """Output buffers of all ranks: one tensor, and the list of its parts."""
    st["out"][name] = torch.empty((st["t"],) + tuple(shape), dtype=dtype, device=DEV)
    st[name] = list(st["out"][name].unbind(0))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    t, b, s = case["t"], case["b"], case["s"]
    st = dict(case, out={})
    if own:
        from sp_boundary_norm_gb300 import binding as sp
    if case["op"] == "axes":
        heads, d = case["heads"], case["d"]
        sections = [int(v) for v in case["sections"].split(",")]
        # the heads of one rank's fused projection: what follows them in a row is not read
        rows = [_rand((b, s, heads + 1, d), gen, dt) for _ in range(t)]
        st["x"] = [r[:, :, :heads] for r in rows]
        _buffers(st, "y", (b, s, heads, d), dt)
        st["positions"] = _coordinates(len(sections), b, s, gen)
        st["sections"] = sections
        st["axis"], st["inv_freq"] = _axes_table(sections, case["order"], case["freq"])
        if own:
            st["table"] = sp.sp_rope_axes_table(
                sections, base=10000.0, order=case["order"], frequencies=case["freq"],
                factors=[2.0] + [1.0] * (len(sections) - 1))
        return st
    c, seqs, back = case["c"], case["seqs"], case["back"]
    st["cu"] = _offsets(s, seqs, rng) if seqs else None
    n_states = seqs or b
    f32 = torch.float32
    if case["op"] == "conv":
        w = case["width"]
        st["x"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
        st["weight"] = _rand((t * c, w), gen, dt, 0.5)
        st["bias"] = _rand((t * c,), gen, dt, 0.1)
        shape = (n_states, w - 1, c)
        st["x0"] = [_rand(shape, gen, dt) for _ in range(t)] if case["state"] else None
        _buffers(st, "y", (b, s, c), dt)
        st["xT"] = st["dxT"] = st["dx0"] = None
        if case["state"]:
            _buffers(st, "xT", shape, dt)
        if back:
            st["dy"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
            _buffers(st, "dx", (b, s, c), dt)
            if case["state"]:
                st["dxT"] = [_rand(shape, gen, dt) for _ in range(t)]
                _buffers(st, "dx0", shape, dt)
            st["out"]["dweight"] = torch.empty((t * c, w), dtype=f32, device=DEV)
            st["out"]["dbias"] = torch.empty((t * c,), dtype=f32, device=DEV)
            if own:
                st["workspace"] = torch.empty(
                    sp.sp_causal_conv_bwd_workspace_bytes(b, s, c, w, t, dtype=dt),
                    dtype=torch.uint8, device=DEV)
        return st
    n, groups = case["n"], case["groups"]
    st["u"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
    st["dt"] = [_rand((b, s, c), gen, dt, 0.5) for _ in range(t)]
    # steps between 0.001 and 0.1, as such layers begin with
    step = torch.exp(torch.rand((t * c,), generator=gen, device=DEV) * math.log(100.0)) * 1e-3
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    st["A"] = -torch.arange(1, n + 1, device=DEV, dtype=f32) * torch.exp(
        _rand((t * c, n), gen, f32, 0.2))
    st["D"] = _rand((t * c,), gen, f32, 0.1, 1.0)
    # one rank's B and C lie beside each other in the projection's rows
    rows = [_rand((b, s, 2 * groups * n), gen, dt) for _ in range(t)]
    st["B"] = [r[..., :groups * n] for r in rows]
    st["C"] = [r[..., groups * n:] for r in rows]
    st["z"] = [_rand((b, s, c), gen, dt) for _ in range(t)] if case["gated"] else None
    shape = (n_states, c, n)
    st["h0"] = [_rand(shape, gen, f32) for _ in range(t)] if case["state"] else None
    _buffers(st, "y", (b, s, c), dt)
    st["hT"] = st["dhT"] = st["dh0"] = st["dz"] = None
    if case["state"]:
        _buffers(st, "hT", shape, f32)
    if back:
        st["dy"] = [_rand((b, s, c), gen, dt) for _ in range(t)]
        for name in ("du", "ddt") + (("dz",) if case["gated"] else ()):
            _buffers(st, name, (b, s, c), dt)
        for name in ("dB", "dC"):
            _buffers(st, name, (b, s, groups * n), dt)
        if case["state"]:
            st["dhT"] = [_rand(shape, gen, f32) for _ in range(t)]
            _buffers(st, "dh0", shape, f32)
        for name in ("A", "D", "dt_bias"):
            st["out"]["d" + name] = torch.empty_like(st[name])
    if own:
        size = sp.sp_selective_scan_fwd_workspace_bytes(b, s, c, n, groups, t)
        if back:
            shape = sp.sp_selective_scan_states_shape(b, s, c, n)
            st["states"] = [torch.empty(shape, dtype=f32, device=DEV) for _ in range(t)]
            size = max(size, sp.sp_selective_scan_bwd_workspace_bytes(b, s, c, n, groups, t))
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# -------------------------------------------------------------------- passes

def run(st):
    if own:
        return {"axes": _own_axes, "conv": _own_conv, "ssm": _own_ssm}[st["op"]](st)
    return {"axes": _plain_axes, "conv": _plain_conv, "ssm": _plain_ssm}[st["op"]](st)


def _own_axes(st):
    from sp_boundary_norm_gb300 import binding as sp
    where = dict(layout=st["layout"], positions=st["positions"])
    if st["back"]:
        sp.sp_rope_axes_bwd(st["x"], st["table"], dx=st["y"], **where)
    else:
        sp.sp_rope_axes_fwd(st["x"], st["table"], y=st["y"], **where)
    return st["out"]


def _own_conv(st):
    from sp_boundary_norm_gb300 import binding as sp
    how = dict(act=st["act"], x0=st["x0"], cu_seqlens=st["cu"])
    sp.sp_causal_conv_fwd(st["x"], st["weight"], st["bias"], y=st["y"], xT=st["xT"], **how)
    if st["back"]:
        sp.sp_causal_conv_bwd(st["x"], st["weight"], st["bias"], st["dy"], dxT=st["dxT"],
                              dx=st["dx"], dx0=st["dx0"], dweight=st["out"]["dweight"],
                              dbias=st["out"]["dbias"], workspace=st["workspace"], **how)
    return st["out"]


def _own_ssm(st):
    from sp_boundary_norm_gb300 import binding as sp
    args = (st["u"], st["dt"], st["A"], st["B"], st["C"])
    how = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"], h0=st["h0"], cu_seqlens=st["cu"],
               workspace=st["workspace"])
    sp.sp_selective_scan_fwd(*args, y=st["y"], hT=st["hT"], states=st.get("states"), **how)
    if st["back"]:
        sp.sp_selective_scan_bwd(*args, st["states"], st["dy"], dhT=st["dhT"], du=st["du"],
                                 ddt=st["ddt"], dz=st["dz"], dB=st["dB"], dC=st["dC"],
                                 dA=st["out"]["dA"], dD=st["out"]["dD"],
                                 ddt_bias=st["out"]["ddt_bias"], dh0=st["dh0"], **how)
    return st["out"]


def _plain_axes(st):
    x = torch.stack(st["x"]).float()
    half = sum(st["sections"])
    pos = st["positions"].double().movedim(0, -1)     # 32 bits would lose far positions' angles
    ang = pos[..., st["axis"]] * st["inv_freq"]
    cos, sin = torch.cos(ang).float()[..., None, :], torch.sin(ang).float()[..., None, :]
    if st["back"]:
        sin = -sin
    if st["layout"] == "half":
        u, v = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
    else:
        u, v = x[..., :2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
    return {"y": torch.cat((turned, x[..., 2 * half:]), -1).to(st["x"][0].dtype)}


def _places(st):
    """First token (of all the batch's) and length of every sequence; of every token its
    sequence and its place there."""
    b, s = st["b"], st["s"]
    tok = torch.arange(b * s, device=DEV)
    if st["cu"] is None:
        begin = torch.arange(b, device=DEV) * s
        return begin, torch.full_like(begin, s), tok // s, tok % s
    cu = st["cu"].long()
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return cu[:-1], cu[1:] - cu[:-1], seq, tok - cu[seq]


def _plain_conv(st):
    t, b, s, c, w = st["t"], st["b"], st["s"], st["c"], st["width"]
    dt = st["x"][0].dtype
    x = torch.stack(st["x"]).float().view(t, b * s, c)
    weight = st["weight"].float().view(t, 1, c, w)
    bias = st["bias"].float().view(t, 1, c)
    begin, length, seq, place = _places(st)
    n = begin.numel()
    x0 = (torch.stack(st["x0"]).float() if st["x0"] is not None
          else torch.zeros((t, n, w - 1, c), device=DEV))

    def back(xs, k):
        """xs k tokens earlier, from the state before a sequence's begin."""
        if k == 0:
            return xs
        old = x0[:, seq, (w - 1 + place - k).clamp(0, w - 2)]
        moved = torch.cat((torch.zeros_like(xs[:, :k]), xs[:, :max(0, b * s - k)]), 1)[:, :b * s]
        return torch.where((place >= k)[:, None], moved, old)

    taps = [back(x, w - 1 - j) for j in range(w)]
    q = bias + sum(weight[..., j] * taps[j] for j in range(w))
    sig = torch.sigmoid(q)
    y = q * sig if st["act"] == "silu" else q
    out = {"y": y.view(t, b, s, c).to(dt)}
    # the last w - 1 inputs of a sequence, some of them from before it where it is short
    last = length[:, None] - (w - 1) + torch.arange(w - 1, device=DEV)
    rows = torch.arange(n, device=DEV)[:, None]
    from_x = (last >= 0)
    at = (begin[:, None] + last).clamp(0, b * s - 1)
    if st["state"]:
        old = x0[:, rows, (w - 1 + last).clamp(0, w - 2)]
        out["xT"] = torch.where(from_x[..., None], x[:, at], old).to(dt)
    if not st["back"]:
        return out
    dq = torch.stack(st["dy"]).float().view_as(q)
    if st["act"] == "silu":
        dq = dq * (sig * (1 + q * (1 - sig)))
    left = (length[seq] - place)[:, None]             # tokens from here to the sequence's end
    ahead = [torch.where(left > k, torch.cat((dq[:, k:], torch.zeros_like(dq[:, :k])), 1)[:, :b * s],
                         0.0) for k in range(w)]
    dx = sum(weight[..., j] * ahead[w - 1 - j] for j in range(w))
    dx0 = torch.zeros((t, n, w - 1, c), device=DEV)
    for j in range(w - 1):                            # tap j of token m - j reads x0[m]
        for m in range(j, w - 1):
            has = (length > m - j)[:, None]
            dx0[:, :, m] += torch.where(has, weight[..., j] * dq[:, (begin + m - j).clamp(max=b * s - 1)],
                                        0.0)
    if st["dxT"] is not None:
        dxT = torch.stack(st["dxT"]).float()
        dx.index_put_((torch.arange(t, device=DEV)[:, None], at[from_x]),
                      dxT[:, from_x], accumulate=True)
        old = (~from_x).nonzero()
        dx0.index_put_((torch.arange(t, device=DEV)[:, None], old[:, 0],
                        w - 1 + last[old[:, 0], old[:, 1]]), dxT[:, old[:, 0], old[:, 1]],
                       accumulate=True)
    out.update(dx=dx.view(t, b, s, c).to(dt), dx0=dx0.to(dt) if st["state"] else None,
               dweight=torch.stack([(dq * tap).sum(1) for tap in taps], -1).view(t * c, w),
               dbias=dq.sum(1).view(t * c))
    return out


def _scan(a, u):
    """h[i] = a[i] h[i-1] + u[i] along dim 2, h[-1] = 0, by doubling steps."""
    step, n = 1, a.shape[2]
    while step < n:
        u = torch.cat((u[:, :, :step], u[:, :, step:] + a[:, :, step:] * u[:, :, :-step]), 2)
        if 2 * step < n:
            a = torch.cat((a[:, :, :step], a[:, :, step:] * a[:, :, :-step]), 2)
        step *= 2
    return u


def _plain_ssm(st):
    t, b, s, c, n, groups = (st[k] for k in ("t", "b", "s", "c", "n", "groups"))
    dt = st["u"][0].dtype
    u = torch.stack(st["u"]).float()
    pre = torch.stack(st["dt"]).float() + st["dt_bias"].view(t, 1, 1, c)
    step = pre.clamp(min=0) + torch.log1p(torch.exp(-pre.abs()))          # softplus
    A, D = st["A"].view(t, 1, 1, c, n), st["D"].view(t, 1, 1, c)

    def spread(xs):                                   # a group's B or C to its channels
        x = torch.stack(xs).float().view(t, b, s, groups, 1, n)
        return x.expand(t, b, s, groups, c // groups, n).reshape(t, b, s, c, n)

    begin, length, seq, place = _places(st)
    full = length > 0
    rows = torch.nonzero(full)[:, 0]
    first = (place == 0).view(b, s)
    last = (place == length[seq] - 1).view(b, s)
    h0 = (torch.stack(st["h0"]) if st["h0"] is not None
          else torch.zeros((t, begin.numel(), c, n), device=DEV))
    a = torch.exp(step[..., None] * A)
    add = (step * u)[..., None] * spread(st["B"])
    add[:, first] += a[:, first] * h0[:, rows]
    keep = a.clone()
    keep[:, first] = 0.0
    h = _scan(keep, add)
    del add
    inner = (h * spread(st["C"])).sum(-1) + D * u
    z = torch.stack(st["z"]).float() if st["gated"] else None
    sig = torch.sigmoid(z) if st["gated"] else None
    y = inner * z * sig if st["gated"] else inner
    out = {"y": y.to(dt)}
    if st["state"]:
        out["hT"] = h0.clone()
        out["hT"][:, rows] = h[:, last]
    if not st["back"]:
        return out
    dy = torch.stack(st["dy"]).float()
    if st["gated"]:
        out["dz"] = (dy * inner * (sig * (1 + z * (1 - sig)))).to(dt)
    e = dy * z * sig if st["gated"] else dy
    d = spread(st["C"]) * e[..., None]
    dh0 = torch.zeros_like(h0) if st["dhT"] is None else torch.stack(st["dhT"]).clone()
    d[:, last] += dh0[:, rows]
    # G[i] = d[i] + a[i+1] G[i+1] inside a sequence: the same scan from the end
    keep = torch.cat((keep[:, :, 1:], torch.zeros_like(keep[:, :, :1])), 2)
    G = _scan(keep.flip(2), d.flip(2)).flip(2)
    del keep, d

    def gather(x):                                    # and back, over a group's channels
        return x.view(t, b, s, groups, c // groups, n).sum(4).view(t, b, s, groups * n).to(dt)

    out["dC"] = gather(h * e[..., None])
    before = torch.cat((torch.zeros_like(h[:, :, :1]), h[:, :, :-1]), 2)
    before[:, first] = h0[:, rows]
    del h
    g = a * G
    dh0[:, rows] = g[:, first]
    g = g * before
    del a, before
    out["dA"] = (g * step[..., None]).sum((1, 2)).view(t * c, n)
    dstep = (g * A).sum(-1)
    del g
    out["dB"] = gather(G * (step * u)[..., None])
    through = (G * spread(st["B"])).sum(-1)
    dpre = (dstep + u * through) * torch.sigmoid(pre)
    out.update(du=(step * through + D * e).to(dt), ddt=dpre.to(dt),
               dD=(e * u).sum((1, 2)).view(-1), ddt_bias=dpre.sum((1, 2)).view(-1),
               dh0=dh0 if st["state"] else None)
    return out


# --------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"axes": _exact_axes, "conv": _exact_conv, "ssm": _exact_ssm}[case["op"]](st)


def _spans(st):
    """(batch row, first token, end) of every sequence."""
    if st["cu"] is None:
        return [(r, 0, st["s"]) for r in range(st["b"])]
    cu = st["cu"].tolist()
    return [(0, p, q) for p, q in zip(cu, cu[1:])]


def _exact_axes(st):
    """Each pair as a complex number, times exp(i coordinate frequency)."""
    sections, pairs = st["sections"], sum(st["sections"])
    left, freq, turn = list(sections), [0.0] * pairs, []
    for i in range(pairs):
        if st["order"] == "blocks":
            k = next(k for k in range(len(left)) if left[k])
        else:                                         # the axis that has been served least
            k = min((k for k in range(len(left)) if left[k]),
                    key=lambda k: (sections[k] - left[k], k))
        j = sections[k] - left[k]
        left[k] -= 1
        rate = i / pairs if st["freq"] == "shared" else j / sections[k]
        freq[i] = math.exp(-math.log(10000.0) * rate) / (2.0 if k == 0 else 1.0)
        turn.append(st["positions"][k].double() * freq[i])
    ang = torch.stack(turn, -1)
    turn = torch.polar(torch.ones_like(ang), -ang if st["back"] else ang)
    out = []
    for x in torch.stack(st["x"]):
        y = x.double()
        part = y[..., :2 * pairs]
        two = part.unflatten(-1, (2, pairs)).transpose(-1, -2) if st["layout"] == "half" \
            else part.unflatten(-1, (pairs, 2))
        z = torch.view_as_real(torch.view_as_complex(two.contiguous()) * turn[:, :, None])
        y[..., :2 * pairs] = (z.transpose(-1, -2) if st["layout"] == "half" else z).flatten(-2)
        out.append(y)
    return {"y": torch.stack(out)}


def _exact_conv(st):
    """Sequence by sequence: windows over its inputs behind its state; the gradients by
    differentiating that."""
    c, w, back = st["c"], st["width"], st["back"]
    out = {name: [] for name in st["out"]}
    spans = _spans(st)
    for r, x in enumerate(st["x"]):
        x = x.double().requires_grad_(back)
        x0 = (st["x0"][r].double() if st["state"]
              else torch.zeros((len(spans), w - 1, c), dtype=torch.float64, device=DEV))
        x0.requires_grad_(back)
        weight = st["weight"][r * c:(r + 1) * c].double().requires_grad_(back)
        bias = st["bias"][r * c:(r + 1) * c].double().requires_grad_(back)
        if st["cu"] is None:
            runs = [torch.cat((x0, x), 1)]
        else:
            runs = [torch.cat((x0[j], x[row, p:q]))[None] for j, (row, p, q) in enumerate(spans)]
        ends = torch.cat([v[:, v.shape[1] - (w - 1):] for v in runs])
        ys = []
        for v in runs:
            if v.shape[1] < w:
                continue
            q = torch.einsum("bsck,ck->bsc", v.unfold(1, w, 1), weight) + bias
            ys.append(q / (1 + torch.exp(-q)) if st["act"] == "silu" else q)
        y = ys[0] if st["cu"] is None else torch.cat(ys, 1)
        out["y"].append(y.detach())
        if st["state"]:
            out["xT"].append(ends.detach())
        if back:
            loss = (y * st["dy"][r].double()).sum()
            if st["state"]:
                loss = loss + (ends * st["dxT"][r].double()).sum()
            got = torch.autograd.grad(loss, (x, x0, weight, bias))
            out["dx"].append(got[0])
            if st["state"]:
                out["dx0"].append(got[1])
            out["dweight"].append(got[2])
            out["dbias"].append(got[3])
    return {name: (torch.cat if name in ("dweight", "dbias") else torch.stack)(parts)
            for name, parts in out.items()}


def _exact_ssm(st):
    """Token by token; the gradients by the chain rule backwards through the tokens."""
    t, s, c, n, groups, back = (st[k] for k in ("t", "s", "c", "n", "groups", "back"))
    f64 = torch.float64

    def tokens_first(xs):
        return torch.stack(xs, 1).permute(2, 0, 1, 3).to(f64)        # (s, b, t, width)

    def ranks(x):
        return x.permute(2, 1, 0, 3)

    u, raw = tokens_first(st["u"]), tokens_first(st["dt"])
    raw = raw + st["dt_bias"].to(f64).view(t, c)
    d = torch.logaddexp(raw, torch.zeros_like(raw))
    B, C = tokens_first(st["B"]), tokens_first(st["C"])
    b = u.shape[1]
    A = st["A"].to(f64).view(t, groups, c // groups, n)
    D = st["D"].to(f64).view(t, c)
    cell = (b, t, groups, c // groups, n)
    chan = (b, t, groups, c // groups, 1)
    shared = (b, t, groups, 1, n)
    spans = _spans(st)
    packed = st["cu"] is not None
    begins = {p: j for j, (_, p, q) in enumerate(spans) if q > p}
    ends = {q - 1: j for j, (_, p, q) in enumerate(spans) if q > p}
    seqs = len(spans)
    held = (seqs, 1) + cell[1:] if packed else (1,) + cell
    h0 = (torch.stack(st["h0"], 1).to(f64).view(held) if st["h0"] is not None
          else torch.zeros(held, dtype=f64, device=DEV))
    hT = h0.clone()
    hs = torch.empty((s,) + cell, dtype=f64, device=DEV) if back else None
    inner = torch.empty_like(u)
    du = d * u
    h = None
    for i in range(s):
        if i in begins:
            h = h0[begins[i] if packed else 0]
        a = torch.exp(d[i].view(chan) * A)
        h = torch.addcmul(du[i].view(chan) * B[i].view(shared), a, h)
        if back:
            hs[i] = h
        inner[i] = (h * C[i].view(shared)).sum(-1).view(b, t, c)
        if i in ends:
            hT[ends[i] if packed else 0] = h
    inner += D * u
    z = tokens_first(st["z"]) if st["gated"] else None
    gate = z / (1 + torch.exp(-z)) if st["gated"] else None

    def state(x):
        return x.reshape(seqs, t, c, n).transpose(0, 1) if st["state"] else None

    out = {"y": ranks(inner * gate if st["gated"] else inner), "hT": state(hT)}
    if not back:
        return out
    dy = tokens_first(st["dy"])
    e = dy * gate if st["gated"] else dy
    dz = None
    if st["gated"]:
        sig = 1 / (1 + torch.exp(-z))
        dz = ranks(dy * inner * (sig + gate * (1 - sig)))
    dhT = (torch.stack(st["dhT"], 1).to(f64).view(held) if st["dhT"] is not None
           else torch.zeros(held, dtype=f64, device=DEV))
    dh0 = dhT.clone()
    dA = torch.zeros((t, groups, c // groups, n), dtype=f64, device=DEV)
    dB, dC, through, dstep = (torch.empty_like(x) for x in (B, C, u, u))
    G = torch.zeros(cell, dtype=f64, device=DEV)
    for i in reversed(range(s)):
        if i in ends:
            G = dhT[ends[i] if packed else 0]
        G = torch.addcmul(G, C[i].view(shared), e[i].view(chan))
        dC[i] = (hs[i] * e[i].view(chan)).sum(3).view(b, t, -1)
        dB[i] = (G * du[i].view(chan)).sum(3).view(b, t, -1)
        through[i] = (G * B[i].view(shared)).sum(-1).view(b, t, c)
        G = G * torch.exp(d[i].view(chan) * A)
        if i in begins:
            j = begins[i] if packed else 0
            dh0[j] = G
            g = G * h0[j]
        else:
            g = G * hs[i - 1]
        dstep[i] = (g * A).sum(-1).view(b, t, c)
        dA += (g * d[i].view(chan)).sum(0)
    dpre = (dstep + u * through) / (1 + torch.exp(-raw))
    out.update(dz=dz, dB=ranks(dB), dC=ranks(dC), dA=dA.view(t * c, n),
               du=ranks(d * through + D * e), ddt=ranks(dpre), dD=(e * u).sum((0, 1)).view(-1),
               ddt_bias=dpre.sum((0, 1)).view(-1), dh0=state(dh0))
    return out
