"""Rotary positions with several axes, the causal convolution and the selective scan on
the GPU against the float64 oracle.

Tolerances.  An output of type T is its exact value rounded once, off by at most
u |exact| with u = 2^-8 (bf16), 2^-11 (fp16; plus 2^-25, half the smallest subnormal),
2^-24 (float32), plus what the float32 arithmetic before it loses, relative to the
magnitude that the oracle returns beside the value:

- rotary: 2^-21, as with one axis (the same angles and products).
- convolution: four products and a bias, 5 2^-24 of their magnitude; silu's exponential
  is off by 2^-22 plus |q| 2^-24, its reciprocal by 2^-23, the products by a rounding
  each: 2^-20 of |y| for |q| <= 16, and q's own error passes with silu's slope, at most
  1.1.  In all 2^-19 of the magnitude.  Backward: twice that and the sums over a run of
  parameters, below 2^10 roundings in a row per thread and block: 2^-13 for those.
- scan: the step d is softplus of x = dt + dt_bias, |x| <= 8 in these tests: its
  exponential is off by 8 2^-24 (bias) + 8 2^-24 (product) + 2^-22, the rest by 2^-22:
  2^-20 of d.  A decay a = exp(d A) is off by 2^-22 of itself and by |d A| a 2^-19.5 <=
  0.37 2^-19.5 from d and the product's rounding: below 2^-20 of 1.  So over n tokens a
  state is off by at most (2^-19 + n 2^-20) of the largest magnitude that a state has;
  sums over states and channels add (n_state + channels) 2^-24.  The outputs take one
  state, gradients a product of two and a step: S = 2^-18 + n 2^-20 + 2^-15 for those.
"""
import numpy as np
import pytest
import torch

from oracle import state_space as orc
from sp_boundary_norm_gb300 import binding as sp

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 0.0, FP: 2.0 ** -25, F32: 0.0}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


def rand(shape, gen, dtype, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, dtype=F32) * scale + shift
    return x.to(dtype).to(DEV)


def nans(t, shape, dtype):
    return [torch.full(shape, NAN, dtype=dtype, device=DEV) for _ in range(t)]


def f64(x):
    return None if x is None else x.double().cpu().numpy()


def close(got, want, mag, rel, what):
    dtype = got.dtype
    got = f64(got)
    assert np.isfinite(got).all(), what
    tol = STEP[dtype] * np.abs(want) + LEAST[dtype] + rel * mag
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, the worst "
                           f"{(np.abs(got - want) - tol).max():.3g} over its tolerance")


def bits(x):
    return x.contiguous().view(torch.int32 if x.dtype == F32 else torch.int16)


def same(a, b):
    return len(a) == len(b) and all(torch.equal(bits(p), bits(q)) for p, q in zip(a, b))


def offsets(lens):
    return torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device=DEV)


def tensors(o):
    """Every tensor of a run's outputs, by name; saved states are internal."""
    return {f"{k}{i}": x for k, v in o.items() if k != "states" and v is not None
            for i, x in enumerate(v if isinstance(v, list) else [v])}


def same_runs(a, b):
    a, b = tensors(a), tensors(b)
    return a.keys() == b.keys() and all(torch.equal(bits(a[k]), bits(b[k])) for k in a)


# ------------------------------------------------------------ several axes --

AXES = [
    # t, b, s, heads, d, sections, order, frequencies, layout, dtype
    (1, 1, 1, 1, 2, [1], "blocks", "shared", "half", F32),
    (2, 3, 5, 7, 64, [8, 12, 12], "blocks", "shared", "half", BF),
    (8, 1, 17, 9, 128, [16, 24, 24], "cyclic", "shared", "half", BF),
    (2, 2, 33, 3, 128, [32, 32], "blocks", "own", "interleaved", FP),
    (1, 2, 9, 5, 80, [20, 20], "cyclic", "own", "interleaved", FP),
    (1, 2, 9, 5, 80, [3, 1, 6], "blocks", "own", "half", BF),
    (3, 1, 4, 2, 96, [7, 1, 9, 7], "cyclic", "shared", "half", F32),
    (1, 1, 3, 1, 512, [100, 56, 100], "cyclic", "own", "half", F32),
    (1, 1, 3, 2, 520, [250, 6], "blocks", "shared", "interleaved", F32),
    (2, 1, 6, 4, 15, [1, 2], "blocks", "shared", "interleaved", BF),
    (1, 1, 700, 3, 40, [1] * 8, "cyclic", "shared", "half", BF),
    (16, 1, 2, 70, 16, [4, 4], "blocks", "own", "half", BF),
]


@pytest.mark.parametrize("t,b,s,heads,d,sections,order,frequencies,layout,dtype", AXES)
@pytest.mark.parametrize("back", [False, True])
def test_axes(t, b, s, heads, d, sections, order, frequencies, layout, dtype, back):
    gen = torch.Generator().manual_seed(7)
    x = [rand((b, s, heads, d), gen, dtype) for _ in range(t)]
    pos = torch.randint(-(1 << 40), 1 << 40, (len(sections), b, s), generator=gen).to(DEV)
    factors = [1.0 + k for k in range(len(sections))]
    tab = sp.sp_rope_axes_table(sections, order=order, frequencies=frequencies, factors=factors,
                                mscale=1.1)
    axis, _ = orc.axes_table(sections, 10000.0, order, frequencies, factors)
    m = float(np.float32(1.1))

    def call(src, dst):
        if back:
            sp.sp_rope_axes_bwd(src, tab, layout=layout, positions=pos, dx=dst)
        else:
            sp.sp_rope_axes_fwd(src, tab, layout=layout, positions=pos, y=dst)

    y = nans(t, (b, s, heads, d), dtype)
    call(x, y)
    # turns by integers, from the frequencies that the table holds (positions this far show
    # its own rounding): position times turns modulo 2^64
    p = pos.cpu().numpy()
    with np.errstate(over="ignore"):
        turn = (p[axis].astype(np.uint64) *
                np.array([tab.turns[i] for i in range(len(axis))], np.uint64)[:, None, None])
    ang = np.moveaxis(turn.astype(np.float64) * 2.0 ** -64 * 2 * np.pi, 0, -1)
    one = np.arange(len(axis))
    for r in range(t):
        # (an angle a pair: each pair an axis of its own, one radian a unit)
        want, mag = orc.rope_axes(f64(x[r]), np.moveaxis(ang, -1, 0), one, np.ones(len(axis)), layout,
                                  m, back)
        close(y[r], want, mag, 2.0 ** -21, f"rank {r}")
        rot = 2 * len(axis)
        assert torch.equal(bits(y[r][..., rot:]), bits(x[r][..., rot:]))
    kept = [v.clone() for v in x]
    call(kept, kept)
    assert same(kept, y)


def test_axes_near_positions_and_one_axis():
    """The angles of small positions against the frequencies' formula; one axis gives the
    bits of the plain form."""
    gen = torch.Generator().manual_seed(8)
    x = [rand((2, 50, 3, 64), gen, F32)]
    y, z = nans(1, (2, 50, 3, 64), F32), nans(1, (2, 50, 3, 64), F32)
    pos = torch.randint(0, 4096, (3, 2, 50), generator=gen)
    tab = sp.sp_rope_axes_table([8, 12, 12], base=500000.0)
    axis, freq = orc.axes_table([8, 12, 12], 500000.0)
    sp.sp_rope_axes_fwd(x, tab, positions=pos.to(DEV), y=y)
    want, mag = orc.rope_axes(f64(x[0]), pos.numpy(), axis, freq)
    close(y[0], want, mag, 2.0 ** -21, "formula")
    one = torch.arange(100, device=DEV).view(1, 2, 50)
    sp.sp_rope_axes_fwd(x, sp.sp_rope_axes_table([24]), positions=one, y=y)
    sp.sp_rope_fwd(x, sp.sp_rope_table(48), positions=one[0], y=z)
    assert same(y, z)


def test_axes_strided_heads():
    """Queries and keys as slices of a fused projection's rows; what lies between stays."""
    gen = torch.Generator().manual_seed(9)
    row = rand((2, 9, 5 * 48 + 8), gen, BF)
    keep = row.clone()
    q = lambda r: r[..., :3 * 48].unflatten(2, (3, 48))
    tab = sp.sp_rope_axes_table([6, 10], order="cyclic")
    pos = torch.randint(0, 1 << 20, (2, 2, 9), generator=gen).to(DEV)
    want = nans(1, (2, 9, 3, 48), BF)
    sp.sp_rope_axes_fwd([q(keep).contiguous()], tab, positions=pos, y=want)
    sp.sp_rope_axes_fwd([q(row)], tab, positions=pos, y=[q(row)])
    assert same([q(row)], want) and torch.equal(row[..., 3 * 48:], keep[..., 3 * 48:])


# ----------------------------------------------------- causal convolution --

def conv_inputs(t, n, b, s, c, w, dtype, seed, state):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda shape, *a: [rand(shape, gen, dtype, *a) for _ in range(t)]
    return dict(x=mk((b, s, c)), dy=mk((b, s, c)), weight=rand((t * c, w), gen, dtype, 0.5),
                bias=rand((t * c,), gen, dtype, 0.3), x0=mk((n, w - 1, c)) if state else None,
                dxT=mk((n, w - 1, c)) if state else None)


def run_conv(i, n, act, cu, state):
    t, like = len(i["x"]), i["x"][0]
    b, s, c = like.shape
    w, dt = i["weight"].shape[1], like.dtype
    o = dict(y=nans(t, (b, s, c), dt), dx=nans(t, (b, s, c), dt),
             xT=nans(t, (n, w - 1, c), dt) if state else None,
             dx0=nans(t, (n, w - 1, c), dt) if state else None,
             dweight=torch.full((t * c, w), NAN, device=DEV), dbias=torch.full((t * c,), NAN, device=DEV))
    how = dict(act=act, x0=i["x0"], cu_seqlens=cu)
    sp.sp_causal_conv_fwd(i["x"], i["weight"], i["bias"], y=o["y"], xT=o["xT"], **how)
    ws = torch.empty(sp.sp_causal_conv_bwd_workspace_bytes(b, s, c, w, t, dtype=dt), dtype=torch.uint8,
                     device=DEV)
    sp.sp_causal_conv_bwd(i["x"], i["weight"], i["bias"], i["dy"], dxT=i["dxT"], dx=o["dx"], dx0=o["dx0"],
                          dweight=o["dweight"], dbias=o["dbias"], workspace=ws, **how)
    return o


def check_conv(i, o, act, lens, state):
    cu = None if lens is None else np.concatenate(([0], np.cumsum(lens)))
    c = i["x"][0].shape[2]
    for r in range(len(i["x"])):
        p = slice(r * c, (r + 1) * c)
        rank = lambda k: None if i[k] is None else f64(i[k][r])
        wt, bias = f64(i["weight"][p]), None if i["bias"] is None else f64(i["bias"][p])
        f = orc.causal_conv(rank("x"), wt, bias, act, rank("x0"), cu)
        close(o["y"][r], f["y"], f["mag"], 2.0 ** -19, f"y[{r}]")
        g = orc.causal_conv_bwd(rank("x"), wt, rank("dy"), bias, act, rank("x0"), cu, rank("dxT"))
        close(o["dx"][r], g["dx"], g["mag_dx"], 2.0 ** -18, f"dx[{r}]")
        if state:
            assert np.array_equal(f64(o["xT"][r]), f["xT"]), f"xT[{r}]"
            close(o["dx0"][r], g["dx0"], g["mag_dx0"], 2.0 ** -18, f"dx0[{r}]")
        close(o["dweight"][p], g["dweight"], g["mag_dweight"], 2.0 ** -13, f"dweight[{r}]")
        close(o["dbias"][p], g["dbias"], g["mag_dbias"], 2.0 ** -13, f"dbias[{r}]")


CONV = [
    # t, b, s, c, width, dtype
    (1, 1, 1, 8, 4, BF), (2, 5, 1, 72, 4, BF), (1, 3, 2, 64, 3, F32), (2, 2, 3, 8, 4, FP),
    (1, 3, 4, 136, 2, BF), (1, 1, 17, 264, 4, F32), (2, 1, 129, 64, 3, BF), (1, 2, 300, 200, 4, BF),
    (8, 1, 515, 64, 4, BF), (1, 1, 1031, 24, 2, F32), (3, 2, 257, 40, 3, FP), (1, 130, 33, 128, 4, BF),
    (1, 1, 9000, 16, 4, BF), (16, 2, 70, 8, 4, F32),
]


@pytest.mark.parametrize("t,b,s,c,w,dtype", CONV)
@pytest.mark.parametrize("act,state", [("silu", True), ("none", True), ("silu", False)])
def test_conv_dense(t, b, s, c, w, dtype, act, state):
    i = conv_inputs(t, b, b, s, c, w, dtype, 11, state)
    o = run_conv(i, b, act, None, state)
    check_conv(i, o, act, None, state)
    assert same_runs(o, run_conv(i, b, act, None, state))


LENS = [[1], [0, 1, 0], [2, 3, 1], [40], [0, 0, 70, 0, 3, 1, 1, 1, 0], [1] * 37,
        [16] * 9 + [0] * 40 + [17], [5, 600, 0, 2, 1000, 31, 33], list(range(30)),
        [0] * 70 + [300] + [0] * 70 + [9], [3, 61, 64, 128, 4, 60]]


@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
@pytest.mark.parametrize("dtype,c,w,act,state", [
    (BF, 72, 4, "silu", True), (F32, 64, 3, "none", True), (FP, 64, 2, "silu", False), (BF, 8, 4, "none", True)])
def test_conv_packed(lens, dtype, c, w, act, state):
    n, s = len(lens), sum(lens)
    i = conv_inputs(2, n, 1, s, c, w, dtype, 12, state)
    o = run_conv(i, n, act, offsets(lens), state)
    check_conv(i, o, act, lens, state)


def test_conv_optional_arguments():
    """No bias, no states, one gradient of the two, states without gradients."""
    i = conv_inputs(2, 3, 3, 50, 32, 4, BF, 13, True)
    full = run_conv(i, 3, "silu", None, True)
    i["bias"] = None
    o = run_conv(i, 3, "silu", None, True)
    check_conv(i, o, "silu", None, True)
    assert not same(o["y"], full["y"])
    dx = nans(2, (3, 50, 32), BF)
    sp.sp_causal_conv_bwd(i["x"], i["weight"], None, i["dy"], act="silu", x0=i["x0"], dxT=i["dxT"], dx=dx)
    assert same(dx, o["dx"])
    ws = torch.empty(sp.sp_causal_conv_bwd_workspace_bytes(3, 50, 32, 4, 2), dtype=torch.uint8, device=DEV)
    db = torch.full((64,), NAN, device=DEV)
    sp.sp_causal_conv_bwd(i["x"], i["weight"], None, i["dy"], act="silu", x0=i["x0"], dxT=i["dxT"], dx=dx,
                          dbias=db, workspace=ws)
    assert same([db], [o["dbias"]])


@pytest.mark.parametrize("lens", [None, [7, 0, 1, 2, 90]], ids=["dense", "packed"])
def test_conv_pieces_with_one_state(lens):
    """A sequence in pieces, down to single tokens, the state updated in place: the bits of
    the whole."""
    n = 3 if lens is None else len(lens)
    b, s = (3, 100) if lens is None else (1, 100)
    i = conv_inputs(2, n, b, s, 40, 4, BF, 14, True)
    cu = None if lens is None else offsets(lens)
    want = run_conv(i, n, "silu", cu, True)
    state = [v.clone() for v in i["x0"]]
    if lens is not None:
        y = nans(2, (b, s, 40), BF)
        sp.sp_causal_conv_fwd(i["x"], i["weight"], i["bias"], act="silu", x0=state, cu_seqlens=cu, y=y,
                              xT=state)
        assert same(y, want["y"]) and same(state, want["xT"])
        return
    parts = [[] for _ in range(2)]
    for lo, hi in ((0, 1), (1, 2), (2, 2), (2, 70), (70, 73), (73, 100)):
        y = nans(2, (b, hi - lo, 40), BF)
        sp.sp_causal_conv_fwd([v[:, lo:hi].contiguous() for v in i["x"]], i["weight"], i["bias"],
                              act="silu", x0=state, y=y, xT=state)
        for p, v in zip(parts, y):
            p.append(v)
    assert same([torch.cat(p, 1) for p in parts], want["y"]) and same(state, want["xT"])


def test_conv_strided_rows():
    """Slices of a wider projection's rows in and out; the rest stays."""
    i = conv_inputs(1, 2, 2, 37, 64, 4, BF, 15, True)
    want = run_conv(i, 2, "silu", None, True)
    wide = torch.full((2, 37, 3 * 64 + 8), 7.0, dtype=BF, device=DEV)
    x, y, dx = wide[..., :64], wide[..., 72:136], wide[..., 136:]
    x.copy_(i["x"][0])
    how = dict(act="silu", x0=i["x0"])
    sp.sp_causal_conv_fwd([x], i["weight"], i["bias"], y=[y], **how)
    sp.sp_causal_conv_bwd([x], i["weight"], i["bias"], i["dy"], dxT=i["dxT"], dx=[dx], **how)
    assert same([y, dx], [want["y"][0], want["dx"][0]])
    assert (wide[..., 64:72] == 7).all() and torch.equal(x, i["x"][0])


def test_conv_far_values():
    """Pre-activations where the exponential overflows or vanishes: silu and its slope are
    finite."""
    x = [torch.tensor([-3e4, -90.0, -88.0, -20.0, 0.0, 20.0, 90.0, 3e4]).repeat(8).view(1, 64, 1)
         .expand(1, 64, 8).contiguous().to(DEV)]
    for dtype in (F32, BF):
        i = dict(x=[x[0].to(dtype)], dy=[torch.ones(1, 64, 8, dtype=dtype, device=DEV)], x0=None, dxT=None,
                 weight=torch.tensor([[0.0, 1.0]] * 8, dtype=dtype, device=DEV), bias=None)
        o = run_conv(i, 1, "silu", None, False)
        v = f64(i["x"][0])
        sg = np.exp(-np.logaddexp(0, -v))
        slope = sg * (1 + v * (1 - sg))
        assert np.isfinite(f64(o["y"][0])).all() and np.isfinite(f64(o["dx"][0])).all()
        # a flushed sigmoid (below 2^-126) takes away |q| 2^-126; 1 - sigmoid near 0 is off
        # by 2^-24 of 1, times q where the slope is 1 + that
        assert (np.abs(f64(o["y"][0]) - v * sg) <= STEP[dtype] * np.abs(v * sg) + 2.0 ** -19 * np.abs(v * sg)
                + 2e-33).all()
        assert (np.abs(f64(o["dx"][0]) - slope) <= STEP[dtype] * np.abs(slope) + 2.0 ** -19
                + np.abs(v * sg) * 2.0 ** -24 * 2).all()


# --------------------------------------------------------- selective scan --

def ssm_inputs(t, m, b, s, c, n, groups, dtype, seed, state, gated=True, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda shape, dt=dtype, *a: [rand(shape, gen, dt, *a) for _ in range(t)]
    clip = lambda xs, m: [x.clamp(-m, m) for x in xs]
    rows = mk((b, s, 2 * groups * n + 8))
    step = torch.exp(torch.rand((t * c,), generator=gen) * np.log(300.0)) * 1e-3   # 0.001 .. 0.3
    return dict(u=mk((b, s, c)), dt=clip(mk((b, s, c), dtype, 0.5 * scale), 1.0),
                dt_bias=(step + torch.log(-torch.expm1(-step))).to(DEV),
                A=-torch.exp(rand((t * c, n), gen, F32, 0.8).clamp(-2.5, 2.5)) * 2,
                D=rand((t * c,), gen, F32), B=[r[..., :groups * n] for r in rows],
                C=[r[..., groups * n:2 * groups * n] for r in rows],
                z=clip(mk((b, s, c), dtype, 2.0), 8.0) if gated else None, dy=mk((b, s, c)),
                h0=mk((m, c, n), F32) if state else None, dhT=mk((m, c, n), F32) if state else None)


def scratch(size):
    return torch.empty(size, dtype=torch.uint8, device=DEV) if size else None


def run_ssm(i, m, cu, state, soft=True, back=True):
    t, like = len(i["u"]), i["u"][0]
    b, s, c = like.shape
    n, dt = i["A"].shape[1], like.dtype
    width = i["B"][0].shape[2]
    groups = width // n
    gated = i["z"] is not None
    o = dict(y=nans(t, (b, s, c), dt), hT=nans(t, (m, c, n), F32) if state else None,
             states=nans(t, sp.sp_selective_scan_states_shape(b, s, c, n), F32) if back else None)
    args = (i["u"], i["dt"], i["A"], i["B"], i["C"])
    how = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], softplus=soft, h0=i["h0"], cu_seqlens=cu)
    sp.sp_selective_scan_fwd(*args, y=o["y"], hT=o["hT"], states=o["states"],
                             workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(b, s, c, n, groups, t)),
                             **how)
    if not back:
        return o
    o.update(du=nans(t, (b, s, c), dt), ddt=nans(t, (b, s, c), dt),
             dz=nans(t, (b, s, c), dt) if gated else None, dB=nans(t, (b, s, width), dt),
             dC=nans(t, (b, s, width), dt), dh0=nans(t, (m, c, n), F32) if state else None,
             dA=torch.full((t * c, n), NAN, device=DEV), dD=torch.full((t * c,), NAN, device=DEV),
             ddt_bias=torch.full((t * c,), NAN, device=DEV))
    sp.sp_selective_scan_bwd(*args, o["states"], i["dy"], dhT=i["dhT"],
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(b, s, c, n, groups, t)),
                             **{k: o[k] for k in ("du", "ddt", "dB", "dC", "dz", "dA", "dD", "ddt_bias", "dh0")},
                             **how)
    return o


def check_ssm(i, o, lens, state, soft=True, ranks=None):
    cu = None if lens is None else np.concatenate(([0], np.cumsum(lens)))
    b, s, c = i["u"][0].shape
    longest = s if lens is None else max(lens)
    S = 2.0 ** -18 + longest * 2.0 ** -20 + 2.0 ** -15
    for r in range(len(i["u"]) if ranks is None else ranks):
        p = slice(r * c, (r + 1) * c)
        rank = lambda k: None if i[k] is None else f64(i[k][r])
        par = lambda k: None if i[k] is None else f64(i[k][p])
        w = orc.selective_scan(rank("u"), rank("dt"), par("A"), rank("B"), rank("C"), par("D"), rank("z"),
                               par("dt_bias"), soft, rank("h0"), cu, rank("dy"), rank("dhT"))
        for k in o:
            if k == "states" or o[k] is None:
                continue
            got = o[k][r] if isinstance(o[k], list) else o[k][p]
            close(got, w[k], w["mag_" + k], S, f"{k}[{r}]")


SSM = [
    # t, b, s, c, n, groups, dtype
    (1, 1, 1, 8, 8, 1, BF), (2, 5, 1, 72, 16, 1, BF), (1, 1, 2, 64, 32, 2, F32), (2, 2, 15, 8, 64, 1, FP),
    (1, 3, 16, 136, 16, 1, BF), (1, 1, 17, 64, 8, 8, F32), (2, 1, 31, 72, 16, 3, BF), (1, 2, 33, 24, 64, 3, BF),
    (2, 1, 129, 64, 32, 1, BF), (1, 2, 100, 200, 16, 1, F32), (8, 1, 65, 16, 16, 2, FP), (1, 1, 300, 8, 8, 1, F32),
    (1, 3, 5, 264, 32, 1, FP), (1, 20, 8, 40, 16, 1, BF),
]


@pytest.mark.parametrize("t,b,s,c,n,groups,dtype", SSM)
@pytest.mark.parametrize("state,gated,soft", [(True, True, True), (False, False, True), (True, False, False)])
def test_ssm_dense(t, b, s, c, n, groups, dtype, state, gated, soft):
    i = ssm_inputs(t, b, b, s, c, n, groups, dtype, 21, state, gated)
    if not soft:                        # steps as they are: make them positive and small
        i["dt"] = [(x.abs() * 0.1) for x in i["dt"]]
        i["dt_bias"] = None
    o = run_ssm(i, b, None, state, soft)
    check_ssm(i, o, None, state, soft)
    assert same_runs(o, run_ssm(i, b, None, state, soft))
    # without saving states, which few tokens' own form takes
    f = run_ssm(i, b, None, state, soft, back=False)
    check_ssm(i, f, None, state, soft)


@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
@pytest.mark.parametrize("dtype,c,n,groups,state,gated", [
    (BF, 72, 16, 1, True, True), (F32, 32, 8, 2, True, False), (FP, 40, 32, 1, False, True),
    (BF, 16, 64, 2, True, True)])
def test_ssm_packed(lens, dtype, c, n, groups, state, gated):
    m, s = len(lens), sum(lens)
    i = ssm_inputs(2, m, 1, s, c, n, groups, dtype, 22, state, gated)
    o = run_ssm(i, m, offsets(lens), state)
    check_ssm(i, o, lens, state, ranks=1)


@pytest.mark.parametrize("lens", [None, [1, 700, 0, 15, 17, 1276], [2009]], ids=["dense", "q6", "q1"])
@pytest.mark.parametrize("dtype,t,c,n", [(BF, 1, 72, 16), (FP, 1, 8, 64), (F32, 2, 24, 8), (F32, 1, 40, 32)])
def test_ssm_few_channels(lens, dtype, t, c, n):
    """Long sequences of few channels, cut into chunks that run side by side."""
    m, s = (1, 2009) if lens is None else (len(lens), 2009)
    assert sp.sp_selective_scan_fwd_workspace_bytes(1, s, c, n, 1, t) > 0
    i = ssm_inputs(t, m, 1, s, c, n, 1, dtype, 23 + c, True)
    check_ssm(i, run_ssm(i, m, None if lens is None else offsets(lens), True), lens, True, ranks=1)


def test_ssm_no_token():
    """s == 0 and packed sequences that are all empty: states and their gradients pass."""
    for cu, b, m in ((None, 3, 3), (torch.zeros(5, dtype=torch.int32, device=DEV), 1, 4)):
        i = ssm_inputs(2, m, b, 0, 16, 16, 1, BF, 24, True)
        o = run_ssm(i, m, cu, True)
        assert same(o["hT"], i["h0"]) and same(o["dh0"], i["dhT"])
        assert all((o[k] == 0).all() for k in ("dA", "dD", "ddt_bias"))
        c = conv_inputs(2, m, b, 0, 16, 4, BF, 24, True)
        o = run_conv(c, m, "silu", cu, True)
        assert same(o["xT"], c["x0"]) and same(o["dx0"], c["dxT"])
        assert (o["dweight"] == 0).all() and (o["dbias"] == 0).all()


def test_ssm_optional_arguments():
    """Without D, bias, states and parameter gradients; B and C shared by the ranks."""
    i = ssm_inputs(2, 2, 2, 40, 48, 16, 2, BF, 25, False)
    i["D"] = i["dt_bias"] = None
    i["dt"] = [x - 3 for x in i["dt"]]
    i["B"], i["C"] = [i["B"][0]] * 2, [i["C"][0]] * 2
    o = run_ssm(i, 2, None, False)
    check_ssm(i, o, None, False)
    got = {k: nans(2, o[k][0].shape, BF) for k in ("du", "ddt", "dB", "dC", "dz")}
    sp.sp_selective_scan_bwd(i["u"], i["dt"], i["A"], i["B"], i["C"], o["states"], i["dy"], z=i["z"],
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(2, 40, 48, 16, 2, 2)), **got)
    assert all(same(got[k], o[k]) for k in got)


@pytest.mark.parametrize("n", [8, 16, 32, 64])
def test_ssm_decoding_follows_the_prompt(n):
    """A prompt, then tokens one to four at a time with the state updated in place."""
    i = ssm_inputs(2, 9, 9, 60, 72, n, 1, F32, 26, True)
    want = run_ssm(i, 9, None, True, back=False)
    state = [v.clone() for v in i["h0"]]
    parts = [[] for _ in range(2)]
    cut = lambda k, lo, hi: None if i[k] is None else [v[:, lo:hi].contiguous() for v in i[k]]
    for lo, hi in ((0, 49), (49, 50), (50, 54), (54, 57), (57, 57), (57, 59), (59, 60)):
        y = nans(2, (9, hi - lo, 72), F32)
        sp.sp_selective_scan_fwd(cut("u", lo, hi), cut("dt", lo, hi), i["A"], cut("B", lo, hi),
                                 cut("C", lo, hi), D=i["D"], z=cut("z", lo, hi), dt_bias=i["dt_bias"],
                                 h0=state, y=y, hT=state)
        for p, v in zip(parts, y):
            p.append(v)
    got = dict(y=[torch.cat(p, 1) for p in parts], hT=state)
    check_ssm(i, got, None, True)
    check_ssm(i, want, None, True)


def test_ssm_packed_states_in_place():
    """hT over h0 where few channels' chunks would run side by side."""
    lens = [5, 0, 900, 1, 700, 394]
    i = ssm_inputs(1, 6, 1, 2000, 16, 16, 1, BF, 27, True)
    want = run_ssm(i, 6, offsets(lens), True, back=False)
    check_ssm(i, want, lens, True)
    state = [i["h0"][0].clone()]
    y = nans(1, (1, 2000, 16), BF)
    ws = scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, 2000, 16, 16, 1, 1))
    sp.sp_selective_scan_fwd(i["u"], i["dt"], i["A"], i["B"], i["C"], D=i["D"], z=i["z"], dt_bias=i["dt_bias"],
                             h0=state, cu_seqlens=offsets(lens), y=y, hT=state, workspace=ws)
    check_ssm(i, dict(y=y, hT=state), lens, True)


def test_ssm_strided_rows():
    """Slices of wider rows in and out; the rest stays."""
    i = ssm_inputs(1, 2, 2, 37, 64, 16, 1, BF, 28, True)
    want = run_ssm(i, 2, None, True)
    wide = torch.full((2, 37, 5 * 72), 7.0, dtype=BF, device=DEV)
    at = lambda k, w=64: wide[..., 72 * k:72 * k + w]
    u, y, du, ddt, dz = (at(k) for k in range(5))
    narrow = torch.full((2, 37, 2 * 24), 7.0, dtype=BF, device=DEV)
    dB, dC = narrow[..., :16], narrow[..., 24:40]
    u.copy_(i["u"][0])
    how = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], h0=i["h0"])
    states = nans(1, sp.sp_selective_scan_states_shape(2, 37, 64, 16), F32)
    sp.sp_selective_scan_fwd([u], i["dt"], i["A"], i["B"], i["C"], y=[y], states=states, **how)
    sp.sp_selective_scan_bwd([u], i["dt"], i["A"], i["B"], i["C"], states, i["dy"], dhT=i["dhT"], du=[du],
                             ddt=[ddt], dB=[dB], dC=[dC], dz=[dz],
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(2, 37, 64, 16, 1, 1)), **how)
    assert same([y, du, ddt, dz, dB, dC], [want[k][0] for k in ("y", "du", "ddt", "dz", "dB", "dC")])
    assert (wide.unflatten(2, (5, 72))[..., 64:] == 7).all() and (narrow[..., 16:24] == 7).all()
    assert (narrow[..., 40:] == 7).all()


@pytest.mark.parametrize("c", [8, 4096])
def test_ssm_what_is_not_finite_stays_in_its_sequence(c):
    """An infinity or a NaN of one sequence: the others' outputs keep their bits."""
    lens = [20, 0, 500, 33, 100]
    i = ssm_inputs(1, 5, 1, 653, c, 16, 1, BF, 29, True)
    cu = offsets(lens)
    clean = run_ssm(i, 5, cu, True)
    for value in (NAN, float("inf")):
        i2 = {k: [x.clone() for x in v] if isinstance(v, list) else v for k, v in i.items()}
        i2["h0"][0][2] = value
        i2["u"][0][0, 300] = value
        o = run_ssm(i2, 5, cu, True)
        keep = torch.ones(653, dtype=torch.bool, device=DEV)
        keep[20:520] = False
        for k in ("y", "du", "ddt", "dz", "dB", "dC"):
            assert torch.equal(bits(o[k][0][0, keep]), bits(clean[k][0][0, keep])), k
        for k in ("hT", "dh0"):
            assert torch.equal(bits(o[k][0][[0, 1, 3, 4]]), bits(clean[k][0][[0, 1, 3, 4]])), k
        assert not torch.isfinite(o["y"][0][0, 300:520]).any()


BEGINNINGS = [1, 2, 5, 16, 0, 16, 3, 40, 1, 1, 130, 7, 8, 8, 17]


@pytest.mark.parametrize("dtype,c,n,groups", [(BF, 72, 16, 1), (F32, 64, 8, 2), (FP, 48, 32, 1), (BF, 24, 64, 1),
                                              (F32, 136, 16, 1), (FP, 640, 16, 1)])
@pytest.mark.parametrize("gated", [True, False])
def test_ssm_packed_from_zeros(dtype, c, n, groups, gated):
    """Sequences that begin anywhere in a run of 16 tokens, several in one, without states."""
    lens = BEGINNINGS
    i = ssm_inputs(2, len(lens), 1, sum(lens), c, n, groups, dtype, 44, False, gated)
    o = run_ssm(i, len(lens), offsets(lens), False)
    check_ssm(i, o, lens, False)
    assert same_runs(o, run_ssm(i, len(lens), offsets(lens), False))


@pytest.mark.parametrize("which", ["dhT", "h0"])
def test_ssm_packed_with_one_kind_of_state(which):
    """Only the gradient of the last states, or only the first states."""
    lens = BEGINNINGS
    i = ssm_inputs(1, len(lens), 1, sum(lens), 40, 16, 1, F32, 45, True)
    if which == "dhT":
        i["h0"] = None
    else:
        i["dhT"] = None
    check_ssm(i, run_ssm(i, len(lens), offsets(lens), True), lens, True)


@pytest.mark.parametrize("c", [8, 4096])
def test_ssm_what_is_not_finite_stays_without_states(c):
    lens = [20, 0, 500, 33, 100]
    cu = offsets(lens)
    i = ssm_inputs(1, 5, 1, 653, c, 16, 1, BF, 46, False)
    clean = run_ssm(i, 5, cu, False)
    keep = torch.ones(653, dtype=torch.bool, device=DEV)
    keep[20:520] = False
    for value in (NAN, float("inf")):
        i2 = {k: [x.clone() for x in v] if isinstance(v, list) else v for k, v in i.items()}
        i2["u"][0][0, 300] = value
        i2["dy"][0][0, 400] = value
        o = run_ssm(i2, 5, cu, False)
        for k in ("y", "du", "ddt", "dz", "dB", "dC"):
            assert torch.equal(bits(o[k][0][0, keep]), bits(clean[k][0][0, keep])), k
        assert not torch.isfinite(o["y"][0][0, 300:520]).any()


def test_ssm_states_that_grow_behind_padding():
    """A > 0: a chunk's decay overflows while the state that enters it is still zero.
    A decay of d A = 1 is off by at most 2^-19 of itself, so 20 tokens' product by 2^-14,
    inside check_ssm's bound of 2^-9."""
    i = ssm_inputs(1, 1, 1, 2048, 16, 16, 1, F32, 33, False, gated=False)
    i["A"] = i["A"].abs() * 0 + 1
    i["dt"], i["dt_bias"] = [torch.full_like(x, 0.5) for x in i["dt"]], None
    i["u"][0][:, :-20] = 0
    o = run_ssm(i, 1, None, False, back=False)
    assert torch.isfinite(o["y"][0]).all() and (o["y"][0][:, :-20] == 0).all()
    check_ssm(i, o, None, False)


def test_ssm_small_states_that_grow():
    """The same from a first state of 2^-100: d A = 0.1 a token, so e^204.8 2^-100 = 2^195
    is too much for float32, but not before token 1580; compared are 1500.  Each decay is
    off by 2^-22.8 and the rounding of d A, below 0.1 2^-23: 1500 tokens 2^-12."""
    i = ssm_inputs(1, 1, 1, 2048, 16, 16, 1, F32, 34, True, gated=False)
    i["A"] = i["A"].abs() * 0 + 0.1
    i["dt"], i["dt_bias"] = [torch.ones_like(x) for x in i["dt"]], None
    i["u"][0].zero_()
    i["h0"][0].fill_(2.0 ** -100)
    i["C"] = [torch.full_like(x, 1 / 16) for x in i["C"]]
    y = f64(run_ssm(i, 1, None, True, soft=False, back=False)["y"][0])[0, :1500]
    want = 2.0 ** -100 * np.exp(0.1 * np.arange(1, 1501))[:, None]
    assert (np.abs(y - want) <= 2.0 ** -11 * want).all()


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("s", [1, 3, 600])
def test_ssm_masked_tokens(dtype, s):
    """Steps of -infinity or of the type's lowest value: such a token leaves the state as
    it is, takes no part of u, and every gradient is finite."""
    i = ssm_inputs(2, 2, 2, s, 72, 16, 1, dtype, 35, True)
    for x in i["dt"]:
        x[0, : (s + 1) // 2] = -float("inf")
        x[1, s // 2:] = torch.finfo(dtype).min
    o = run_ssm(i, 2, None, True)
    check_ssm(i, o, None, True)
    assert all((o["ddt"][r][0, : (s + 1) // 2] == 0).all() for r in range(2))
    check_ssm(i, run_ssm(i, 2, None, True, back=False), None, True)


def test_sixteen_ranks():
    """The most ranks, with every argument."""
    i = ssm_inputs(16, 2, 2, 33, 16, 16, 2, BF, 36, True)
    check_ssm(i, run_ssm(i, 2, None, True), None, True)
    c = conv_inputs(16, 3, 1, 50, 16, 4, BF, 36, True)
    check_conv(c, run_conv(c, 3, "silu", offsets([20, 2, 28]), True), "silu", [20, 2, 28], True)


def test_long_memory_keeps_its_digits():
    """Steps near 0.001: states that gather over thousands of tokens, in norm."""
    i = ssm_inputs(1, 1, 1, 6000, 64, 16, 1, F32, 30, True)
    i["dt"] = [x * 0.1 for x in i["dt"]]
    i["dt_bias"] = torch.full((64,), -6.9, device=DEV)
    o = run_ssm(i, 1, None, True)
    w = orc.selective_scan(*(f64(i[k][0]) if isinstance(i[k], list) else f64(i[k]) for k in ("u", "dt", "A", "B", "C")),
                           f64(i["D"]), f64(i["z"][0]), f64(i["dt_bias"]), True, f64(i["h0"][0]), None,
                           f64(i["dy"][0]), f64(i["dhT"][0]))
    # a decay is off by at most 2^-22.8 whatever its step: over the memory of 1 / (0.001
    # 0.16) = 6000 tokens at most 8e-4, to one side; the states' norm is that of channels
    # of all memories, and the error of a decay is mostly its rounding: 2^-13 holds both
    for k in ("y", "hT", "du", "ddt", "dB", "dC", "dA", "dh0", "dz"):
        got, want = f64(o[k][0] if isinstance(o[k], list) else o[k]), w[k]
        assert np.linalg.norm(got - want) <= 2.0 ** -13 * np.linalg.norm(want), k


def test_many_sequences():
    """More packed sequences than one search step reaches, many of them empty."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, size=2100).tolist()
    s = sum(lens)
    i = ssm_inputs(1, 2100, 1, s, 8, 8, 1, F32, 31, True)
    check_ssm(i, run_ssm(i, 2100, offsets(lens), True), lens, True)
    c = conv_inputs(1, 2100, 1, s, 8, 4, F32, 31, True)
    check_conv(c, run_conv(c, 2100, "silu", offsets(lens), True), "silu", lens, True)


def test_bad_prefix_sums_are_reported():
    """Prefix sums that fall, start late or end early: the status word says so, nothing
    outside the buffers is written (guards around the outputs stay)."""
    own = torch.zeros(1, dtype=torch.int32, device=DEV)
    i = ssm_inputs(1, 3, 1, 90, 16, 16, 1, BF, 32, True)
    c = conv_inputs(1, 3, 1, 90, 16, 4, BF, 32, True)
    for cu in ([0, 50, 20, 90], [5, 10, 20, 90], [0, 10, 20, 60], [0, 10, 200, 90], [-7, 10, 20, 90]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        guard = torch.full((1, 90, 32), 7.0, dtype=BF, device=DEV)
        y = [guard[..., 8:24]]
        for call in (lambda: sp.sp_selective_scan_fwd(i["u"], i["dt"], i["A"], i["B"], i["C"], h0=i["h0"],
                                                      cu_seqlens=cu, y=y, hT=nans(1, (3, 16, 16), F32), status=own),
                     lambda: sp.sp_causal_conv_fwd(c["x"], c["weight"], c["bias"], x0=c["x0"], cu_seqlens=cu, y=y,
                                                   xT=nans(1, (3, 3, 16), BF), status=own),
                     lambda: sp.sp_causal_conv_bwd(c["x"], c["weight"], c["bias"], c["dy"], x0=c["x0"],
                                                   dxT=c["dxT"], cu_seqlens=cu, dx=y, dx0=nans(1, (3, 3, 16), BF),
                                                   status=own)):
            own.zero_()
            call()
            assert own.item() == 6          # SP_ERR_DEVICE_CHECK
            assert (guard[..., :8] == 7).all() and (guard[..., 24:] == 7).all()


@pytest.mark.parametrize("state", [True, False])
def test_bad_prefix_sums_of_the_scan_and_its_gradients(state):
    """The same for the backward, and where sequences have no states."""
    own = torch.zeros(1, dtype=torch.int32, device=DEV)
    i = ssm_inputs(1, 3, 1, 600, 16, 16, 1, BF, 47, state)
    A, B, C = i["A"], i["B"], i["C"]
    for cu in ([0, 50, 20, 600], [5, 10, 20, 600], [0, 10, 20, 60], [0, 10, 900, 600], [-7, 10, 20, 600]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        guard = torch.full((1, 600, 4 * 32), 7.0, dtype=BF, device=DEV)
        y, du, ddt, dz = ([guard[..., 32 * k + 8:32 * k + 24]] for k in range(4))
        saved = nans(1, sp.sp_selective_scan_states_shape(1, 600, 16, 16), F32)
        m = lambda: nans(1, (3, 16, 16), F32) if state else None
        how = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], h0=i["h0"], cu_seqlens=cu, status=own)
        sp.sp_selective_scan_fwd(i["u"], i["dt"], A, B, C, y=y, hT=m(), states=saved, **how,
                                 workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, 600, 16, 16, 1, 1)))
        assert own.item() == 6
        own.zero_()
        sp.sp_selective_scan_bwd(i["u"], i["dt"], A, B, C, saved, i["dy"], dhT=i["dhT"], du=du, ddt=ddt, dz=dz,
                                 dB=nans(1, (1, 600, 16), BF), dC=nans(1, (1, 600, 16), BF), dh0=m(), **how,
                                 workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(1, 600, 16, 16, 1, 1)))
        assert own.item() == 6
        own.zero_()
        around = guard.view(1, 600, 4, 32)
        assert (around[..., :8] == 7).all() and (around[..., 24:] == 7).all()


# ----------------------------------------------------------------- together --

def layer(x, p, cu):
    """A state space layer of one rank as it is used between g and the next g*:
    projections -> convolution -> scan with its gate -> norm of the heads, forward and
    backward (gradient of the output = the output)."""
    e = lambda shape, dt=BF: torch.empty(shape, dtype=dt, device=DEV)
    _, s, _ = x.shape
    c, n = p["A"].shape
    proj = x @ p["w"]                                    # x, z, dt, B, C side by side
    xin, z, dt = (proj[..., k * c:(k + 1) * c] for k in range(3))
    B, C = proj[..., 3 * c:3 * c + n], proj[..., 3 * c + n:]
    u, y, states = e((1, s, c)), e((1, s, c)), e(sp.sp_selective_scan_states_shape(1, s, c, n), F32)
    sp.sp_causal_conv_fwd([xin], p["conv"], p["bias"], act="silu", cu_seqlens=cu, y=[u])
    scan = ([u], [dt], p["A"], [B], [C])
    how = dict(D=p["D"], z=[z], dt_bias=p["dt_bias"], cu_seqlens=cu)
    sp.sp_selective_scan_fwd(*scan, y=[y], states=[states],
                             workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, s, c, n, 1, 1)), **how)
    out, rstd = e((s, 1, c)), e((s, 2), F32)
    sp.sp_group_norm_fwd([y.view(s, 1, c)], p["gamma"], groups=2, norm="rmsnorm", eps=1e-5, y=[out], rstd=[rstd])
    dy, dproj, du = e((s, 1, c)), e((1, s, 3 * c + 2 * n)), e((1, s, c))
    grads = {k: e(p[k].shape, F32) for k in ("A", "D", "dt_bias", "conv", "bias", "gamma")}
    sp.sp_group_norm_bwd([out], [y.view(s, 1, c)], None, [rstd], p["gamma"], groups=2, norm="rmsnorm", dx=[dy],
                         dgamma=grads["gamma"],
                         workspace=scratch(sp.sp_group_norm_bwd_workspace_bytes(s, 1, c, 2, 1)))
    sp.sp_selective_scan_bwd(*scan, [states], [dy.view(1, s, c)], du=[du], ddt=[dproj[..., 2 * c:3 * c]],
                             dB=[dproj[..., 3 * c:3 * c + n]], dC=[dproj[..., 3 * c + n:]],
                             dz=[dproj[..., c:2 * c]], dA=grads["A"], dD=grads["D"], ddt_bias=grads["dt_bias"],
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(1, s, c, n, 1, 1)), **how)
    sp.sp_causal_conv_bwd([xin], p["conv"], p["bias"], [du], act="silu", cu_seqlens=cu, dx=[dproj[..., :c]],
                          dweight=grads["conv"], dbias=grads["bias"],
                          workspace=scratch(sp.sp_causal_conv_bwd_workspace_bytes(1, s, c, 4, 1)))
    return dict(out=out, dproj=dproj, **grads)


def layer_float(proj, p, cu):
    """The same in float64 torch operations, differentiable."""
    c, n = p["A"].shape
    s = proj.shape[0]
    xin, z, dt = (proj[:, k * c:(k + 1) * c] for k in range(3))
    B, C = proj[:, 3 * c:3 * c + n], proj[:, 3 * c + n:]
    rows = []
    for lo, hi in zip(cu, cu[1:]):
        xs = torch.cat((torch.zeros(3, c, dtype=torch.float64), xin[lo:hi]))
        h = torch.zeros(c, n, dtype=torch.float64)
        for i in range(hi - lo):
            q = (xs[i:i + 4] * p["conv"].t()).sum(0) + p["bias"]
            u = q * torch.sigmoid(q)
            d = torch.nn.functional.softplus(dt[lo + i] + p["dt_bias"], threshold=100.0)
            h = torch.exp(d[:, None] * p["A"]) * h + (d * u)[:, None] * B[lo + i]
            rows.append(((h * C[lo + i]).sum(-1) + p["D"] * u) * z[lo + i] * torch.sigmoid(z[lo + i]))
    y = torch.stack(rows).view(s, 2, c // 2)
    out = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-5)
    return out.reshape(s, c) * p["gamma"]


def layer_params(c, n, gen):
    p = dict(w=rand((256, 3 * c + 2 * n), gen, BF, 1 / 16), conv=rand((c, 4), gen, BF, 0.5),
             bias=rand((c,), gen, BF, 0.1), gamma=rand((c,), gen, BF, 0.1, 1.0), D=rand((c,), gen, F32),
             dt_bias=rand((c,), gen, F32, 0.5, -2.0), A=-torch.exp(rand((c, n), gen, F32, 0.5)))
    return p


def test_layer_and_its_graph():
    """The operators after each other as a layer uses them, on a side stream and replayed
    from a CUDA graph; forward and gradients against float64."""
    gen = torch.Generator().manual_seed(41)
    cu_np = [0, 21, 21, 22, 96]
    cu = torch.tensor(cu_np, dtype=torch.int32, device=DEV)
    p, x = layer_params(64, 16, gen), rand((1, 96, 256), gen, BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(x, p, cu)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = layer(x, p, cu)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert same_runs(got, kept)
    q = {k: v.double().cpu().requires_grad_(True) for k, v in p.items()}
    proj = (x @ p["w"])[0].double().cpu().requires_grad_(True)
    out = layer_float(proj, q, cu_np)
    (out * got["out"][:, 0].double().cpu()).sum().backward()
    # bf16 rounds each of up to six values in a row, 2^-8 each, against the norm of the result
    pairs = [(got["out"][:, 0], out.detach()), (got["dproj"][0], proj.grad)]
    pairs += [(got[k], q[k].grad) for k in ("A", "D", "dt_bias", "conv", "bias", "gamma")]
    for k, (a, b) in enumerate(pairs):
        assert (a.double().cpu() - b).norm() < 6 * 2.0 ** -8 * b.norm(), k


def test_layer_decodes_in_a_graph():
    """A prompt through the convolution and the scan, then tokens one by one from a captured
    step that keeps its states in place: as one call over all tokens.  Both round u and y to
    bf16 once and differ before that by the arithmetic, 2^-15 of a magnitude of at most 16
    times the result in norm: 2 2^-8 + 2^-10 < 3 2^-8."""
    t, b, s, c, n, prompt = 2, 3, 40, 64, 16, 29
    gen = torch.Generator().manual_seed(42)
    i = ssm_inputs(t, b, b, s, c, n, 1, BF, 43, False)
    x = [rand((b, s, c), gen, BF) for _ in range(t)]
    weight, bias = rand((t * c, 4), gen, BF, 0.5), rand((t * c,), gen, BF, 0.1)
    how = dict(D=i["D"], dt_bias=i["dt_bias"])

    def run(x, dt, z, B, C, x0, h0, xT, hT):
        u, y = nans(t, x[0].shape, BF), nans(t, x[0].shape, BF)
        sp.sp_causal_conv_fwd(x, weight, bias, act="silu", x0=x0, y=u, xT=xT)
        ws = scratch(sp.sp_selective_scan_fwd_workspace_bytes(b, x[0].shape[1], c, n, 1, t))
        sp.sp_selective_scan_fwd(u, dt, i["A"], B, C, z=z, h0=h0, y=y, hT=hT, workspace=ws, **how)
        return y

    rows = [x, i["dt"], i["z"], i["B"], i["C"]]
    piece = lambda lo, hi: [[r[:, lo:hi].contiguous() for r in k] for k in rows]
    xT, hT = nans(t, (b, 3, c), BF), nans(t, (b, c, n), F32)
    want = run(*piece(0, s), None, None, nans(t, (b, 3, c), BF), nans(t, (b, c, n), F32))
    got = [[y] for y in run(*piece(0, prompt), None, None, xT, hT)]
    token = piece(prompt, prompt + 1)
    before = [v.clone() for v in xT + hT]
    run(*token, xT, hT, xT, hT)                          # (a first call outside the capture)
    for v, k in zip(xT + hT, before):
        v.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(*token, xT, hT, xT, hT)
    for k in range(prompt, s):
        for have, new in zip(token, piece(k, k + 1)):
            for a, v in zip(have, new):
                a.copy_(v)
        graph.replay()
        for r in range(t):
            got[r].append(y[r].clone())
    for r in range(t):
        a, w = torch.cat(got[r], 1).double(), want[r].double()
        assert (a - w).norm() < 3 * 2.0 ** -8 * w.norm(), r


def test_layer_over_ranks_is_each_rank():
    """Eight ranks in one call give the bits of eight calls."""
    i = ssm_inputs(8, 2, 2, 70, 24, 16, 1, BF, 42, True)
    o = run_ssm(i, 2, None, True)
    c = conv_inputs(8, 2, 2, 70, 24, 4, BF, 42, True)
    w = run_conv(c, 2, "silu", None, True)
    for r in (0, 5, 7):
        p = slice(r * 24, (r + 1) * 24)
        one = {k: [v[r]] if isinstance(v, list) else v[p] if v is not None else None for k, v in i.items()}
        a = run_ssm(one, 2, None, True)
        for k in ("y", "du", "ddt", "dz", "dB", "dC", "hT", "dh0"):
            assert same([a[k][0]], [o[k][r]]), k
        one = {k: [v[r]] if isinstance(v, list) else v[p] for k, v in c.items()}
        a = run_conv(one, 2, "silu", None, True)
        for k in ("y", "dx", "xT", "dx0"):
            assert same([a[k][0]], [w[k][r]]), k


def test_two_streams_at_once():
    """Two calls of every operator that may overlap on the device, a workspace each."""
    a, b = (ssm_inputs(1, 1, 1, 1500, 64, 16, 1, BF, k, True) for k in (43, 44))
    p, q = (conv_inputs(1, 1, 1, 1500, 64, 4, BF, k, True) for k in (43, 44))
    want = [run_ssm(v, 1, None, True) for v in (a, b)], [run_conv(v, 1, "silu", None, True) for v in (p, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [], []
        for st, v, w in zip(streams, (a, b), (p, q)):
            with torch.cuda.stream(st):
                got[0].append(run_ssm(v, 1, None, True))
                got[1].append(run_conv(w, 1, "silu", None, True))
        torch.cuda.synchronize()
        for g, w in zip(got[0] + got[1], want[0] + want[1]):
            assert same_runs(g, w)


class LongWay:
    """The compiled short way, taking nothing."""
    def __getattr__(self, name):
        return lambda *args: None


def test_short_and_long_way_agree(monkeypatch):
    quick = sp._quick()
    cu = offsets([5, 0, 35])
    i = ssm_inputs(2, 3, 1, 40, 72, 16, 1, FP, 45, True)
    d = ssm_inputs(2, 2, 2, 20, 16, 8, 2, F32, 46, False, False)
    c, e = conv_inputs(2, 3, 1, 40, 72, 4, FP, 45, True), conv_inputs(2, 2, 2, 9, 8, 3, F32, 46, False)
    e["bias"] = None
    x = [rand((2, 5, 3, 32), torch.Generator().manual_seed(99), F32)]
    pos = torch.arange(20, device=DEV).view(2, 2, 5)
    tab = sp.sp_rope_axes_table([4, 4])

    def everything():
        y = nans(1, (2, 5, 3, 32), F32)
        sp.sp_rope_axes_bwd(x, tab, positions=pos, layout="interleaved", dx=y)
        o = y
        for r in (run_ssm(i, 3, cu, True), run_ssm(d, 2, None, False), run_conv(c, 3, "silu", cu, True),
                  run_conv(e, 2, "none", None, False)):
            o += list(tensors(r).values())
        return o

    a = everything()
    monkeypatch.setattr(sp, "_module", LongWay())
    b = everything()
    assert same(a, b)
    monkeypatch.setattr(sp, "_module", quick)
    with pytest.raises(ValueError):
        sp.sp_rope_axes_fwd(x, tab, positions=pos.int(), y=x)
    with pytest.raises(ValueError):
        sp.sp_causal_conv_fwd(c["x"], c["weight"][:-1], y=c["x"])
    with pytest.raises(ValueError):
        sp.sp_selective_scan_fwd(i["u"], i["dt"], i["A"].half(), i["B"], i["C"], y=i["dy"])
    with pytest.raises(sp.SpError, match="workspace"):
        sp.sp_selective_scan_fwd(*(rand_long(2000, 8)), y=nans(1, (1, 2000, 8), BF))


def rand_long(s, c):
    i = ssm_inputs(1, 1, 1, s, c, 16, 1, BF, 47, False)
    return i["u"], i["dt"], i["A"], i["B"], i["C"]


def test_offsets_beyond_32_bits():
    """Rows so far apart that elements and bytes pass 2^32: the same bits as dense rows."""
    rows, ld = 4400, 1 << 20
    wide = torch.empty(rows * ld, dtype=BF, device=DEV)        # 9.2 GB
    gen = torch.Generator().manual_seed(91)
    at = iter(range(0, ld, 1024))

    def far(x):
        b, s, c = x.shape
        v = wide.as_strided((b, s, c), (s * ld, ld, 1), next(at))
        v.copy_(x)
        return v

    x = rand((1, rows, 3 * 64), gen, BF)
    y, v, w = torch.empty_like(x), far(x), far(torch.zeros_like(x))
    heads = lambda z: [z.unflatten(2, (3, 64))]
    pos = torch.randint(0, 1 << 30, (2, 1, rows), generator=gen).to(DEV)
    tab = sp.sp_rope_axes_table([10, 14])
    sp.sp_rope_axes_fwd(heads(x), tab, positions=pos, y=heads(y))
    sp.sp_rope_axes_fwd(heads(v), tab, positions=pos, y=heads(w))
    assert same([y], [w])
    for lens in (None, [7, 3993, 400]):
        m, cu = (1, None) if lens is None else (3, offsets(lens))
        c = conv_inputs(1, m, 1, rows, 72, 4, BF, 92, True)
        want = run_conv(c, m, "silu", cu, True)
        c.update({k: [far(c[k][0])] for k in ("x", "dy")})
        y, dx = [far(torch.zeros_like(c["x"][0]))], [far(torch.zeros_like(c["x"][0]))]
        how = dict(act="silu", x0=c["x0"], cu_seqlens=cu)
        sp.sp_causal_conv_fwd(c["x"], c["weight"], c["bias"], y=y, **how)
        sp.sp_causal_conv_bwd(c["x"], c["weight"], c["bias"], c["dy"], dxT=c["dxT"], dx=dx, **how)
        assert same(y, want["y"]) and same(dx, want["dx"])
        i = ssm_inputs(1, m, 1, rows, 72, 16, 1, BF, 93, True)
        want = run_ssm(i, m, cu, True)
        i.update({k: [far(i[k][0])] for k in ("u", "dt", "B", "C", "z", "dy")})
        o = {k: [far(torch.zeros_like(want[k][0]))] for k in ("y", "du", "ddt", "dz", "dB", "dC")}
        args = (i["u"], i["dt"], i["A"], i["B"], i["C"])
        how = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], h0=i["h0"], cu_seqlens=cu)
        states = nans(1, sp.sp_selective_scan_states_shape(1, rows, 72, 16), F32)
        sp.sp_selective_scan_fwd(*args, y=o["y"], states=states,
                                 workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, rows, 72, 16, 1, 1)), **how)
        sp.sp_selective_scan_bwd(*args, states, i["dy"], dhT=i["dhT"], du=o["du"], ddt=o["ddt"], dB=o["dB"],
                                 dC=o["dC"], dz=o["dz"],
                                 workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(1, rows, 72, 16, 1, 1)), **how)
        for k in o:
            assert same(o[k], want[k]), k
