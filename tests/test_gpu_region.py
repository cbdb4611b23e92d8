"""The operators between g and the next g* on the GPU against the float64 oracle.

Tolerances.  An output of type T is its exact value rounded once, off by at most
u |exact| with u = 2^-8 (bf16), 2^-11 (fp16; plus 2^-25, half the smallest
subnormal), 2^-24 (float32), plus what the float32 arithmetic before it loses,
a multiple of 2^-24 of the magnitude that the oracle returns beside the value:

- rotary, 2^-21 (|u| + |v|) mscale: the half-turns fraction is off by 2^-25 + 2^-31
  (pi times that in radians), sincospif by an ulp, mscale, its products with cosine
  and sine, two products and a sum by a rounding each: under 8 units of 2^-24.
- recurrence, (2^-18 + n 2^-22) max |h| over n tokens: a gate's exponential is off by
  2^-22 plus the rounding of g log2(e), 24 2^-24 for |g| <= 16; the reciprocal adds
  2^-23; k [or a] scales the new term, so the state keeps at most 2^-19 of the
  magnitude from it, and each token adds at most 3 roundings to the state and one to
  each of the products of factors that carry it from run to run: n 2^-22.
  dgate is a product of a state, a gradient and a k: three times that.
- group norm, 2^-15 of (|x| + |mean|) rstd |gamma| + |beta|: sums of at most 64
  values in a row, then 6 + 16 + 16 partial sums: below 2^7 roundings, 2^-17, of the
  mean magnitude in the mean and as much in the variance; 2^-13 for the backward,
  whose products hold two such sums.  dgamma and dbeta add up to 2^9 terms in a row
  per thread and block: 2^-14 of the sum of magnitudes.
"""
import itertools
import numpy as np
import pytest
import torch

from oracle import region as orc
from sp_boundary_norm_gb300 import binding as sp

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 0.0, FP: 2.0 ** -25, F32: 0.0}


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


def rand(shape, gen, dtype, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, dtype=torch.float32) * scale + shift
    return x.to(dtype).to(DEV)


def f64(x):
    return x.double().cpu().numpy()


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
    return all(torch.equal(bits(p), bits(q)) for p, q in zip(a, b))


# ------------------------------------------------------------------ rotary --

ROPE = [
    # t, b, s, heads, d, rot, layout, dtype
    (1, 1, 1, 1, 2, 2, "half", F32),
    (1, 1, 1, 1, 8, 2, "interleaved", BF),
    (2, 3, 5, 7, 64, 64, "half", BF),
    (2, 2, 33, 3, 128, 128, "interleaved", BF),
    (8, 1, 17, 9, 128, 128, "half", FP),
    (1, 2, 9, 5, 80, 20, "interleaved", FP),
    (1, 2, 9, 5, 80, 20, "half", FP),
    (3, 1, 4, 2, 96, 48, "half", F32),
    (1, 1, 3, 1, 512, 512, "half", F32),
    (1, 1, 3, 1, 520, 512, "interleaved", F32),
    (2, 1, 6, 4, 14, 6, "half", BF),
    (2, 1, 6, 4, 15, 6, "interleaved", BF),
    (1, 1, 2, 33, 40, 24, "half", BF),
    (16, 1, 2, 70, 16, 16, "half", BF),
]


@pytest.mark.parametrize("t,b,s,heads,d,rot,layout,dtype", ROPE)
@pytest.mark.parametrize("back", [False, True])
def test_rope(t, b, s, heads, d, rot, layout, dtype, back):
    gen = torch.Generator().manual_seed(7)
    x = [rand((b, s, heads, d), gen, dtype) for _ in range(t)]
    y = [torch.full_like(q, float("nan")) for q in x]
    tab = sp.sp_rope_table(rot, base=10000.0, mscale=1.1)
    freq = orc.frequencies(rot)
    fn = (lambda out: sp.sp_rope_bwd(x, tab, layout=layout, first_position=123456, dx=out)) if back \
        else (lambda out: sp.sp_rope_fwd(x, tab, layout=layout, first_position=123456, y=out))
    fn(y)
    m = float(np.float32(1.1))
    for r in range(t):
        want, mag = orc.rope(f64(x[r]), orc.positions(b, s, 123456), freq, layout, m, back)
        close(y[r], want, mag, 2.0 ** -21, f"rank {r}")
        assert torch.equal(bits(y[r][..., rot:]), bits(x[r][..., rot:]))
    again = [torch.empty_like(q) for q in x]
    fn(again)
    assert same(y, again)
    fn(x)                                    # in place
    assert same(y, x)


@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=4.0)),
    ("parts", dict(factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0, mscale=1.25))])
def test_rope_far_positions(scaling, kw):
    """Positions up to 2^40 and below zero, scaled frequencies."""
    gen = torch.Generator().manual_seed(8)
    x = [rand((4, 5, 2, 64), gen, F32)]
    y = [torch.empty_like(x[0])]
    pos = torch.tensor([0, 1, -1, 2 ** 31, 2 ** 40, -2 ** 33, 131071, 999983, 2 ** 24 + 1, 77] * 2)
    tab = sp.sp_rope_table(64, base=500000.0, scaling=scaling, **kw)
    sp.sp_rope_fwd(x, tab, positions=pos.view(4, 5).to(DEV), y=y)
    freq = orc.frequencies(64, 500000.0, scaling, **{k: v for k, v in kw.items() if k != "mscale"})
    # a frequency of 53 bits times a position p is off by about p 2^-53 radians of its own
    near = np.abs(pos.view(4, 5).numpy())[..., None, None] < 2 ** 26
    want, mag = orc.rope(f64(x[0]), pos.view(4, 5).numpy(), freq, "half", kw.get("mscale", 1.0))
    far = np.broadcast_to(np.where(near, 0.0, 2.0 ** -10), want.shape)
    close(y[0], want, mag * (1 + far * 2 ** 21), 2.0 ** -21, scaling)


def test_rope_packed_positions_and_strides():
    """Packed sequences (empty, of one token), heads cut from a fused projection
    on both sides; what lies between is untouched."""
    gen = torch.Generator().manual_seed(9)
    lens = [0, 5, 1, 0, 0, 40, 1, 30, 0]
    cu = np.concatenate(([0], np.cumsum(lens)))
    s = int(cu[-1])
    wide = [rand((1, s, 12, 40), gen, BF) for _ in range(2)]
    out = [torch.full((1, s, 9, 40), 3.0, dtype=BF, device=DEV) for _ in range(2)]
    x, y = [w[:, :, 2:7] for w in wide], [w[:, :, 1:6] for w in out]
    tab = sp.sp_rope_table(32)
    sp.sp_rope_fwd(x, tab, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                   first_position=3, y=y)
    for r in range(2):
        want, mag = orc.rope(f64(x[r]), orc.positions(1, s, 3, cu), orc.frequencies(32))
        close(y[r], want, mag, 2.0 ** -21, f"rank {r}")
        assert (out[r][:, :, 0] == 3).all() and (out[r][:, :, 6:] == 3).all()
    # every second head (head stride 80), odd strides: elements one by one
    odd = torch.zeros((1, 7, 5 * 41 + 3), dtype=BF, device=DEV)
    view = odd.as_strided((1, 7, 5, 40), (7 * 208, 208, 41, 1))
    src = rand((1, 7, 5, 40), gen, BF)
    view.copy_(src)
    sp.sp_rope_fwd([view], tab, y=[view])
    want, mag = orc.rope(f64(src), orc.positions(1, 7), orc.frequencies(32))
    close(view, want, mag, 2.0 ** -21, "odd strides")
    assert (odd.as_strided((7, 5), (208, 41), 40) == 0).all()


@pytest.mark.parametrize("t,heads,d,rot,layout,dtype", [
    (1, 5, 80, 20, "half", BF), (1, 5, 80, 20, "interleaved", FP), (2, 1, 32, 32, "half", F32),
    (1, 1, 8, 2, "interleaved", BF), (1, 3, 15, 6, "half", BF), (1, 2, 128, 128, "half", BF),
    (1, 1, 512, 512, "interleaved", FP)])
@pytest.mark.parametrize("where", ["dense", "packed", "positions"])
def test_rope_many_small_tokens(t, heads, d, rot, layout, dtype, where):
    """Enough tokens that a warp takes several at once, the last group cut short; a
    sample of them against the oracle."""
    gen = torch.Generator().manual_seed(19)
    b, s = (1, 40003) if where == "packed" else (3, 13339)
    x = [rand((b, s, heads, d), gen, dtype) for _ in range(t)]
    y = [torch.full_like(q, float("nan")) for q in x]
    rng = np.random.default_rng(3)
    cu = pos = None
    want_pos = orc.positions(b, s, 9)
    if where == "packed":
        cu = np.concatenate(([0, 0, 1], np.sort(rng.integers(1, s, 300)), [s]))
        want_pos = orc.positions(1, s, 9, cu)
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if where == "positions":
        want_pos = rng.integers(0, 1 << 20, (b, s))
        pos = torch.tensor(want_pos, device=DEV)
    tab = sp.sp_rope_table(rot)
    how = dict(layout=layout, positions=pos, first_position=9, cu_seqlens=cu)
    sp.sp_rope_fwd(x, tab, y=y, **how)
    at = np.unique(np.concatenate((rng.integers(0, s, 300), np.arange(20), np.arange(s - 20, s))))
    for r in range(t):
        want, mag = orc.rope(f64(x[r])[:, at], want_pos[:, at], orc.frequencies(rot), layout)
        close(y[r][:, at], want, mag, 2.0 ** -21, where)
    back = [torch.empty_like(q) for q in x]
    sp.sp_rope_bwd(x, tab, dx=back, **how)
    for r in range(t):
        want, mag = orc.rope(f64(x[r])[:, at], want_pos[:, at], orc.frequencies(rot), layout, back=True)
        close(back[r][:, at], want, mag, 2.0 ** -21, where)


def test_rope_many_sequences():
    """More packed sequences than one search step reaches."""
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, size=2100)
    cu = np.concatenate(([0], np.cumsum(lens)))
    s = int(cu[-1])
    x = [rand((1, s, 1, 8), torch.Generator().manual_seed(2), F32)]
    y = [torch.empty_like(x[0])]
    sp.sp_rope_fwd(x, sp.sp_rope_table(8), y=y,
                   cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    want, mag = orc.rope(f64(x[0]), orc.positions(1, s, 0, cu), orc.frequencies(8))
    close(y[0], want, mag, 2.0 ** -21, "packed")


def test_rope_back_is_the_transpose():
    gen = torch.Generator().manual_seed(10)
    x, dy = rand((2, 6, 3, 32), gen, F32), rand((2, 6, 3, 32), gen, F32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    tab = sp.sp_rope_table(24, mscale=1.5)
    sp.sp_rope_fwd([x], tab, layout="interleaved", y=[y])
    sp.sp_rope_bwd([dy], tab, layout="interleaved", dx=[dx])
    a, b = (y.double() * dy.double()).sum().item(), (x.double() * dx.double()).sum().item()
    # each of the 1152 terms is off by at most 2^-21 of its magnitude on either side
    size = (y.double().abs() * dy.double().abs()).sum().item() * 2
    assert abs(a - b) <= 2 * 2.0 ** -21 * size * 1.5


# ---------------------------------------------------------- gated recurrence --

def scan_inputs(t, n, b, s, c, dtype, seed, state, spread=2.0, shift=1.0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda shape, dt, *a: [rand(shape, gen, dt, *a) for _ in range(t)]
    return dict(gate=mk((b, s, c), dtype, spread, shift), value=mk((b, s, c), dtype),
                dy=mk((b, s, c), dtype), h0=mk((n, c), F32) if state else None,
                dhT=mk((n, c), F32) if state else None)


def run_scan(i, n, tied, cu, state):
    t, like = len(i["gate"]), i["gate"][0]
    b, s, c = like.shape
    nan = lambda shape, dt: [torch.full(shape, float("nan"), dtype=dt, device=DEV) for _ in range(t)]
    o = dict(y=nan((b, s, c), like.dtype), hT=nan((n, c), F32) if state else None,
             states=nan(sp.sp_gated_scan_states_shape(b, s, c), F32),
             dgate=nan((b, s, c), like.dtype), dvalue=nan((b, s, c), like.dtype),
             dh0=nan((n, c), F32) if state else None)
    how = dict(h0=i["h0"], tied=tied, cu_seqlens=cu)
    sp.sp_gated_scan_fwd(i["gate"], i["value"], y=o["y"], hT=o["hT"], states=o["states"], **how)
    sp.sp_gated_scan_bwd(i["gate"], i["value"], o["states"], i["dy"], dhT=i["dhT"],
                         dgate=o["dgate"], dvalue=o["dvalue"], dh0=o["dh0"], **how)
    return o


def check_scan(i, o, tied, lens, n_tokens, state):
    cu = None if lens is None else np.concatenate(([0], np.cumsum(lens)))
    rel = 2.0 ** -18 + n_tokens * 2.0 ** -22
    for r in range(len(i["gate"])):
        g, v = f64(i["gate"][r]), f64(i["value"][r])
        h0 = f64(i["h0"][r]) if state else None
        f = orc.gated_scan(g, v, h0, tied, cu)
        top = f["mag"].max((0, 1)) if f["mag"].size else np.zeros(g.shape[2])
        if f["magT"].size:
            top = np.maximum(top, f["magT"].max(0))
        close(o["y"][r], f["y"], top, rel, f"y[{r}]")
        if state:
            close(o["hT"][r], f["hT"], top, rel, f"hT[{r}]")
        w = orc.gated_scan_bwd(g, v, f64(i["dy"][r]), h0, f64(i["dhT"][r]) if state else None,
                               tied, cu)
        for name in ("dgate", "dvalue") + (("dh0",) if state else ()):
            got, mag = o[name][r], w["mag_" + name]
            top = mag.max(tuple(range(mag.ndim - 1))) if mag.size else 0
            close(got, w[name], top, 3 * rel, f"{name}[{r}]")


SCAN = [
    # t, b, s, c, dtype
    (1, 1, 1, 8, BF), (2, 5, 1, 72, BF), (1, 1, 2, 64, F32), (2, 2, 15, 8, FP), (1, 3, 16, 136, BF),
    (1, 1, 17, 64, F32), (2, 1, 129, 64, BF), (1, 2, 300, 200, BF), (8, 1, 515, 64, BF),
    (1, 1, 1031, 24, F32), (3, 2, 257, 40, FP), (1, 1, 4100, 8, BF), (1, 130, 33, 128, BF),
]


@pytest.mark.parametrize("t,b,s,c,dtype", SCAN)
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("state", [True, False])
def test_scan_dense(t, b, s, c, dtype, tied, state):
    i = scan_inputs(t, b, b, s, c, dtype, 11, state)
    o = run_scan(i, b, tied, None, state)
    check_scan(i, o, tied, None, s, state)
    assert all(same(o[k], v) for k, v in run_scan(i, b, tied, None, state).items()
               if v is not None and k != "states")


LENS = [[1], [0, 1, 0], [40], [0, 0, 70, 0, 3, 1, 1, 1, 0], [1] * 37, [16] * 9 + [0] * 40 + [17],
        [5, 600, 0, 2, 1000, 31, 33], list(range(30)), [0] * 70 + [300] + [0] * 70 + [9]]


@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("dtype,c,state", [(BF, 72, True), (F32, 64, True), (FP, 64, False)])
def test_scan_packed(lens, tied, dtype, c, state):
    n, s = len(lens), sum(lens)
    i = scan_inputs(2, n, 1, s, c, dtype, 12, state)
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device=DEV)
    o = run_scan(i, n, tied, cu, state)
    check_scan(i, o, tied, lens, max(lens), state)


@pytest.mark.parametrize("lens", [None, [1, 1700, 0, 15, 17, 2767], [4500]], ids=["dense", "q6", "q1"])
@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("dtype,t,s,c", [(BF, 1, 4500, 72), (FP, 1, 4500, 64), (F32, 1, 4500, 72),
                                         (BF, 2, 4500, 520), (F32, 3, 4500, 264)])
def test_scan_few_channels(lens, tied, dtype, t, s, c):
    """Long sequences of few channels: large blocks, long clusters."""
    n = 1 if lens is None else len(lens)
    cu = None if lens is None else torch.tensor(np.concatenate(([0], np.cumsum(lens))),
                                                dtype=torch.int32, device=DEV)
    i = scan_inputs(t, n, 1, s, c, dtype, 77 + c, True)
    check_scan(i, run_scan(i, n, tied, cu, True), tied, lens, s, True)


def test_scan_no_token():
    """s == 0 and packed sequences that are all empty: states and their gradients pass."""
    for cu, b, n in ((None, 3, 3), (torch.zeros(5, dtype=torch.int32, device=DEV), 1, 4)):
        i = scan_inputs(2, n, b, 0, 16, BF, 13, True)
        o = run_scan(i, n, True, cu, True)
        assert same(o["hT"], i["h0"]) and same(o["dh0"], i["dhT"])
        i["h0"] = i["dhT"] = None
        hT = [torch.full((n, 16), 5.0, device=DEV) for _ in range(2)]
        sp.sp_gated_scan_fwd(i["gate"], i["value"], y=o["y"], hT=hT, cu_seqlens=cu)
        assert all((h == 0).all() for h in hT)


def test_scan_keeps_sequences_apart():
    """What an earlier or later sequence holds (NaN, infinities, a state of them)
    reaches no other, forward or backward; a whole row of the packed batch at a time."""
    lens = [30, 17, 0, 200, 1, 90]
    cu_np = np.concatenate(([0], np.cumsum(lens)))
    cu = torch.tensor(cu_np, dtype=torch.int32, device=DEV)
    i = scan_inputs(1, 6, 1, sum(lens), 64, BF, 14, True)
    clean = run_scan(i, 6, True, cu, True)
    for bad in (0, 3):
        j = {k: [x.clone() for x in v] for k, v in i.items()}
        lo, hi = cu_np[bad], cu_np[bad + 1]
        for k in ("gate", "value", "dy"):
            j[k][0][0, lo:hi:3] = float("nan")
            j[k][0][0, lo + 1:hi:3] = float("inf")
        j["h0"][0][bad] = float("-inf")
        j["dhT"][0][bad] = float("nan")
        o = run_scan(j, 6, True, cu, True)
        keep = torch.ones(sum(lens), dtype=torch.bool, device=DEV)
        keep[lo:hi] = False
        seqs = torch.arange(6, device=DEV) != bad
        for k in ("y", "dgate", "dvalue"):
            assert same([clean[k][0][0, keep]], [o[k][0][0, keep]]), k
        for k in ("hT", "dh0"):
            assert same([clean[k][0][seqs]], [o[k][0][seqs]]), k
        assert not torch.isfinite(o["y"][0][0, lo:hi]).all()


def test_scan_extreme_gates():
    """Gates that shut (sigmoid 0) and open (sigmoid 1) completely in every type."""
    for dtype in (BF, FP, F32):
        i = scan_inputs(1, 1, 1, 100, 64, dtype, 15, True, spread=0.0, shift=0.0)
        i["gate"][0][0, ::2] = 300.0
        i["gate"][0][0, 1::2] = -300.0
        o = run_scan(i, 1, True, None, True)
        v = f64(i["value"][0])[0]
        want = np.where(np.arange(100)[:, None] % 2 == 1, v, np.roll(v, 1, 0))
        want[0] = f64(i["h0"][0])[0]
        # the first token rounds h0 to the type once, every other value is one
        close(o["y"][0][0], want, np.abs(want) + 1, 2.0 ** -23, str(dtype))
        for k in ("dgate", "dvalue", "dh0", "hT"):
            assert torch.isfinite(o[k][0]).all(), (dtype, k)
        i["gate"][0][0, 50] = float("nan")
        o = run_scan(i, 1, True, None, True)
        assert torch.isnan(o["y"][0][0, 50]).all() and torch.isfinite(o["y"][0][0, :50]).all()


def test_scan_slices_in_place_states_and_untouched_rows():
    """Gate and value as slices of one projection, gradients into slices of one
    buffer, hT over h0; nothing beside the slices is written."""
    gen = torch.Generator().manual_seed(16)
    proj, dproj = rand((2, 50, 160), gen, BF), torch.full((2, 50, 160), 7.0, dtype=BF, device=DEV)
    i = dict(gate=[proj[..., :72]], value=[proj[..., 80:152]], dy=[rand((2, 50, 72), gen, BF)],
             h0=[rand((2, 72), gen, F32)], dhT=[rand((2, 72), gen, F32)])
    want = run_scan(i, 2, True, None, True)
    state, y = i["h0"][0].clone(), torch.empty((2, 50, 72), dtype=BF, device=DEV)
    st = [torch.empty(sp.sp_gated_scan_states_shape(2, 50, 72), device=DEV)]
    sp.sp_gated_scan_fwd(i["gate"], i["value"], h0=[state], hT=[state], y=[y], states=st)
    assert same([y, state], [want["y"][0], want["hT"][0]])
    grad = torch.empty_like(i["dhT"][0])
    sp.sp_gated_scan_bwd(i["gate"], i["value"], st, i["dy"], h0=i["h0"], dhT=i["dhT"],
                         dgate=[dproj[..., :72]], dvalue=[dproj[..., 80:152]], dh0=[grad])
    assert same([dproj[..., :72], dproj[..., 80:152], grad],
                [want["dgate"][0], want["dvalue"][0], want["dh0"][0]])
    assert (dproj[..., 72:80] == 7).all() and (dproj[..., 152:] == 7).all()


def test_scan_steps_are_the_sequence():
    """Token by token through the decoding form, the state in place, is the scan:
    y of each form is within its own bound of the exact value."""
    i = scan_inputs(2, 3, 3, 40, 72, BF, 17, True)
    o = run_scan(i, 3, True, None, True)
    state = [h.clone() for h in i["h0"]]
    steps = []
    for k in range(40):
        y = [torch.empty((3, 1, 72), dtype=BF, device=DEV) for _ in range(2)]
        sp.sp_gated_scan_fwd([g[:, k:k + 1] for g in i["gate"]], [v[:, k:k + 1] for v in i["value"]],
                             h0=state, hT=state, y=y)
        steps.append(y)
    o["y"] = [torch.cat([y[r] for y in steps], 1) for r in range(2)]
    o["hT"] = state
    check_scan(i, o, True, None, 40, True)


def test_scan_bad_metadata_is_flagged_and_harmless():
    """cu_seqlens that decrease, start late, end early or late: the status word says
    so, the call stays inside its buffers and ends."""
    i = scan_inputs(1, 3, 1, 100, 64, BF, 18, True)
    x = [rand((1, 100, 2, 32), torch.Generator().manual_seed(1), BF)]
    tab = sp.sp_rope_table(32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for cu in ([0, 60, 20, 100], [5, 20, 60, 100], [0, 20, 60, 90], [0, 20, 60, 1000],
               [-7, -3, 2000000000, -1]):
        m = torch.tensor(cu, dtype=torch.int32, device=DEV)
        fence = [torch.full((1, 100 * 64 + 4096), 9.0, dtype=BF, device=DEV) for _ in range(3)]
        y = [f[0, 2048:2048 + 6400].view(1, 100, 64) for f in fence]
        hT = torch.full((3 + 32, 64), 9.0, device=DEV)
        st = [torch.empty(sp.sp_gated_scan_states_shape(1, 100, 64), device=DEV)]
        how = dict(h0=i["h0"], cu_seqlens=m, status=status)
        for call in (lambda: sp.sp_gated_scan_fwd(i["gate"], i["value"], y=[y[0]], hT=[hT[16:19]],
                                                  states=st, **how),
                     lambda: sp.sp_gated_scan_bwd(i["gate"], i["value"], st, i["dy"],
                                                  dhT=i["dhT"], dgate=[y[1]], dvalue=[y[2]],
                                                  dh0=[hT[16:19]], **how),
                     lambda: sp.sp_rope_fwd(x, tab, cu_seqlens=m, y=[torch.empty_like(x[0])],
                                            status=status)):
            status.zero_()
            call()
            torch.cuda.synchronize()
            assert status.item() == 6, cu
        for f in fence:
            assert (f[0, :2048] == 9).all() and (f[0, 2048 + 6400:] == 9).all()
        assert (hT[:16] == 9).all() and (hT[19:] == 9).all()


# ---------------------------------------------------------------- group norm --

NORM = [
    # t, n, l, c, groups, dtype
    (1, 1, 1, 8, 1, BF), (2, 5, 1, 64, 8, BF), (8, 33, 1, 128, 1, BF), (2, 301, 1, 256, 2, FP),
    (1, 7, 1, 640, 16, BF), (1, 9, 1, 96, 1, F32), (1, 3, 1, 4096, 1, BF), (1, 2, 1, 4000, 1, F32),
    (2, 3, 1, 16384, 64, BF), (1, 4, 2, 64, 2, BF), (1, 3, 7, 80, 2, F32), (2, 6, 32, 512, 16, BF),
    (1, 2, 33, 24, 3, FP), (1, 2, 64, 2048, 8, BF), (1, 2, 65, 4096, 1, BF), (1, 1, 700, 40, 1, F32),
    (2, 3, 513, 320, 8, BF), (1, 1, 5001, 64, 8, BF), (1, 40, 100, 72, 9, FP), (1, 2, 2000, 1280, 32, BF),
    (1, 1, 9000, 4096, 2, BF), (1, 1, 3001, 3200, 1, F32), (2, 700, 21, 512, 8, BF),
    (1, 900, 24, 40, 5, FP), (1, 500, 17, 1280, 16, F32), (1, 11, 5, 1600, 1, F32),
    (3, 5, 50, 1360, 17, BF), (1, 3, 4, 2048, 1, BF), (1, 5, 3, 4096, 16, FP),
]


def norm_inputs(t, n, l, c, dtype, seed, shift=0.0, gen=None):
    gen = torch.Generator().manual_seed(seed)
    off = torch.randn(c, generator=gen) + shift
    return dict(x=[(torch.randn((n, l, c), generator=gen) + off).to(dtype).to(DEV) for _ in range(t)],
                dy=[rand((n, l, c), gen, dtype) for _ in range(t)],
                gamma=rand((t * c,), gen, dtype, 0.3, 1.0), beta=rand((t * c,), gen, dtype, 0.5))


def run_norm(i, groups, norm, act, eps=1e-5, params=True):
    t, like = len(i["x"]), i["x"][0]
    n, l, c = like.shape
    nan = lambda shape, dt: torch.full(shape, float("nan"), dtype=dt, device=DEV)
    ln = norm == "layernorm"
    o = dict(y=[nan((n, l, c), like.dtype) for _ in range(t)],
             mean=[nan((n, groups), F32) for _ in range(t)] if ln else None,
             rstd=[nan((n, groups), F32) for _ in range(t)],
             dx=[nan((n, l, c), like.dtype) for _ in range(t)],
             dgamma=nan((t * c,), F32) if params else None,
             dbeta=nan((t * c,), F32) if params and ln else None)
    how = dict(groups=groups, norm=norm, act=act)
    beta = i["beta"] if ln else None
    sp.sp_group_norm_fwd(i["x"], i["gamma"], beta, eps=eps, y=o["y"], mean=o["mean"],
                         rstd=o["rstd"], **how)
    ws = torch.full((max(16, sp.sp_group_norm_bwd_workspace_bytes(n, l, c, groups, t, like.dtype)),),
                    255, dtype=torch.uint8, device=DEV) if params else None
    sp.sp_group_norm_bwd(i["dy"], i["x"], o["mean"], o["rstd"], i["gamma"], beta, dx=o["dx"],
                         dgamma=o["dgamma"], dbeta=o["dbeta"], workspace=ws, **how)
    return o


def check_norm(i, o, groups, norm, act, eps=1e-5):
    t, c = len(i["x"]), i["x"][0].shape[2]
    ln = norm == "layernorm"
    for r in range(t):
        x, dy = f64(i["x"][r]), f64(i["dy"][r])
        gamma, beta = f64(i["gamma"][r * c:(r + 1) * c]), f64(i["beta"][r * c:(r + 1) * c])
        f = orc.group_norm(x, gamma, beta, groups, eps, norm, act)
        close(o["y"][r], f["y"], f["mag"], 2.0 ** -15, f"y[{r}]")
        top = np.abs(x).max() if x.size else 0
        if ln:
            close(o["mean"][r], f["mean"], top, 2.0 ** -16, f"mean[{r}]")
        close(o["rstd"][r], f["rstd"], f["rstd"], 2.0 ** -15, f"rstd[{r}]")
        w = orc.group_norm_bwd(dy, x, gamma, beta, groups, eps, norm, act)
        close(o["dx"][r], w["dx"], w["mag_dx"], 2.0 ** -13, f"dx[{r}]")
        for name in ("dgamma", "dbeta"):
            if o[name] is not None:
                close(o[name][r * c:(r + 1) * c], w[name], w["mag_" + name], 2.0 ** -14,
                      f"{name}[{r}]")


@pytest.mark.parametrize("t,n,l,c,groups,dtype", NORM)
@pytest.mark.parametrize("norm,act", [("layernorm", "silu"), ("rmsnorm", "silu"),
                                      ("layernorm", "none"), ("rmsnorm", "none")])
def test_group_norm(t, n, l, c, groups, dtype, norm, act):
    i = norm_inputs(t, n, l, c, dtype, 21)
    o = run_norm(i, groups, norm, act)
    check_norm(i, o, groups, norm, act)
    again = run_norm(i, groups, norm, act)
    for k, v in o.items():
        if v is not None:
            assert same(v, again[k]) if isinstance(v, list) else same([v], [again[k]]), k


@pytest.mark.parametrize("n,l,c,groups", [(40, 1, 256, 4), (6, 5, 80, 2), (2, 900, 128, 4)])
def test_group_norm_mean_far_above_the_spread(n, l, c, groups):
    """A mean of 1000 standard deviations: the statistics keep their digits."""
    i = norm_inputs(1, n, l, c, F32, 22, shift=1000.0)
    o = run_norm(i, groups, "layernorm", "none")
    f = orc.group_norm(f64(i["x"][0]), f64(i["gamma"]), f64(i["beta"]), groups, 1e-5)
    # the mean is off by at most 2^-17 of 1000 by its own sums, in float32 by half a
    # step of 1000 at least; an error e of it moves the variance by e^2 only
    close(o["mean"][0], f["mean"], 1000.0, 2.0 ** -17, "mean")
    close(o["rstd"][0], f["rstd"], f["rstd"], 2.0 ** -12, "rstd")


def test_group_norm_constant_groups_and_outliers():
    """No spread at all (rstd = eps^-1/2, y = beta), one value far from all others."""
    for n, l, c, groups in ((9, 1, 128, 2), (3, 6, 40, 1), (2, 800, 64, 4)):
        i = norm_inputs(1, n, l, c, F32, 23)
        i["x"][0].fill_(3.25)
        o = run_norm(i, groups, "layernorm", "none")
        want = i["beta"].expand(n, l, c)
        # every sum of equal values is exact but for the division by the count: the mean
        # is off by at most 2^-17 of 3.25, times rstd = 316 and gamma below 3
        assert ((o["y"][0] - want).abs() <= 3.25 * 2.0 ** -17 * 317 * 3).all()
        i = norm_inputs(1, n, l, c, F32, 24)
        i["x"][0][:, 0, 0] = 5000.0
        o = run_norm(i, groups, "layernorm", "silu")
        check_norm(i, o, groups, "layernorm", "silu")


def test_group_norm_rows_of_a_wider_buffer():
    """x, dy, y and dx as slices; nothing beside them is written.  No parameter gradients."""
    for n, l, c, groups in ((12, 1, 64, 4), (2, 3, 40, 5), (2, 700, 64, 2)):
        gen = torch.Generator().manual_seed(25)
        wide = rand((n, l, 2 * c + 16), gen, BF)
        i = norm_inputs(1, n, l, c, BF, 26)
        i["x"], i["dy"] = [wide[..., :c]], [wide[..., c + 8:2 * c + 8]]
        want = run_norm(i, groups, "layernorm", "silu")
        out = torch.full((n, l, 2 * c + 16), 7.0, dtype=BF, device=DEV)
        y, dx = out[..., :c], out[..., c + 8:2 * c + 8]
        how = dict(groups=groups, act="silu")
        mean, rstd = [torch.empty_like(want["mean"][0])], [torch.empty_like(want["rstd"][0])]
        sp.sp_group_norm_fwd(i["x"], i["gamma"], i["beta"], eps=1e-5, y=[y], mean=mean, rstd=rstd, **how)
        sp.sp_group_norm_bwd(i["dy"], i["x"], mean, rstd, i["gamma"], i["beta"], dx=[dx], **how)
        assert same([y, dx, mean[0], rstd[0]],
                    [want["y"][0], want["dx"][0], want["mean"][0], want["rstd"][0]])
        assert (out[..., c:c + 8] == 7).all() and (out[..., 2 * c + 8:] == 7).all()


def test_group_norm_no_row():
    i = norm_inputs(2, 0, 4, 64, BF, 27)
    o = run_norm(i, 2, "layernorm", "silu")
    assert (o["dgamma"] == 0).all() and (o["dbeta"] == 0).all()


# ----------------------------------------------------------------- together --

def mixer(x, w, b, s, cu, tab, groups):
    """The region as it is used: g's output -> column-parallel projections of one rank
    -> per-head norm and rotary of the queries; recurrence -> group norm with SiLU of
    the values; forward and backward.  w: projection (h, 3c); c = heads * d."""
    heads, d = 2, 64
    c = heads * d
    e = lambda shape, dt=BF: torch.empty(shape, dtype=dt, device=DEV)
    proj = x @ w
    gate, value, q = proj[..., :c], proj[..., c:2 * c], proj[..., 2 * c:]
    one = torch.ones(c, dtype=BF, device=DEV)
    zero = torch.zeros(c, dtype=BF, device=DEV)
    tok = b * s
    qn, qr = e((tok, 1, c)), e((b, s, heads, d))
    qrs = e((tok, heads), F32)
    sp.sp_group_norm_fwd([q.reshape(tok, 1, c)], one, groups=heads, norm="rmsnorm", eps=1e-6,
                         y=[qn], rstd=[qrs])
    sp.sp_rope_fwd([qn.view(b, s, heads, d)], tab, cu_seqlens=cu, y=[qr])
    hid, states = e((b, s, c)), e(sp.sp_gated_scan_states_shape(b, s, c), F32)
    sp.sp_gated_scan_fwd([gate], [value], cu_seqlens=cu, y=[hid], states=[states])
    out, mean, rstd = e((tok, 1, c)), e((tok, groups), F32), e((tok, groups), F32)
    sp.sp_group_norm_fwd([hid.view(tok, 1, c)], one, zero, groups=groups, act="silu", eps=1e-5,
                         y=[out], mean=[mean], rstd=[rstd])
    mix = out.view(b, s, c) * qr.view(b, s, c)
    # backward with the gradient of mix = mix
    dout, dqr = (mix * qr.view(b, s, c)).view(tok, 1, c), (mix * out.view(b, s, c))
    ws = torch.empty(sp.sp_group_norm_bwd_workspace_bytes(tok, 1, c, groups, 1), dtype=torch.uint8,
                     device=DEV)
    dhid, dg, db = e((tok, 1, c)), e((c,), F32), e((c,), F32)
    sp.sp_group_norm_bwd([dout], [hid.view(tok, 1, c)], [mean], [rstd], one, zero, groups=groups,
                         act="silu", dx=[dhid], dgamma=dg, dbeta=db, workspace=ws)
    dproj = e((b, s, 3 * c))
    sp.sp_gated_scan_bwd([gate], [value], [states], [dhid.view(b, s, c)], cu_seqlens=cu,
                         dgate=[dproj[..., :c]], dvalue=[dproj[..., c:2 * c]])
    dqn = e((b, s, heads, d))
    sp.sp_rope_bwd([dqr.view(b, s, heads, d)], tab, cu_seqlens=cu, dx=[dqn])
    dq = dproj.view(tok, 1, 3 * c)[..., 2 * c:]
    sp.sp_group_norm_bwd([dqn.view(tok, 1, c)], [q.reshape(tok, 1, c)], None, [qrs], one,
                         groups=heads, norm="rmsnorm", dx=[dq])
    return mix, dproj, dg, db


def mixer_float(proj, s, cu, freq):
    """The same in float64 torch operations, differentiable; (s, 3c) of one batch row."""
    c = proj.shape[1] // 3
    gate, value, q = proj[:, :c], proj[:, c:2 * c], proj[:, 2 * c:]
    qh = q.view(s, 2, 64)
    qn = qh * torch.rsqrt((qh * qh).mean(-1, keepdim=True) + 1e-6)
    ang = torch.from_numpy(orc.positions(1, s, 0, cu)[0][:, None, None] * freq)
    u, v = qn[..., :32], qn[..., 32:]
    qr = torch.cat((u * ang.cos() - v * ang.sin(), v * ang.cos() + u * ang.sin()), -1).reshape(s, c)
    rows, h = [], None
    for i in range(s):
        if i in cu[:-1]:
            h = torch.zeros(c, dtype=torch.float64)
        a = torch.sigmoid(gate[i])
        h = a * h + (1 - a) * value[i]
        rows.append(h)
    hid = torch.stack(rows).view(s, 2, 64)
    z = (hid - hid.mean(-1, keepdim=True)) * torch.rsqrt(hid.var(-1, unbiased=False, keepdim=True) + 1e-5)
    z = z.reshape(s, c)
    return z * torch.sigmoid(z) * qr


def test_mixer_of_a_layer_and_its_graph():
    """The operators after each other between g and the next g*, on a side stream and
    replayed from a CUDA graph; forward and gradients against float64."""
    gen = torch.Generator().manual_seed(31)
    cu_np = np.array([0, 21, 21, 22, 96])
    s, c = 96, 128
    x, w = rand((1, s, 256), gen, BF), rand((256, 3 * c), gen, BF, 1 / 16)
    cu = torch.tensor(cu_np, dtype=torch.int32, device=DEV)
    tab = sp.sp_rope_table(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mixer(x, w, 1, s, cu, tab, 2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = mixer(x, w, 1, s, cu, tab, 2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, kept)
    proj = (x @ w)[0].double().cpu().requires_grad_(True)
    mix = mixer_float(proj, s, cu_np, orc.frequencies(64))
    (mix * f_const(got[0])).sum().backward()
    # bf16 rounds each of up to six values in a row, 2^-8 each, against the rms of the result
    for a, b in ((got[0][0], mix.detach()), (got[1][0], proj.grad)):
        diff = (a.double().cpu() - b).norm() / b.norm()
        assert diff < 6 * 2.0 ** -8, diff


def f_const(x):
    return x[0].double().cpu()


def test_two_streams_at_once():
    """Two calls of every operator that may overlap on the device, one workspace each."""
    a, b = scan_inputs(1, 1, 1, 3000, 64, BF, 41, True), scan_inputs(1, 1, 1, 3000, 64, BF, 42, True)
    p, q = norm_inputs(1, 2, 1500, 128, BF, 43), norm_inputs(1, 2, 1500, 128, BF, 44)
    want = [run_scan(v, 1, True, None, True) for v in (a, b)], [run_norm(v, 4, "layernorm", "silu") for v in (p, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [], []
        for st, v, w in zip(streams, (a, b), (p, q)):
            with torch.cuda.stream(st):
                got[0].append(run_scan(v, 1, True, None, True))
                got[1].append(run_norm(w, 4, "layernorm", "silu"))
        torch.cuda.synchronize()
        for g, w in zip(got[0] + got[1], want[0] + want[1]):
            for k, v in w.items():
                if v is not None and k != "states":
                    assert same(v, g[k]) if isinstance(v, list) else same([v], [g[k]]), k


class LongWay:
    """The compiled short way, taking nothing."""
    def __getattr__(self, name):
        return lambda *args: None


def test_short_and_long_way_agree(monkeypatch):
    """The compiled call gives what the binding's own call gives, for every order of
    strides: the same bits, or a refusal."""
    quick, long = sp._quick(), LongWay()
    base = rand((3, 6, 4, 64), torch.Generator().manual_seed(95), BF)
    whole = [slice(None), slice(None, 1), slice(1, None), slice(None, None, 2), slice(2, 2)]
    last = [slice(None), slice(16, 32), slice(None, None, 2), slice(8, 16)]
    tab, seen = sp.sp_rope_table(8), dict.fromkeys(("both", "neither"), 0)
    g, bt = rand((2 * 64,), torch.Generator().manual_seed(96), BF), torch.zeros(128, dtype=BF, device=DEV)

    def outcome(way, call):
        monkeypatch.setattr(sp, "_module", way)
        try:
            return call()
        except (ValueError, sp.SpError) as e:
            return type(e)

    for i, j, k, m in itertools.product(whole, whole, whole, last):
        x = base[i, j, k, m]
        for v in (x, x.transpose(1, 2), x.transpose(0, 1)):
            def rope():
                y = [torch.zeros(v.shape, dtype=BF, device=DEV) for _ in range(2)]
                sp.sp_rope_fwd([v, v], tab, y=y)
                return y

            def norm():
                z, d = v[:, :, 0], v.shape[-1]
                y = [torch.zeros(z.shape, dtype=BF, device=DEV) for _ in range(2)]
                st = [[torch.zeros(z.shape[0], 1, device=DEV) for _ in range(2)] for _ in range(2)]
                sp.sp_group_norm_fwd([z, z], g[:2 * d], bt[:2 * d], groups=1, eps=1e-5, y=y,
                                     mean=st[0], rstd=st[1])
                return y + st[0] + st[1]

            for call in (rope, norm) if v.shape[2] else (rope,):
                a, b = outcome(quick, call), outcome(long, call)
                assert isinstance(a, list) == isinstance(b, list)
                assert same(a, b) if isinstance(a, list) else a is b
                seen["both" if isinstance(a, list) else "neither"] += 1
    assert min(seen.values()) > 50


def test_short_and_long_way_agree_on_every_operator(monkeypatch):
    quick = sp._quick()
    cu = torch.tensor([0, 5, 5, 40], dtype=torch.int32, device=DEV)
    i = scan_inputs(2, 3, 1, 40, 72, FP, 97, True)
    n = norm_inputs(2, 5, 7, 64, F32, 98)
    x = [rand((2, 5, 3, 32), torch.Generator().manual_seed(99), F32)]
    pos = torch.arange(10, device=DEV).view(2, 5)
    tab, own = sp.sp_rope_table(16), torch.zeros(1, dtype=torch.int32, device=DEV)

    def everything():
        y = [torch.zeros_like(x[0])]
        sp.sp_rope_bwd(x, tab, positions=pos, layout="interleaved", dx=y, status=own)
        o = [y[0]]
        for r in (run_scan(i, 3, False, cu, True), run_norm(n, 4, "layernorm", "silu"),
                  run_norm(n, 4, "rmsnorm", "none", params=False)):
            for v in r.values():
                o += v if isinstance(v, list) else [] if v is None else [v]
        return o

    a = everything()
    monkeypatch.setattr(sp, "_module", LongWay())
    b = everything()
    assert len(a) == len(b) and same(a, b)
    monkeypatch.setattr(sp, "_module", quick)
    # what the short way must leave alone
    bad = torch.zeros(1, dtype=torch.int32)
    for how in (dict(status=bad), dict(status=own.float()), dict(positions=pos.int()),
                dict(positions=pos.t()), dict(cu_seqlens=cu), dict(layout="both")):
        with pytest.raises((ValueError, TypeError)):
            sp.sp_rope_fwd(x, tab, y=[torch.zeros_like(x[0])], **how)
    with pytest.raises(TypeError):
        sp.sp_group_norm_fwd(n["x"], n["gamma"], None, groups=4, eps=1e-5, y=n["x"], mean=None,
                             rstd=None)
    with pytest.raises(ValueError):
        sp.sp_group_norm_fwd(n["x"], n["gamma"][:-1], n["beta"], groups=4, eps=1e-5, y=n["x"],
                             mean=None, rstd=None)


def test_offsets_beyond_32_bits():
    """Rows so far apart that elements and bytes pass 2^32: the same bits as dense
    rows, whatever the form; slices of one buffer beside each other."""
    rows, ld = 4400, 1 << 20
    wide = torch.empty(rows * ld, dtype=BF, device=DEV)        # 9.2 GB
    assert wide.numel() > 2 ** 32
    gen = torch.Generator().manual_seed(91)
    at = iter(range(0, ld, 1024))

    def far(x):
        """A copy of (b, s, c) x as a slice of the wide buffer."""
        b, s, c = x.shape
        v = wide.as_strided((b, s, c), (s * ld, ld, 1), next(at))
        v.copy_(x)
        return v

    def near(b, s, c):
        return rand((b, s, c), gen, BF)

    # rotary
    x, tab = near(1, rows, 3 * 64), sp.sp_rope_table(48)
    y, v = torch.empty_like(x), far(x)
    w = far(torch.zeros_like(x))
    heads = lambda z: [z.unflatten(2, (3, 64))]
    sp.sp_rope_fwd(heads(x), tab, y=heads(y))
    sp.sp_rope_fwd(heads(v), tab, y=heads(w))
    assert same([y], [w])
    # recurrence, dense and packed
    cu = torch.tensor([0, 7, 4000, rows], dtype=torch.int32, device=DEV)
    for b, s, how in ((1, rows, None), (4, rows // 4, None), (1, rows, cu)):
        n = b if how is None else 3
        i = scan_inputs(1, n, b, s, 72, BF, 92, True)
        want = run_scan(i, n, True, how, True)
        i.update({k: [far(i[k][0])] for k in ("gate", "value", "dy")})
        o = {k: [far(torch.zeros_like(want[k][0]))]
             for k in ("y", "dgate", "dvalue")}
        o.update({k: [torch.empty_like(want[k][0])] for k in ("hT", "states", "dh0")})
        sp.sp_gated_scan_fwd(i["gate"], i["value"], h0=i["h0"], cu_seqlens=how, y=o["y"],
                             hT=o["hT"], states=o["states"])
        sp.sp_gated_scan_bwd(i["gate"], i["value"], o["states"], i["dy"], h0=i["h0"],
                             dhT=i["dhT"], cu_seqlens=how, dgate=o["dgate"], dvalue=o["dvalue"],
                             dh0=o["dh0"])
        for k in ("y", "dgate", "dvalue", "hT", "dh0"):
            assert same(o[k], want[k]), (b, k)
    # group norm: rows, tiles, held, units
    for n, l in ((rows, 1), (rows // 4, 4), (rows // 50, 50), (2, rows // 2)):
        i = norm_inputs(1, n, l, 128, BF, 93)
        want = run_norm(i, 4, "layernorm", "silu")
        i["x"], i["dy"] = [far(i["x"][0])], [far(i["dy"][0])]
        y, dx = [far(torch.zeros_like(want["y"][0]))], [far(torch.zeros_like(want["y"][0]))]
        mean, rstd = (torch.empty((n, 4), device=DEV) for _ in range(2))
        sp.sp_group_norm_fwd(i["x"], i["gamma"], i["beta"], groups=4, eps=1e-5, act="silu", y=y,
                             mean=[mean], rstd=[rstd])
        sp.sp_group_norm_bwd(i["dy"], i["x"], [mean], [rstd], i["gamma"], i["beta"], groups=4,
                             act="silu", dx=dx)
        assert same(y, want["y"]) and same(dx, want["dx"]), (n, l)
