"""The operators between g and the next g* where digits are easily lost, against
float64: gates that shut or stay open, values that are not finite, groups without
spread, widths and counts at a rule's edge.

Units of rounding: an output of type T is its exact value rounded once (STEP), and
what float32 arithmetic does before is counted in 2^-24 per operation.  For the
recurrence, with e = exp(-gate), a = 1 / (1 + e) and k = e a:
- e is off by DELTA: the power of two by 2^-22; for 16-bit types its argument
  gate * log2(e) by 2^-24 |gate| (the product) and 2^-26 |gate| (the constant), for
  float32 that rest is multiplied in, which leaves 2^-24;
- a is off by k DELTA and by RHO = 2^-23 + 2^-24 (the reciprocal, 1 + e);
- k is off by a DELTA, RHO and a rounding.
"""
import numpy as np
import pytest
import torch

from oracle import region as orc
from sp_boundary_norm_gb300 import binding as sp
from test_gpu_region import (BF, DEV, F32, FP, LEAST, STEP, check_norm, f64, norm_inputs,
                             rand, run_norm)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RHO = 3 * U


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


def delta(gate, dtype):
    """Relative error of exp(-gate)."""
    return 4 * U + (U if dtype is F32 else 1.25 * U * np.abs(gate))


def within(got, want, bound, what):
    """Elementwise: got is `want` rounded once, off before by at most `bound`."""
    dtype, got = got.dtype, f64(got)
    tol = STEP[dtype] * (np.abs(want) + bound) + LEAST[dtype] + bound
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, the worst by "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g} tolerances")


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def empties(like, n):
    return [torch.full_like(like, float("nan")) for _ in range(n)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tied", [True, False])
def test_scan_gradient_of_saturated_gates(dtype, tied):
    """dgate = dy a k (h0 - v): one token a sequence, gates up to 80 either way, where
    a k is 1e-35 and still a normal number."""
    gate = torch.linspace(-80, 80, 512).view(8, 1, 64).to(dtype).to(DEV)
    value, dy = torch.zeros_like(gate), torch.ones_like(gate)
    h0 = torch.ones((8, 64), device=DEV)
    y, dgate, dvalue = empties(gate, 3)
    st = torch.empty(sp.sp_gated_scan_states_shape(8, 1, 64), device=DEV)
    sp.sp_gated_scan_fwd([gate], [value], h0=[h0], tied=tied, y=[y], states=[st])
    sp.sp_gated_scan_bwd([gate], [value], [st], [dy], h0=[h0], tied=tied, dgate=[dgate],
                         dvalue=[dvalue])
    g = f64(gate)
    want = sigmoid(g) * sigmoid(-g)
    # a and k each once, two products, the difference h0 - v is exact
    within(dgate, want, want * (delta(g, dtype) + 2 * RHO + 3 * U), "dgate")


def spans_of(b, s, cu):
    """(batch row, first token, behind the last, sequence)."""
    if cu is None:
        return [(i, 0, s, i) for i in range(b)]
    return [(0, lo, hi, j) for j, (lo, hi) in enumerate(zip(cu[:-1], cu[1:]))]


def scan_exact(g, v, h0, tied, cu, dtype, dy, dhT):
    """The recurrence and its gradients in float64, and beside each a bound on what
    float32 arithmetic may lose of it, carried from token to token like the value.

    A state passes a token as a product with a (k DELTA + RHO), rounded once there and,
    in what carries it from run to run and block to block, less than twice more; k v
    adds its own a DELTA + RHO and four roundings; a value is put together from its run's
    entry and its place in at most 8.  The gradients' way back is the same with dy, one
    sum more.  Terms of second order: a hundredth at 65,537 tokens."""
    b, s, c = g.shape
    a, k, d = sigmoid(g), sigmoid(-g), delta(g, dtype)
    ra, rk = k * d + RHO, a * d + RHO + U
    o = {n: np.zeros_like(g) for n in ("y", "dgate", "dvalue", "y_", "dgate_", "dvalue_")}
    hT, hT_, dh0, dh0_ = h0.copy(), np.zeros_like(h0), dhT.copy(), np.zeros_like(h0)
    for i, lo, hi, j in spans_of(b, s, cu):
        h, m, e = h0[j], np.abs(h0[j]), np.zeros(c)
        state = [(h, m, e)]
        for p in range(lo, hi):
            ai, ki = a[i, p], k[i, p] if tied else 1.0
            w, x = ki * v[i, p], np.abs(ki * v[i, p])
            h, e = ai * h + w, ai * (e + (ra[i, p] + 3 * U) * m) + (x * (rk[i, p] + 3 * U) if tied else 0)
            m = ai * m + x
            o["y"][i, p], o["y_"][i, p] = h, e + 8 * U * m
            state.append((h, m, e + 8 * U * m))
        if hi > lo:
            hT[j], hT_[j] = h, e + 8 * U * m
        q, m, e = dhT[j], np.abs(dhT[j]), np.zeros(c)
        for p in reversed(range(lo, hi)):
            ai, ki = a[i, p], k[i, p]
            dh, dm = dy[i, p] + q, np.abs(dy[i, p]) + m
            de = e + 8 * U * dm
            prev, pm, pe = state[p - lo]
            diff, fm = (prev - v[i, p], pm + np.abs(v[i, p])) if tied else (prev, pm)
            o["dgate"][i, p] = dh * ai * ki * diff
            o["dgate_"][i, p] = ai * ki * (de * fm + dm * (pe + U * fm)
                                           + dm * fm * (ra[i, p] + rk[i, p] + 3 * U))
            o["dvalue"][i, p] = dh * ki if tied else dh
            o["dvalue_"][i, p] = ki * (de + dm * (rk[i, p] + U)) if tied else de
            q, e, m = ai * dh, ai * (e + (ra[i, p] + 4 * U) * dm), ai * dm
        dh0[j], dh0_[j] = q, e + 8 * U * m
    o.update(hT=hT, hT_=hT_, dh0=dh0, dh0_=dh0_)
    # products of many shut gates leave the range of normal numbers: not counted
    return {n: 1.01 * x + 2.0 ** -100 if n.endswith("_") else x for n, x in o.items()}


def run_scan(gate, value, dy, h0, dhT, tied, cu):
    """Forward and backward of lists of rank buffers; every output."""
    t, like = len(gate), gate[0]
    y, dgate, dvalue = (empties(like, t) for _ in range(3))
    hT, dh0 = empties(h0[0], t), empties(h0[0], t)
    st = [torch.empty(sp.sp_gated_scan_states_shape(*like.shape), device=DEV) for _ in range(t)]
    how = dict(h0=h0, tied=tied, cu_seqlens=cu)
    sp.sp_gated_scan_fwd(gate, value, y=y, hT=hT, states=st, **how)
    sp.sp_gated_scan_bwd(gate, value, st, dy, dhT=dhT, dgate=dgate, dvalue=dvalue, dh0=dh0, **how)
    return dict(y=y, hT=hT, dgate=dgate, dvalue=dvalue, dh0=dh0)


def offsets(lens):
    cu = np.concatenate(([0], np.cumsum(lens)))
    return cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("t,b,s,c,dtype,lens", [
    (1, 1, 1, 8, F32, None), (3, 64, 1, 72, BF, None), (2, 7, 1, 64, F32, None), (2, 9, 1, 64, FP, None),
    (2, 2, 17, 64, F32, None), (1, 3, 300, 72, FP, None), (1, 1, 700, 136, F32, None),
    (8, 1, 3000, 64, BF, None), (1, 1, 20001, 8, F32, None), (4, 1, 9000, 72, BF, None),
    (1, 1, 0, 72, F32, [5, 600, 0, 2, 1000, 31, 33]), (2, 1, 0, 64, BF, [1] * 40 + [0, 17, 3000]),
    (1, 1, 0, 520, FP, [4000, 1, 1500])])
@pytest.mark.parametrize("tied", [True, False])
def test_scan_keeps_the_digits_of_shut_gates(t, b, s, c, dtype, lens, tied):
    """Gates of -3 to -20 between open ones, after states of 1e4, and gradients that come
    from the last tokens only: every element within its own rounding errors."""
    cu_np, cu = (None, None) if lens is None else offsets(lens)
    s = s if lens is None else sum(lens)
    n = b if lens is None else len(lens)
    gen = torch.Generator().manual_seed(s + c)
    rnd = lambda *shape: torch.randn(shape, generator=gen)
    gate, value, dy = [], [], []
    for _ in range(t):
        shut = torch.rand((b, s, c), generator=gen) < 0.15
        gate.append(torch.where(shut, -3 - 17 * torch.rand((b, s, c), generator=gen),
                                4 + 2 * rnd(b, s, c)).to(dtype).to(DEV))
        value.append((rnd(b, s, c) * torch.exp(rnd(b, s, c))).to(dtype).to(DEV))
        late = torch.zeros(b, s, c)
        for i, lo, hi, _ in spans_of(b, s, cu_np):
            late[i, max(lo, hi - 3):hi] = 1
        late[..., ::2] = 1                       # every other channel: gradients everywhere
        dy.append((rnd(b, s, c) * late).to(dtype).to(DEV))
    h0 = [(1e4 * rnd(n, c)).to(DEV) for _ in range(t)]
    dhT = [rnd(n, c).to(DEV) for _ in range(t)]
    o = run_scan(gate, value, dy, h0, dhT, tied, cu)
    for r in range(t):
        w = scan_exact(f64(gate[r]), f64(value[r]), f64(h0[r]), tied, cu_np, dtype, f64(dy[r]),
                       f64(dhT[r]))
        for name, got in o.items():
            within(got[r], w[name], w[name + "_"], f"{name}[{r}]")


def scan_plain(g, v, h0, cu):
    """y of the tied recurrence token by token in 32 bits: a = sigmoid(g), a h + k v."""
    one = np.float32(1)
    a = one / (one + np.exp(-g.astype(np.float64)).astype(np.float32))
    kv = one / (one + np.exp(g.astype(np.float64)).astype(np.float32)) * v
    y = np.zeros_like(g)
    for i, lo, hi, j in spans_of(1, g.shape[1], cu):
        h = h0[j]
        for p in range(lo, hi):
            h = a[i, p] * h + kv[i, p]
            y[i, p] = h
    return y


@pytest.mark.parametrize("dtype,lens", [(F32, None), (BF, None), (F32, [40000, 25537])])
def test_scan_keeps_the_digits_of_open_gates(dtype, lens):
    """Memories of hundreds to 1e5 tokens over 65,537 of them: within the bound, and
    (float32) no further from the exact values than the same formula token by token."""
    cu_np, cu = (None, None) if lens is None else offsets(lens)
    n = 1 if lens is None else 2
    gen = torch.Generator().manual_seed(65)
    rnd = lambda *shape: torch.randn(shape, generator=gen)
    gate = (torch.linspace(6, 12, 16) + rnd(1, 65537, 16)).to(dtype).to(DEV)
    value, dy = rnd(1, 65537, 16).to(dtype).to(DEV), rnd(1, 65537, 16).to(dtype).to(DEV)
    h0, dhT = rnd(n, 16).to(DEV), rnd(n, 16).to(DEV)
    o = run_scan([gate], [value], [dy], [h0], [dhT], True, cu)
    w = scan_exact(f64(gate), f64(value), f64(h0), True, cu_np, dtype, f64(dy), f64(dhT))
    for name, got in o.items():
        within(got[0], w[name], w[name + "_"], name)
    if dtype is F32:
        plain = scan_plain(*(x.cpu().numpy() for x in (gate, value, h0)), cu_np)
        off = lambda y: np.abs(y - w["y"]).max((0, 1))
        mine, its = off(f64(o["y"][0])), off(plain)
        print("off, of the state:", (mine / np.abs(w["y"]).max((0, 1))).max(),
              "token by token:", (its / np.abs(w["y"]).max((0, 1))).max())
        assert mine.max() <= its.max()


@pytest.mark.parametrize("s", [1, 12])
@pytest.mark.parametrize("tied", [True, False])
def test_scan_infinite_states_stay_infinite(s, tied):
    """a h + k v of an infinite h is infinite (a > 0), as the definition has it."""
    gate = torch.linspace(-3, 6, 2 * s * 64).view(2, s, 64).to(DEV)
    value, h0 = torch.randn_like(gate), torch.full((2, 64), float("inf"), device=DEV)
    h0[1] = -h0[1]
    y, hT = empties(gate, 1), empties(h0, 1)
    sp.sp_gated_scan_fwd([gate], [value], h0=[h0], tied=tied, y=y, hT=hT)
    assert torch.equal(y[0], h0[:, None].expand(2, s, 64)) and torch.equal(hT[0], h0)


@pytest.mark.parametrize("t,c", [(1, 64), (8, 512)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_packed_sequences_keep_what_is_not_finite(t, c, dtype):
    """One NaN in a sequence of 4000 tokens, where products of a underflow after some 150:
    every later y and hT of the sequence is NaN, every earlier gradient for a NaN in dy, as
    in a dense call of that sequence; nothing else changes."""
    cu_np, cu = offsets([700, 4000, 0, 300])
    lo, hi, s = 700, 4700, 5000
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *shape: torch.randn(shape, generator=gen)
    mk = lambda *shape, d=dtype: [rnd(*shape).to(d).to(DEV) for _ in range(t)]
    gate, value, dy = mk(1, s, c), mk(1, s, c), mk(1, s, c)
    h0, dhT = mk(4, c, d=F32), mk(4, c, d=F32)
    nan = lambda x: torch.isnan(x).all()
    clean = run_scan(gate, value, dy, h0, dhT, True, cu)
    part = lambda xs: [x[:, lo:hi].contiguous() for x in xs]
    one = lambda xs: [x[1:2].contiguous() for x in xs]

    bad = [v.clone() for v in value]
    for v in bad:
        v[0, lo + 5] = float("nan")
    o = run_scan(gate, bad, dy, h0, dhT, True, cu)
    d = run_scan(part(gate), part(bad), part(dy), one(h0), one(dhT), True, None)
    for r in range(t):
        y = o["y"][r][0]
        assert nan(y[lo + 5:hi]) and torch.isfinite(y[:lo + 5]).all() and torch.isfinite(y[hi:]).all()
        assert nan(o["hT"][r][1]) and nan(d["hT"][r]) and nan(d["y"][r][0, 5:])
        for name in ("y", "dgate", "dvalue"):
            a, b = o[name][r][0], clean[name][r][0]
            assert torch.equal(a[:lo], b[:lo]) and torch.equal(a[hi:], b[hi:]), name
        for name in ("hT", "dh0"):
            assert torch.equal(o[name][r][[0, 2, 3]], clean[name][r][[0, 2, 3]]), name

    bad = [v.clone() for v in dy]
    for v in bad:
        v[0, hi - 7] = float("nan")
    o = run_scan(gate, value, bad, h0, dhT, True, cu)
    for r in range(t):
        for name in ("dgate", "dvalue"):
            a, b = o[name][r][0], clean[name][r][0]
            assert nan(a[lo:hi - 6]) and torch.isfinite(a[hi - 6:]).all()
            assert torch.equal(a[:lo], b[:lo]) and torch.equal(a[hi:], b[hi:]), name
        assert nan(o["dh0"][r][1])
        assert torch.equal(o["dh0"][r][[0, 2, 3]], clean["dh0"][r][[0, 2, 3]])

    for h in h0:
        h[1] = float("inf")
    o = run_scan(gate, value, dy, h0, dhT, True, cu)
    for r in range(t):
        y = o["y"][r][0]
        assert not torch.isfinite(y[lo:hi]).any() and not torch.isfinite(o["hT"][r][1]).any()
        assert torch.isfinite(y[:lo]).all() and torch.isfinite(y[hi:]).all()


@pytest.mark.parametrize("s,step,back", [(20000, 0, False), (20000, 3, True), (1600, 0, False)])
def test_scan_waits_end_and_say_so(s, step, back):
    """Block 0 withholds a join's map once: every wait for it runs out, the call's status
    word says so, and the next call is right."""
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *shape: torch.randn(shape, generator=gen).to(DEV)
    gate, value, dy, h0 = [rnd(1, s, 64)], [rnd(1, s, 64)], [rnd(1, s, 64)], [rnd(1, 64)]
    y, dgate, dvalue = (empties(gate[0], 1) for _ in range(3))
    st = [torch.empty(sp.sp_gated_scan_states_shape(1, s, 64), device=DEV)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        if back:
            sp.sp_gated_scan_bwd(gate, value, st, dy, h0=h0, dgate=dgate, dvalue=dvalue,
                                 status=status)
            return dgate + dvalue
        sp.sp_gated_scan_fwd(gate, value, h0=h0, y=y, states=st, status=status)
        return y + st

    sp.sp_gated_scan_fwd(gate, value, h0=h0, y=y, states=st)
    want = [x.clone() for x in call()]
    assert status.item() == 0
    sp.sp_debug_scan_withhold(step)
    call()
    torch.cuda.synchronize()
    assert status.item() == 5
    status.zero_()
    if back:
        sp.sp_gated_scan_fwd(gate, value, h0=h0, y=y, states=st)
    got = call()
    torch.cuda.synchronize()
    assert status.item() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- group norm --

@pytest.mark.parametrize("n,l,c,groups,dtype", [
    (2, 5, 2 * 2056, 2, BF), (3, 3, 2 * 2056, 2, FP), (1, 300, 3 * 2056, 3, BF),
    (2, 5, 2 * 4088, 2, F32), (1, 65, 4 * 4088, 4, BF), (1, 40, 5 * 3000, 5, F32)])
@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
def test_group_norm_wide_odd_groups(n, l, c, groups, dtype, norm):
    """Groups of an odd number of vectors beyond 256, two and more in a row."""
    i = norm_inputs(1, n, l, c, dtype, 51)
    check_norm(i, run_norm(i, groups, norm, "silu"), groups, norm, "silu")


@pytest.mark.parametrize("n,l,c,groups", [
    (9, 1, 128, 2), (7, 1, 240, 2), (3, 1, 4096, 1), (3, 6, 40, 1), (6, 4, 512, 8), (3, 50, 1360, 17),
    (40, 24, 40, 5), (2, 800, 64, 4), (1, 5001, 72, 3), (1, 9000, 4096, 2), (2, 3000, 64, 1)])
@pytest.mark.parametrize("dtype,value,eps", [(BF, 1000.0, 1e-5), (FP, 30000.0, 1e-6),
                                             (F32, -1000.5, 1e-6)])
def test_group_norm_without_spread(n, l, c, groups, dtype, value, eps):
    """All values of a sample alike and far from zero, of which every sum is exact: x - mean
    is zero, so y = beta and dgamma = 0 to the bit, in every form; dx = rstd (dz - mean dz)
    within its own roundings."""
    i = norm_inputs(1, n, l, c, dtype, 52)
    i["x"][0].fill_(value)
    o = run_norm(i, groups, "layernorm", "none", eps)
    assert (o["mean"][0] == value).all()
    assert torch.equal(o["y"][0], i["beta"].expand(n, l, c))
    assert (o["dgamma"] == 0).all()
    rstd = f64(o["rstd"][0])
    assert np.abs(rstd * eps ** 0.5 - 1).max() < 4 * U     # 1 / sqrt, eps in 32 bits
    dz = (f64(i["dy"][0]) * f64(i["gamma"])).reshape(n, l, groups, -1)
    m = dz.mean((1, 3), keepdims=True)
    want = (dz - m) * rstd[:, None, :, None]
    # dz's product, the sum's roundings (below 2^7 in a row and its partial sums: 2^8) and
    # the mean, a difference, a product
    mag = np.abs(dz) + 2.0 ** 8 * np.abs(dz).mean((1, 3), keepdims=True)
    bound = (4 * U * mag * rstd[:, None, :, None]).reshape(n, l, c)
    within(o["dx"][0], want.reshape(n, l, c), bound, "dx")


@pytest.mark.parametrize("n,l,c,groups", [(4, 1, 128, 2), (3, 6, 40, 1), (3, 50, 1360, 17), (2, 800, 64, 2)])
def test_group_norm_infinite_mean(n, l, c, groups):
    """One infinity in a group: its mean is infinite, other groups keep their bits."""
    i = norm_inputs(1, n, l, c, BF, 53)
    want = run_norm(i, groups, "layernorm", "silu")
    i["x"][0][0, 0, 0] = float("inf")
    o = run_norm(i, groups, "layernorm", "silu")
    assert o["mean"][0][0, 0] == float("inf") and not torch.isfinite(o["y"][0][0, 0, 0])
    for name in ("mean", "rstd"):
        assert torch.equal(o[name][0].flatten()[1:], want[name][0].flatten()[1:])
    assert torch.equal(o["y"][0][1:], want["y"][0][1:])


# ------------------------------------------------------------------ sigmoids --

@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_sigmoids_of_the_recurrence(dtype):
    """a and k of one token over all gates, as float32 states: h0 = 1 and no value gives a,
    h0 = 0 and a value of 1 gives k."""
    gate = torch.linspace(-86.5, 86.5, 1 << 16).view(64, 1, 1024).to(dtype).to(DEV)
    one, zero = torch.ones((64, 1024), device=DEV), torch.zeros((64, 1024), device=DEV)
    y, g = torch.empty_like(gate), f64(gate)[:, 0]
    a, k = empties(one, 1)[0], empties(one, 1)[0]
    sp.sp_gated_scan_fwd([gate], [torch.zeros_like(gate)], h0=[one], tied=False, y=[y], hT=[a])
    sp.sp_gated_scan_fwd([gate], [torch.ones_like(gate)], h0=[zero], tied=True, y=[y], hT=[k])
    d = delta(g, dtype)
    within(a, sigmoid(g), sigmoid(g) * (sigmoid(-g) * d + RHO + U), "a")
    within(k, sigmoid(-g), sigmoid(-g) * (sigmoid(g) * d + RHO + 2 * U), "k")
    # beyond: at most 2^-125, and 1
    gate = torch.tensor([88.0, 100.0, 3e4, float("inf")], device=DEV).to(dtype)
    gate = torch.cat((-gate, gate)).view(8, 1, 1).expand(8, 1, 1024).contiguous()
    y = torch.empty_like(gate)
    sp.sp_gated_scan_fwd([gate], [torch.zeros_like(gate)], h0=[one[:8]], tied=False, y=[y], hT=[a[:8]])
    sp.sp_gated_scan_fwd([gate], [torch.ones_like(gate)], h0=[zero[:8]], tied=True, y=[y], hT=[k[:8]])
    assert (a[:4] >= 0).all() and (a[:4] <= 2.0 ** -125).all() and (a[4:8] == 1).all()
    assert (k[4:8] >= 0).all() and (k[4:8] <= 2.0 ** -125).all() and (k[:4] - 1).abs().max() <= 4 * U


@pytest.mark.parametrize("l", [1, 3, 40, 700])
def test_silu_of_group_norm(l):
    """gamma = 0: y = silu(beta), float32, in every form; beside it the library's own."""
    beta = torch.linspace(-95, 95, 4096)
    i = norm_inputs(1, 2, l, 4096, F32, 54)
    i["gamma"].zero_()
    i["beta"].copy_(beta)
    o = run_norm(i, 8, "layernorm", "silu")
    q = f64(i["beta"])
    want = np.broadcast_to(q * sigmoid(q), (2, l, 4096))
    # below -87.3 the sigmoid is flushed: at most 95 * 2^-125 is lost
    bound = np.abs(want) * (sigmoid(-q) * delta(q, F32) + RHO + U) + 95 * 2.0 ** -125
    within(o["y"][0], want, bound, "y")
    near = np.abs(q) < 80
    off = lambda y: (np.abs(y - want) / np.abs(want))[..., near].max() / U
    print("off in 2^-24:", off(f64(o["y"][0])), "torch:",
          off(f64(torch.nn.functional.silu(i["beta"])).reshape(1, 1, -1)))


# -------------------------------------------------------------------- rotary --

@pytest.mark.parametrize("t,heads,d,layout,dtype", [
    (1, 9, 128, "half", BF), (2, 5, 80, "interleaved", FP), (1, 7, 24, "half", F32)])
@pytest.mark.parametrize("s", [1, 37, 811, 1216, 2431, 2433, 4863, 4865, 9727, 9729, 20011])
def test_rope_around_the_chunk_rule(t, heads, d, layout, dtype, s):
    """Token counts on both sides of the rule that cuts few tokens' heads into pieces (of
    whole lane rounds, the last one short) and of the grid's warps, beyond which a warp
    takes one token after the other."""
    gen = torch.Generator().manual_seed(s)
    x = [rand((1, s, heads, d), gen, dtype) for _ in range(t)]
    y = empties(x[0], t)
    tab = sp.sp_rope_table(d - 8)
    sp.sp_rope_fwd(x, tab, layout=layout, first_position=5, y=y)
    at = np.unique(np.concatenate((np.arange(min(s, 20)), np.arange(max(0, s - 20), s),
                                   np.random.default_rng(s).integers(0, s, 200))))
    for r in range(t):
        want, mag = orc.rope(f64(x[r])[:, at], orc.positions(1, s, 5)[:, at],
                             orc.frequencies(d - 8), layout)
        # under 8 units of 2^-24, as for the other rotary tests
        within(y[r][:, at], want, 2.0 ** -21 * mag, f"rank {r}")
        assert torch.isfinite(y[r]).all()


# ------------------------------------------------------------ the widest calls --

@pytest.mark.parametrize("t,heads,d,rot", [(16, 4096, 8, 8), (16, 4095, 10, 4), (1, 1, 16384, 512)])
def test_rope_most_heads_and_widest(t, heads, d, rot):
    gen = torch.Generator().manual_seed(7)
    x = [rand((1, 3, heads, d), gen, BF) for _ in range(t)]
    y = empties(x[0], t)
    sp.sp_rope_fwd(x, sp.sp_rope_table(rot), layout="interleaved", y=y)
    for r in range(t):
        want, mag = orc.rope(f64(x[r]), orc.positions(1, 3), orc.frequencies(rot), "interleaved")
        within(y[r], want, 2.0 ** -21 * mag, f"rank {r}")


@pytest.mark.parametrize("lens", [None, [0] * 3000 + [1, 0, 38] + [0] * 5000])
def test_scan_most_channels_and_many_empty_sequences(lens):
    cu_np, cu = (None, None) if lens is None else offsets(lens)
    n, s, c = 1 if lens is None else len(lens), 39, 16384 if lens is None else 72
    gen = torch.Generator().manual_seed(8)
    mk = lambda shape, dt: [rand(shape, gen, dt) for _ in range(2)]
    gate, value, dy = mk((1, s, c), BF), mk((1, s, c), BF), mk((1, s, c), BF)
    h0, dhT = mk((n, c), F32), mk((n, c), F32)
    o = run_scan(gate, value, dy, h0, dhT, True, cu)
    for r in range(2):
        w = scan_exact(f64(gate[r]), f64(value[r]), f64(h0[r]), True, cu_np, BF, f64(dy[r]), f64(dhT[r]))
        for name, got in o.items():
            within(got[r], w[name], w[name + "_"], f"{name}[{r}]")


@pytest.mark.parametrize("n,l,groups", [(5, 1, 2048), (3, 9, 2048), (2, 300, 4), (70, 2, 16)])
def test_group_norm_most_channels(n, l, groups):
    i = norm_inputs(2, n, l, 16384, FP, 55)
    check_norm(i, run_norm(i, groups, "layernorm", "silu"), groups, "layernorm", "silu")
