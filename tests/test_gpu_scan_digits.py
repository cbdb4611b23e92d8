"""What a state of the selective scan keeps of its digits over thousands of tokens.

Decays alone (u = 0, dy = 0): a last state is its first one times exp(sum of d A), and
the gradient of the first state that of the last times the same.  In units of U = 2^-24,
as roundings whose errors follow no pattern (rms below U / sqrt(3) each): a token multiplies
the state and the product of a step's decays, and each decay has an error of its own, below
2^-22.8 or 2.3 U, which is 0.6 U in the rms.  Four such a token, so sqrt(4 n / 3) U over n
tokens, 3.2e-6 for 2048.  To one side only the power of a step's summed exponents is off,
by at most 2^-25 on the mean where these states have theirs (between -0.5 and 0), once in
eight tokens: 2048 / 8 2^-25 = 7.6e-6 at most.  Their sum in norm is below 2^-16.5; tokens
that take the hardware's power alone are off by 2e-8 each to one side, 4e-5 in all.
"""
import numpy as np
import pytest
import torch

from sp_boundary_norm_gb300 import binding as sp
from _scan_norms import off_in_norm
from test_gpu_state_space import BF, DEV, F32, FP, f64, nans, offsets, run_ssm, scratch, ssm_inputs

pytestmark = pytest.mark.gpu

WITHIN = 2.0 ** -16.5


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


def decays(b, s, c, n, dtype, seed):
    """Steps between 2^-8 and 3 2^-8, rates between -1.5 and -0.3: exponents (of two)
    between -0.026 and -0.0017 a token."""
    gen = torch.Generator().manual_seed(seed)
    uniform = lambda shape, lo, hi: torch.rand(shape, generator=gen) * (hi - lo) + lo
    return dict(dt=uniform((b, s, c), 1.0, 3.0).mul_(2.0 ** -8).to(dtype).to(DEV),
                A=-uniform((c, n), 0.3, 1.5).to(DEV), h=uniform((b, c, n), 1.0, 2.0).to(DEV),
                zero=torch.zeros((b, s, c), dtype=dtype, device=DEV),
                B=uniform((b, s, n), -1.0, 1.0).to(dtype).to(DEV),
                C=uniform((b, s, n), -1.0, 1.0).to(dtype).to(DEV))


def off(got, i, tokens):
    """Relative errors in norm of a state that went through the call's tokens."""
    total = i["dt"][:, tokens].double().sum(1)
    want = i["h"].double() * torch.exp(total[..., None] * i["A"].double())
    return float(((got.double() - want) / want).square().mean().sqrt())


@pytest.mark.parametrize("c,n", [(9728, 16), (2432, 64), (64, 16), (24, 8), (40, 32)])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_slow_states_keep_their_digits(dtype, c, n):
    """In one walk (many channels), in chunks (few)."""
    s = 2048
    i = decays(1, s, c, n, dtype, 51)
    y, hT = nans(1, (1, s, c), dtype), nans(1, (1, c, n), F32)
    states = nans(1, sp.sp_selective_scan_states_shape(1, s, c, n), F32)
    args = ([i["zero"]], [i["dt"]], i["A"], [i["B"]], [i["C"]])
    how = dict(softplus=False, h0=[i["h"]])
    sp.sp_selective_scan_fwd(*args, y=y, hT=hT, states=states, **how,
                             workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, s, c, n, 1, 1)))
    assert off(hT[0], i, slice(None)) <= WITHIN
    out = {k: nans(1, (1, s, c), dtype) for k in ("du", "ddt")}
    out.update({k: nans(1, (1, s, n), dtype) for k in ("dB", "dC")})
    dh0 = nans(1, (1, c, n), F32)
    sp.sp_selective_scan_bwd(*args, states, [i["zero"]], dhT=[i["h"]], dh0=dh0, **out, **how,
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(1, s, c, n, 1, 1)))
    assert off(dh0[0], i, slice(None)) <= WITHIN


@pytest.mark.parametrize("c,n", [(8, 8), (8, 16), (16, 32)])
def test_slow_states_through_many_chunks(c, n):
    """32,768 tokens of few channels, in some 150 chunks: a state goes through the chunks'
    decays, and through the last one's tokens.  A chunk's decay is applied in two halves:
    four roundings each, sqrt(4 150 / 3) U; 220 tokens behind them sqrt(4 220 / 3) U, and
    28 2^-25 to one side: 36 U at most, of which 2^-18.5 is 45.  Halves by the hardware's
    power alone would be off to one side by 1e-8 to 2.5e-8 each, 5e-6 in all (84 U)."""
    s = 1 << 15
    i = decays(1, s, c, n, F32, 56)
    i["dt"] *= 2.0 ** -6
    i["A"] *= 2.0 / 3
    args = ([i["zero"]], [i["dt"]], i["A"], [i["B"]], [i["C"]])
    how = dict(softplus=False, h0=[i["h"]])
    y, hT = nans(1, (1, s, c), F32), nans(1, (1, c, n), F32)
    states = nans(1, sp.sp_selective_scan_states_shape(1, s, c, n), F32)
    sp.sp_selective_scan_fwd(*args, y=y, hT=hT, states=states, **how,
                             workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, s, c, n, 1, 1)))
    assert off(hT[0], i, slice(None)) <= 2.0 ** -18.5
    out = {k: nans(1, (1, s, c), F32) for k in ("du", "ddt")}
    out.update({k: nans(1, (1, s, n), F32) for k in ("dB", "dC")})
    dh0 = nans(1, (1, c, n), F32)
    sp.sp_selective_scan_bwd(*args, states, [i["zero"]], dhT=[i["h"]], dh0=dh0, **out, **how,
                             workspace=scratch(sp.sp_selective_scan_bwd_workspace_bytes(1, s, c, n, 1, 1)))
    assert off(dh0[0], i, slice(None)) <= 2.0 ** -18.5


@pytest.mark.parametrize("n", [8, 16, 32, 64])
@pytest.mark.parametrize("dtype,tokens", [(F32, 1), (BF, 2), (F32, 8), (FP, 16), (F32, 23)])
def test_a_state_updated_in_place_keeps_its_digits(dtype, tokens, n):
    """2048 tokens in calls of a few (decoding), and of more than a whole step."""
    s, c, b = 2048 // tokens * tokens, 40, 3
    i = decays(b, s, c, n, dtype, 52)
    state = [i["h"].clone()]
    for lo in range(0, s, tokens):
        cut = lambda k: [i[k][:, lo:lo + tokens].contiguous()]
        sp.sp_selective_scan_fwd(cut("zero"), cut("dt"), i["A"], cut("B"), cut("C"), softplus=False, h0=state,
                                 y=nans(1, (b, tokens, c), dtype), hT=state)
    assert off(state[0], i, slice(None)) <= WITHIN


@pytest.mark.parametrize("tokens", [1, 15])
def test_packed_states_updated_in_place_keep_their_digits(tokens):
    """The same, the sequences of a call given by their prefix sums."""
    s, c, n, b = 2048 // tokens * tokens, 40, 16, 3
    i = decays(b, s, c, n, F32, 53)
    state, cu = [i["h"].clone()], offsets([tokens] * b)
    for lo in range(0, s, tokens):
        cut = lambda k: [i[k][:, lo:lo + tokens].reshape(1, b * tokens, -1)]
        sp.sp_selective_scan_fwd(cut("zero"), cut("dt"), i["A"], cut("B"), cut("C"), softplus=False, h0=state,
                                 cu_seqlens=cu, y=nans(1, (1, b * tokens, c), F32), hT=state,
                                 workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, b * tokens, c, n, 1, 1)))
    assert off(state[0], i, slice(None)) <= WITHIN


def test_products_that_leave_the_range_on_the_way():
    """Steps of both signs (softplus off): decays of 2^100 and back.  What a step's decays
    have lost is not made up for where their product overflowed or vanished: the states
    stay what their tokens make of them, each off by its decays' 2^-22.8 and by 2^-24 of
    exponents up to 150: below 16 150 2^-24 = 2^-12.7."""
    c, n, s = 8, 16, 64
    for up in ([100.0, 100.0, -120.0, -80.0], [-90.0, -60.0, 75.0, 75.0], [-20.0, 30.0, -20.0, 10.0]):
        x = torch.tensor(up + [0.0] * 12).repeat(4)
        start = 2.0 ** -90 if up[0] > 0 else 1.0
        dt = (x / 1.4426950408889634).view(1, s, 1).expand(1, s, c).contiguous().to(DEV)
        A, h0 = torch.ones(c, n, device=DEV), [torch.full((1, c, n), start, device=DEV)]
        zero, one = torch.zeros(1, s, c, device=DEV), torch.ones(1, s, n, device=DEV)
        hT, y = nans(1, (1, c, n), F32), nans(1, (1, s, c), F32)
        states = nans(1, sp.sp_selective_scan_states_shape(1, s, c, n), F32)
        sp.sp_selective_scan_fwd([zero], [dt], A, [one], [one], softplus=False, h0=h0, y=y, hT=hT, states=states,
                                 workspace=scratch(sp.sp_selective_scan_fwd_workspace_bytes(1, s, c, n, 1, 1)))
        steps = f64(dt[0, :, 0])
        h, want = start, []
        for d in steps:
            h = h * np.exp(d)
            h = h if abs(h) >= 2.0 ** -126 else 0.0          # (a decay below that is flushed)
            want.append(16 * h)
        assert (np.abs(f64(y[0])[0] - np.array(want)[:, None]) <= 2.0 ** -12 * np.array(want)[:, None]).all(), up


@pytest.mark.parametrize("lens,state", [(None, True), ([1, 700, 0, 15, 17, 1276], True),
                                        ([1, 700, 0, 15, 17, 1276], False), ([2009], True)],
                         ids=["dense", "packed", "zeros", "one"])
@pytest.mark.parametrize("dtype,n,groups,gated", [(F32, 8, 3, True), (F32, 16, 1, False), (F32, 32, 1, True),
                                                  (F32, 64, 3, True), (BF, 16, 3, True), (FP, 32, 1, True)])
def test_every_rank_in_norm(lens, state, dtype, n, groups, gated):
    """Long sequences in chunks: every output of every rank, in norm."""
    t, c, m = 3, 24, 1 if lens is None else len(lens)
    assert sp.sp_selective_scan_fwd_workspace_bytes(1, 2009, c, n, groups, t) > 0
    i = ssm_inputs(t, m, 1, 2009, c, n, groups, dtype, 54 + n, state, gated)
    o = run_ssm(i, m, None if lens is None else offsets(lens), state)
    for r in range(t):
        assert off_in_norm(o, i, r, lens) == [], r


@pytest.mark.parametrize("dtype,t,c,n,groups", [(F32, 2, 136, 16, 1), (BF, 3, 72, 8, 3), (F32, 5, 16, 32, 1),
                                                (FP, 2, 40, 64, 1)])
@pytest.mark.parametrize("lens", [[40], [0, 0, 70, 0, 3, 1, 1, 1, 0], [16] * 9 + [0] * 4 + [17],
                                  [5, 60, 0, 2, 100, 31, 33]], ids=range(4))
@pytest.mark.parametrize("state", [True, False])
def test_every_rank_packed_in_norm(lens, dtype, t, c, n, groups, state):
    """Packed sequences with and without states of their own: every rank."""
    i = ssm_inputs(t, len(lens), 1, sum(lens), c, n, groups, dtype, 55, state)
    o = run_ssm(i, len(lens), offsets(lens), state)
    for r in range(t):
        assert off_in_norm(o, i, r, lens) == [], r
