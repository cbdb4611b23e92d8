"""The oracle of the state space layer and of rotary positions with several axes, tied
to something other than itself."""
import numpy as np
import pytest
import torch

from oracle import region, state_space as orc


def test_axes_by_hand():
    axis, w = orc.axes_table([1, 2, 1], base=16.0)
    assert axis.tolist() == [0, 1, 1, 2] and np.allclose(w, [1, 0.5, 0.25, 0.125])
    axis, w = orc.axes_table([1, 3, 2], base=8.0, order="cyclic")
    assert axis.tolist() == [0, 1, 2, 1, 2, 1] and np.allclose(w, 8.0 ** (-np.arange(6) / 6))
    axis, w = orc.axes_table([2, 4], base=16.0, frequencies="own", factors=[4.0, 1.0])
    assert axis.tolist() == [0, 0, 1, 1, 1, 1] and np.allclose(w, [0.25, 1 / 16, 1, 0.5, 0.25, 0.125])


def test_one_axis_is_plain_rotary():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 5, 3, 20))
    axis, w = orc.axes_table([8])
    pos = region.positions(2, 5, 77)
    for layout in ("half", "interleaved"):
        for back in (False, True):
            want, _ = region.rope(x, pos, region.frequencies(16), layout, 1.25, back)
            got, _ = orc.rope_axes(x, pos[None], axis, w, layout, 1.25, back)
            assert np.allclose(got, want)


def test_axes_are_relative_and_separate():
    rng = np.random.default_rng(2)
    axis, w = orc.axes_table([3, 5], order="cyclic", frequencies="own")
    q, k = rng.normal(size=(2, 1, 1, 1, 16))
    at = lambda x, p: orc.rope_axes(x, np.array(p).reshape(2, 1, 1), axis, w)[0]
    dot = lambda i, j: (at(q, i) * at(k, j)).sum()
    assert np.isclose(dot((5, -9), (2, 4)), dot((1000003, 91), (1000000, 104)))
    # the second coordinate turns its own pairs alone
    moved = np.abs(at(q, (3, 7)) - at(q, (3, 8))).ravel() > 1e-12
    assert (moved[:8] == (axis == 1)).all() and (moved[8:] == (axis == 1)).all()


def test_conv_is_torchs():
    rng = np.random.default_rng(3)
    for w in (2, 3, 4):
        x, k, bias = rng.normal(size=(2, 7, 3)), rng.normal(size=(3, w)), rng.normal(size=3)
        t = torch.from_numpy
        want = torch.nn.functional.conv1d(t(x).transpose(1, 2), t(k)[:, None], t(bias),
                                          padding=w - 1, groups=3)[..., :7].transpose(1, 2)
        assert np.allclose(orc.causal_conv(x, k, bias)["y"], want)
        assert np.allclose(orc.causal_conv(x, k, bias, "silu")["y"],
                           torch.nn.functional.silu(want))


def test_conv_states_join_pieces():
    rng = np.random.default_rng(4)
    x, k = rng.normal(size=(1, 11, 2)), rng.normal(size=(2, 4))
    whole = orc.causal_conv(x, k)
    state, rows = None, []
    for lo, hi in ((0, 1), (1, 1), (1, 3), (3, 11)):
        f = orc.causal_conv(x[:, lo:hi], k, x0=state)
        state = f["xT"]
        rows.append(f["y"])
    assert np.allclose(np.concatenate(rows, 1), whole["y"]) and np.allclose(state, whole["xT"])
    # packed sequences are separate calls
    cu = [0, 3, 3, 4, 11]
    x0 = rng.normal(size=(4, 3, 2))
    f = orc.causal_conv(x, k, x0=x0, cu_seqlens=cu)
    for j, (lo, hi) in enumerate(zip(cu, cu[1:])):
        g = orc.causal_conv(x[:, lo:hi], k, x0=x0[j:j + 1])
        assert np.allclose(f["y"][:, lo:hi], g["y"]) and np.allclose(f["xT"][j], g["xT"][0])


def numeric(f, args, name, eps=1e-6):
    """Central differences of f(**args) by args[name]."""
    x = args[name]
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + eps
        hi = f(**args)
        x[i] = keep - eps
        out[i] = (hi - f(**args)) / (2 * eps)
        x[i] = keep
    return out


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 3, 8]])
def test_conv_gradients_by_differences(act, cu):
    rng = np.random.default_rng(5)
    n = 2 if cu is None else 4
    b = 2 if cu is None else 1
    args = dict(x=rng.normal(size=(b, 8, 2)), weight=rng.normal(size=(2, 4)),
                bias=rng.normal(size=2), x0=rng.normal(size=(n, 3, 2)))
    dy, dxT = rng.normal(size=(b, 8, 2)), rng.normal(size=(n, 3, 2))

    def loss(**a):
        f = orc.causal_conv(act=act, cu_seqlens=cu, **a)
        return (f["y"] * dy).sum() + (f["xT"] * dxT).sum()

    got = orc.causal_conv_bwd(dy=dy, act=act, cu_seqlens=cu, dxT=dxT, **args)
    for name in args:
        want = numeric(loss, args, name)
        assert np.allclose(got["d" + name], want, atol=1e-7), name
        assert (got["mag_d" + name] >= np.abs(got["d" + name]) - 1e-12).all()


def test_scan_closed_form():
    """Constant inputs: a geometric sum."""
    n = 9
    u, dt = np.full((1, n, 1), 2.0), np.full((1, n, 1), 0.3)
    A, B, C = np.array([[-1.0, -0.5]]), np.full((1, n, 2), 3.0), np.full((1, n, 2), 0.25)
    d = np.log1p(np.exp(0.3 + 0.1))
    f = orc.selective_scan(u, dt, A, B, C, D=np.array([5.0]), dt_bias=np.array([0.1]))
    a = np.exp(d * A[0])
    want = d * 2 * 3 * (1 - a ** n) / (1 - a)
    assert np.allclose(f["hT"][0, 0], want)
    assert np.isclose(f["y"][0, -1, 0], 0.25 * want.sum() + 10)
    g = orc.selective_scan(u, dt, A, B, C, z=np.full((1, n, 1), 1.5), use_softplus=False)
    a = np.exp(0.3 * A[0])
    want = 0.3 * 2 * 3 * (1 - a ** n) / (1 - a) * 0.25
    assert np.isclose(g["y"][0, -1, 0], want.sum() * 1.5 / (1 + np.exp(-1.5)))


def scan_args(cu, groups, gated, seed=6):
    rng = np.random.default_rng(seed)
    b, s, c, n = (2, 5, 4, 3) if cu is None else (1, cu[-1], 4, 3)
    seqs = b if cu is None else len(cu) - 1
    args = dict(u=rng.normal(size=(b, s, c)), dt=rng.normal(size=(b, s, c)),
                A=-rng.uniform(0.2, 2, size=(c, n)), B=rng.normal(size=(b, s, groups * n)),
                C=rng.normal(size=(b, s, groups * n)), D=rng.normal(size=c),
                dt_bias=rng.normal(size=c), h0=rng.normal(size=(seqs, c, n)))
    if gated:
        args["z"] = rng.normal(size=(b, s, c))
    return args, rng.normal(size=(b, s, c)), rng.normal(size=(seqs, c, n))


@pytest.mark.parametrize("cu,groups,gated,soft", [
    (None, 1, True, True), (None, 2, False, True), ([0, 2, 2, 3, 7], 2, True, False),
    ([0, 0, 4], 4, True, True)])
def test_scan_gradients_by_differences(cu, groups, gated, soft):
    args, dy, dhT = scan_args(cu, groups, gated)

    def loss(**a):
        f = orc.selective_scan(cu_seqlens=cu, use_softplus=soft, **a)
        return (f["y"] * dy).sum() + (f["hT"] * dhT).sum()

    got = orc.selective_scan(cu_seqlens=cu, use_softplus=soft, dy=dy, dhT=dhT, **args)
    # the two losses of a difference are each rounded by 2^-53 of their size, over 2e-6
    # (steps that may be negative let states grow: the loss is some 5e4 there)
    atol = 2e-6 + abs(loss(**args)) * 2.0 ** -52 / 1e-6
    for name in args:
        want = numeric(loss, args, name)
        assert np.allclose(got["d" + name], want, atol=atol), name
        assert (got["mag_d" + name] >= np.abs(got["d" + name]) - 1e-12).all(), name
    assert (got["mag_y"] >= np.abs(got["y"]) - 1e-12).all()


def test_scan_pieces_join_and_sequences_are_separate():
    args, _, _ = scan_args(None, 2, True)
    whole = orc.selective_scan(**args)
    per_token = ("u", "dt", "B", "C", "z")
    state, rows = args["h0"], []
    for lo, hi in ((0, 1), (1, 1), (1, 5)):
        a = {k: v[:, lo:hi] if k in per_token else v for k, v in args.items()}
        f = orc.selective_scan(**dict(a, h0=state))
        state = f["hT"]
        rows.append(f["y"])
    assert np.allclose(np.concatenate(rows, 1), whole["y"]) and np.allclose(state, whole["hT"])
    cu = [0, 2, 2, 3, 7]
    args, _, _ = scan_args(cu, 1, False)
    f = orc.selective_scan(cu_seqlens=cu, **args)
    for j, (lo, hi) in enumerate(zip(cu, cu[1:])):
        a = {k: v[:, lo:hi] if k in per_token else v for k, v in args.items()}
        g = orc.selective_scan(**dict(a, h0=args["h0"][j:j + 1]))
        assert np.allclose(f["y"][:, lo:hi], g["y"]) and np.allclose(f["hT"][j], g["hT"][0])
