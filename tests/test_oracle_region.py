"""The oracle of the operators between g and the next g*, tied to something
other than itself."""
import numpy as np
import pytest
import torch

from oracle import region as orc


def test_rotation_by_hand():
    # a quarter turn at position 1 with frequency pi / 2, both layouts
    w = np.array([np.pi / 2, 0.0])
    x = np.arange(1.0, 6.0).reshape(1, 1, 1, 5)
    y, _ = orc.rope(x, np.array([[1]]), w, "half")
    assert np.allclose(y.ravel(), [-3, 2, 1, 4, 5])
    y, _ = orc.rope(x, np.array([[1]]), w, "interleaved")
    assert np.allclose(y.ravel(), [-2, 1, 3, 4, 5])
    back, _ = orc.rope(y, np.array([[1]]), w, "interleaved", back=True)
    assert np.allclose(back, x)
    y, _ = orc.rope(x, np.array([[1]]), w, "half", mscale=2.0)
    assert np.allclose(y.ravel(), [-6, 4, 2, 8, 5])


def test_rotation_is_the_complex_product_and_relative():
    rng = np.random.default_rng(1)
    w = orc.frequencies(16)
    assert w[0] == 1 and np.isclose(w[4], 0.01)
    q, k = rng.normal(size=(1, 1, 1, 16)), rng.normal(size=(1, 1, 1, 16))
    z = (q[..., ::2] + 1j * q[..., 1::2]) * np.exp(1j * 7 * w)
    y, _ = orc.rope(q, np.array([[7]]), w, "interleaved")
    assert np.allclose(y[..., ::2] + 1j * y[..., 1::2], z)
    dot = lambda i, j: (orc.rope(q, np.array([[i]]), w)[0] * orc.rope(k, np.array([[j]]), w)[0]).sum()
    assert np.isclose(dot(5, 2), dot(1000003, 1000000))


def test_scaled_frequencies():
    plain = orc.frequencies(64, 500000.0)
    assert np.allclose(orc.frequencies(64, 500000.0, "linear", 4.0), plain / 4)
    base = orc.frequencies(64, 500000.0, "base", 4.0)
    assert base[0] == 1 and np.isclose(base[-1], plain[-1] / 4)
    parts = orc.frequencies(64, 500000.0, "parts", 8.0, 8192, 1.0, 4.0)
    turns = 8192 * plain / (2 * np.pi)
    assert np.allclose(parts[turns >= 4], plain[turns >= 4])
    assert np.allclose(parts[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((parts[mid] < plain[mid]) & (parts[mid] > plain[mid] / 8)).all()


def test_packed_positions():
    p = orc.positions(1, 6, first=10, cu_seqlens=[0, 2, 2, 3, 6])
    assert p.tolist() == [[10, 11, 10, 10, 11, 12]]


def test_scan_closed_form_and_packing():
    rng = np.random.default_rng(2)
    g, v = rng.normal(size=(1, 9, 3)), rng.normal(size=(1, 9, 3))
    h0 = rng.normal(size=(4, 3))
    cu = [0, 4, 4, 5, 9]
    for tied in (True, False):
        f = orc.gated_scan(g, v, h0, tied, cu)
        a = 1 / (1 + np.exp(-g))
        u = (1 - a) * v if tied else v
        for j, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
            for i in range(lo, hi):
                want = np.prod(a[0, lo:i + 1], 0) * h0[j]
                for m in range(lo, i + 1):
                    want = want + np.prod(a[0, m + 1:i + 1], 0) * u[0, m]
                assert np.allclose(f["y"][0, i], want)
            assert np.allclose(f["hT"][j], f["y"][0, hi - 1] if hi > lo else h0[j])


def _differences(fn, x, w, step=1e-6):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = fn()
        x[i] = keep - step
        out[i] = ((hi - fn()) * w).sum() / (2 * step)
        x[i] = keep
    return out


@pytest.mark.parametrize("tied", [True, False])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 7]])
def test_scan_gradients_by_differences(tied, cu):
    rng = np.random.default_rng(3)
    b = 1 if cu else 2
    n = len(cu) - 1 if cu else b
    g, v, dy = (rng.normal(size=(b, 7, 2)) for _ in range(3))
    h0, dhT = rng.normal(size=(n, 2)), rng.normal(size=(n, 2))
    got = orc.gated_scan_bwd(g, v, dy, h0, dhT, tied, cu)
    both = np.concatenate((dy.ravel(), dhT.ravel()))

    def run():
        f = orc.gated_scan(g, v, h0, tied, cu)
        return np.concatenate((f["y"].ravel(), f["hT"].ravel()))

    for name, x in (("dgate", g), ("dvalue", v), ("dh0", h0)):
        assert np.allclose(got[name], _differences(run, x, both), atol=1e-8), name


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_gradients_by_differences(norm, act):
    rng = np.random.default_rng(4)
    x, dy = rng.normal(1, 1, size=(2, 3, 8)), rng.normal(size=(2, 3, 8))
    gamma, beta = rng.normal(1, 0.3, size=8), rng.normal(size=8)
    got = orc.group_norm_bwd(dy, x, gamma, beta, 2, 1e-5, norm, act)
    run = lambda: orc.group_norm(x, gamma, beta, 2, 1e-5, norm, act)["y"]
    for name, w in (("dx", x), ("dgamma", gamma)) + ((("dbeta", beta),) if norm == "layernorm" else ()):
        assert np.allclose(got[name], _differences(run, w, dy), atol=1e-7), name


def test_group_norm_is_torchs():
    rng = np.random.default_rng(5)
    x, gamma, beta = rng.normal(2, 3, size=(3, 5, 24)), rng.normal(size=24), rng.normal(size=24)
    got = orc.group_norm(x, gamma, beta, 3, 1e-5)
    t = lambda a: torch.from_numpy(a)
    want = torch.nn.functional.group_norm(t(x).transpose(1, 2), 3, t(gamma), t(beta), 1e-5)
    assert np.allclose(got["y"], want.transpose(1, 2).numpy())
    got = orc.group_norm(x, gamma, beta, 3, 1e-5, act="silu")
    assert np.allclose(got["y"], torch.nn.functional.silu(want).transpose(1, 2).numpy())
