"""Oracle of a state space layer (causal convolution, selective scan) and of rotary
positions with several axes, one rank at a time in float64, from their definitions.

Beside each result the functions give the magnitude that its float32 rounding errors
scale with: the same formula with every term's absolute value, and with the largest
magnitude of a state over all tokens in the place of the state.
Pinned by tests/test_oracle_state_space.py: by hand, by torch's convolution, by the
closed form of a scan with constant inputs, gradients by central differences.
"""
import numpy as np

from .region import _spans, sigmoid


def axes_table(sections, base=10000.0, order="blocks", frequencies="shared", factors=None):
    """Axis and radians per position of each pair of a head."""
    pairs = sum(sections)
    if order == "blocks":
        axis = [k for k, n in enumerate(sections) for _ in range(n)]
    else:
        axis = [k for j in range(max(sections)) for k, n in enumerate(sections) if j < n]
    seen = [0] * len(sections)
    freq = []
    for i, k in enumerate(axis):
        rate = i / pairs if frequencies == "shared" else seen[k] / sections[k]
        seen[k] += 1
        freq.append(base ** -rate / (1.0 if factors is None else factors[k]))
    return np.array(axis), np.array(freq)


def rope_axes(x, pos, axis, freq, layout="half", mscale=1.0, back=False):
    """x: (b, s, heads, d); pos: (axes, b, s).  Returns (y, magnitude)."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    # reduce the angle in extended precision: positions may be far
    turns = np.moveaxis(pos[axis], 0, -1).astype(np.longdouble) * (
        freq.astype(np.longdouble) / (2 * np.pi))
    ang = 2 * np.pi * (turns - np.floor(turns)).astype(np.float64)[:, :, None]
    pairs = x[..., :2 * half]
    z = pairs[..., :half] + 1j * pairs[..., half:] if layout == "half" \
        else pairs[..., ::2] + 1j * pairs[..., 1::2]
    z = z * mscale * np.exp(-1j * ang if back else 1j * ang)
    y, mag = x.copy(), np.zeros_like(x)
    u, v = (slice(0, half), slice(half, 2 * half)) if layout == "half" \
        else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y[..., u], y[..., v] = z.real, z.imag
    mag[..., u] = mag[..., v] = abs(mscale) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    return y, mag


def _silu(q):
    """silu and its derivative."""
    sg = sigmoid(q)
    return q * sg, sg * (1 + q * (1 - sg))


def causal_conv(x, weight, bias=None, act="none", x0=None, cu_seqlens=None):
    """x: (b, s, c); weight: (c, width); x0: (sequences, width - 1, c).  Returns
    dict(y, xT, q, mag)."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    b, s, c = x.shape
    w = weight.shape[1]
    spans = _spans(b, s, cu_seqlens)
    x0 = np.zeros((len(spans), w - 1, c)) if x0 is None else np.asarray(x0, np.float64)
    add = np.zeros(c) if bias is None else np.asarray(bias, np.float64)
    q, mag, xT = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x0)
    for i, lo, hi, j in spans:
        row = np.concatenate((x0[j], x[i, lo:hi]))
        xT[j] = row[len(row) - (w - 1):]
        for k in range(w):
            q[i, lo:hi] += weight[:, k] * row[k:k + hi - lo]
            mag[i, lo:hi] += np.abs(weight[:, k] * row[k:k + hi - lo])
        q[i, lo:hi] += add
        mag[i, lo:hi] += np.abs(add)
    return dict(y=_silu(q)[0] if act == "silu" else q, xT=xT, q=q, mag=mag)


def causal_conv_bwd(x, weight, dy, bias=None, act="none", x0=None, cu_seqlens=None, dxT=None):
    """Returns dict(dx, dx0, dweight, dbias) and their magnitudes (mag_...)."""
    x, weight, dy = (np.asarray(v, np.float64) for v in (x, weight, dy))
    b, s, c = x.shape
    w = weight.shape[1]
    spans = _spans(b, s, cu_seqlens)
    f = causal_conv(x, weight, bias, act, x0, cu_seqlens)
    # q's own error reaches dq through the second derivative of silu, below 1
    dq = dy * _silu(f["q"])[1] if act == "silu" else dy
    dm = np.abs(dy) * (1.1 + f["mag"]) if act == "silu" else np.abs(dy)
    x0 = np.zeros((len(spans), w - 1, c)) if x0 is None else np.asarray(x0, np.float64)
    last = np.zeros_like(x0) if dxT is None else np.asarray(dxT, np.float64)
    out = {n: np.zeros_like(v) for n, v in (("dx", x), ("dx0", x0), ("dweight", weight))}
    out["dbias"] = dq.sum((0, 1))
    mag = {"mag_" + n: np.zeros_like(v) for n, v in out.items()}
    mag["mag_dbias"] = dm.sum((0, 1))
    for i, lo, hi, j in spans:
        n = hi - lo
        row = np.concatenate((x0[j], x[i, lo:hi]))
        d, m = np.zeros((n + w - 1, c)), np.zeros((n + w - 1, c))
        for k in range(w):
            d[k:k + n] += weight[:, k] * dq[i, lo:hi]
            m[k:k + n] += np.abs(weight[:, k]) * dm[i, lo:hi]
            out["dweight"][:, k] += (dq[i, lo:hi] * row[k:k + n]).sum(0)
            mag["mag_dweight"][:, k] += (dm[i, lo:hi] * np.abs(row[k:k + n])).sum(0)
        d[n:] += last[j]
        m[n:] += np.abs(last[j])
        out["dx0"][j], mag["mag_dx0"][j] = d[:w - 1], m[:w - 1]
        out["dx"][i, lo:hi], mag["mag_dx"][i, lo:hi] = d[w - 1:], m[w - 1:]
    return dict(out, **mag)


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, use_softplus=True, h0=None,
                   cu_seqlens=None, dy=None, dhT=None):
    """u, dt, z, dy: (b, s, c); A: (c, n); B, C: (b, s, groups * n); h0, dhT: (sequences,
    c, n).  Returns dict(y, hT) and, with dy, the gradients (du, ddt, dB, dC, dz, dA, dD,
    ddt_bias, dh0), and the magnitude of each (mag_...)."""
    f64 = lambda v: None if v is None else np.asarray(v, np.float64)  # noqa: E731
    u, dt, A, B, C, D, z, dt_bias, h0, dy, dhT = map(
        f64, (u, dt, A, B, C, D, z, dt_bias, h0, dy, dhT))
    b, s, c = u.shape
    n = A.shape[1]
    groups = B.shape[2] // n
    spread = lambda v: np.repeat(v.reshape(b, s, groups, n), c // groups, axis=2)  # noqa: E731
    Bc, Cc = spread(B), spread(C)                          # (b, s, c, n)
    D = np.zeros(c) if D is None else D
    pre = dt + (0 if dt_bias is None else dt_bias)
    d, slope = (softplus(pre), sigmoid(pre)) if use_softplus else (pre, np.ones_like(pre))
    spans = _spans(b, s, cu_seqlens)
    h0 = np.zeros((len(spans), c, n)) if h0 is None else h0
    a = np.exp(d[..., None] * A)
    term = (d * u)[..., None] * Bc
    h, before, hT = np.zeros_like(a), np.zeros_like(a), h0.copy()
    top = np.abs(h0).max(0) if len(spans) else np.zeros((c, n))
    for i, lo, hi, j in spans:
        x, m = h0[j], np.abs(h0[j])
        for t in range(lo, hi):
            before[i, t] = x
            x, m = a[i, t] * x + term[i, t], a[i, t] * m + np.abs(term[i, t])
            h[i, t] = x
            top = np.maximum(top, m)
        hT[j] = x
    inner = (Cc * h).sum(-1) + D * u
    mag_inner = (np.abs(Cc) * top).sum(-1) + np.abs(D * u)
    gate, slope_z = (np.ones_like(u), None) if z is None else _silu(z)
    out = dict(y=inner * gate, hT=hT, mag_y=mag_inner * np.abs(gate),
               mag_hT=np.broadcast_to(top, hT.shape))
    if dy is None:
        return out
    e = dy * gate
    G = np.zeros_like(a)
    dh0 = np.zeros_like(h0) if dhT is None else dhT.copy()
    topG = np.abs(dh0).max(0) if len(spans) else np.zeros((c, n))
    for i, lo, hi, j in spans:
        x, m = dh0[j], np.abs(dh0[j])
        for t in reversed(range(lo, hi)):
            x, m = x + Cc[i, t] * e[i, t][:, None], m + np.abs(Cc[i, t] * e[i, t][:, None])
            G[i, t] = x
            topG = np.maximum(topG, m)
            x, m = a[i, t] * x, a[i, t] * m
            topG = np.maximum(topG, m)                 # (steps below zero let it grow)
        dh0[j] = x
    g = a * G * before
    gm = np.broadcast_to(topG * top, g.shape)
    share = lambda v: v.reshape(b, s, groups, c // groups, n).sum(3).reshape(B.shape)  # noqa: E731
    through, mag_through = (G * Bc).sum(-1), (topG * np.abs(Bc)).sum(-1)
    decay, mag_decay = (g * A).sum(-1), (gm * np.abs(A)).sum(-1)
    ddt = (decay + u * through) * slope
    mag_ddt = (mag_decay + np.abs(u) * mag_through) * slope
    out.update(
        du=d * through + D * e, mag_du=np.abs(d) * mag_through + np.abs(D * e),
        ddt=ddt, mag_ddt=mag_ddt, ddt_bias=ddt.sum((0, 1)), mag_ddt_bias=mag_ddt.sum((0, 1)),
        dB=share(G * (d * u)[..., None]), mag_dB=share(topG * np.abs(d * u)[..., None]),
        dC=share(h * e[..., None]), mag_dC=share(top * np.abs(e)[..., None]),
        dA=(g * d[..., None]).sum((0, 1)), mag_dA=(gm * np.abs(d)[..., None]).sum((0, 1)),
        dD=(e * u).sum((0, 1)), mag_dD=np.abs(e * u).sum((0, 1)),
        dh0=dh0, mag_dh0=np.broadcast_to(topG, dh0.shape))
    if z is not None:
        out.update(dz=dy * inner * slope_z, mag_dz=np.abs(dy) * mag_inner * 1.1)
    return out
