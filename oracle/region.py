"""Oracle of the operators between ``g`` and the next ``g*``: rotary positions,
the gated linear recurrence and group norm with an activation, one rank at a
time in float64, from their definitions.

Beside each result the functions give the magnitude that its float32 rounding
errors scale with (the same formula with every term's absolute value).
Pinned by tests/test_oracle_region.py: rotations by complex numbers worked out
by hand, the recurrence by its closed form, both gradients and group norm's by
central differences, group norm's forward by torch.
"""
import numpy as np


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0,
                low_turns=1.0, high_turns=32.0):
    """Radians per position of each rotated pair."""
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    w = np.array([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)])
    if scaling == "linear":
        w = w / factor
    if scaling == "parts":
        g = np.clip((original_len * w / (2 * np.pi) - low_turns) / (high_turns - low_turns), 0, 1)
        w = g * w + (1 - g) * w / factor
    return w


def positions(b, s, first=0, cu_seqlens=None):
    """(b, s) positions: the index in the batch row or in the packed sequence."""
    p = np.tile(np.arange(s, dtype=np.int64), (b, 1))
    if cu_seqlens is not None:
        for lo, hi in zip(cu_seqlens[:-1], cu_seqlens[1:]):
            p[0, lo:hi] -= lo
    return p + first


def rope(x, pos, freq, layout="half", mscale=1.0, back=False):
    """x: (b, s, heads, d).  Returns (y, magnitude)."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    # reduce the angle in extended precision: positions may be far
    turns = pos[..., None].astype(np.longdouble) * (freq.astype(np.longdouble) / (2 * np.pi))
    ang = 2 * np.pi * (turns - np.floor(turns)).astype(np.float64)[:, :, None]
    cos, sin = mscale * np.cos(ang), mscale * np.sin(-ang if back else ang)
    y, mag = x.copy(), np.abs(x)
    if layout == "half":
        u, v = slice(0, half), slice(half, 2 * half)
    else:
        u, v = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., v] * cos + x[..., u] * sin
    mag[..., u] = mag[..., v] = abs(mscale) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    mag[..., 2 * half:] = 0          # copied: exact
    return y, mag


def _spans(b, s, cu_seqlens):
    """(batch row, first token, behind the last, sequence) of every sequence."""
    if cu_seqlens is None:
        return [(i, 0, s, i) for i in range(b)]
    return [(0, int(lo), int(hi), j)
            for j, (lo, hi) in enumerate(zip(cu_seqlens[:-1], cu_seqlens[1:]))]


def sigmoid(x):
    """1 / (1 + exp(-x)) without overflow."""
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def gated_scan(gate, value, h0=None, tied=True, cu_seqlens=None):
    """gate, value: (b, s, c); h0: (sequences, c).  Returns dict(y, hT, mag, magT)."""
    g, v = np.asarray(gate, np.float64), np.asarray(value, np.float64)
    b, s, c = g.shape
    a, k = sigmoid(g), sigmoid(-g)
    spans = _spans(b, s, cu_seqlens)
    h0 = np.zeros((len(spans), c)) if h0 is None else np.asarray(h0, np.float64)
    y, mag = np.zeros_like(g), np.zeros_like(g)
    hT, magT = h0.copy(), np.abs(h0)
    for i, lo, hi, j in spans:
        h, m = h0[j], np.abs(h0[j])
        for q in range(lo, hi):
            w = k[i, q] * v[i, q] if tied else v[i, q]
            h, m = a[i, q] * h + w, a[i, q] * m + np.abs(w)
            y[i, q], mag[i, q] = h, m
        hT[j], magT[j] = h, m
    return dict(y=y, hT=hT, mag=mag, magT=magT)


def gated_scan_bwd(gate, value, dy, h0=None, dhT=None, tied=True, cu_seqlens=None):
    """Returns dict(dgate, dvalue, dh0) and their magnitudes (mag_...)."""
    g, v, dy = (np.asarray(x, np.float64) for x in (gate, value, dy))
    b, s, c = g.shape
    a, k = sigmoid(g), sigmoid(-g)
    spans = _spans(b, s, cu_seqlens)
    f = gated_scan(gate, value, h0, tied, cu_seqlens)
    h0 = np.zeros((len(spans), c)) if h0 is None else np.asarray(h0, np.float64)
    dhT = np.zeros((len(spans), c)) if dhT is None else np.asarray(dhT, np.float64)
    out = {n: np.zeros_like(g) for n in ("dgate", "dvalue", "mag_dgate", "mag_dvalue")}
    out["dh0"], out["mag_dh0"] = dhT.copy(), np.abs(dhT)
    for i, lo, hi, j in spans:
        q, m = dhT[j], np.abs(dhT[j])
        for p in reversed(range(lo, hi)):
            d, dm = dy[i, p] + q, np.abs(dy[i, p]) + m
            prev, pm = (f["y"][i, p - 1], f["mag"][i, p - 1]) if p > lo else (h0[j], np.abs(h0[j]))
            ak = a[i, p] * k[i, p]
            out["dgate"][i, p] = d * ak * (prev - v[i, p] if tied else prev)
            out["mag_dgate"][i, p] = dm * ak * (pm + np.abs(v[i, p]) if tied else pm)
            out["dvalue"][i, p] = d * (k[i, p] if tied else 1.0)
            out["mag_dvalue"][i, p] = dm * (k[i, p] if tied else 1.0)
            q, m = a[i, p] * d, a[i, p] * dm
        out["dh0"][j], out["mag_dh0"][j] = q, m
    return out


def group_norm(x, gamma, beta, groups, eps, norm="layernorm", act="none"):
    """x: (n, l, c).  Returns dict(y, mean, rstd, mag, z, q)."""
    x = np.asarray(x, np.float64)
    n, l, c = x.shape
    xg = x.reshape(n, l, groups, c // groups)
    ln = norm == "layernorm"
    mean = xg.mean((1, 3)) if ln else np.zeros((n, groups))
    d = xg - mean[:, None, :, None]
    rstd = 1 / np.sqrt((d * d).mean((1, 3)) + eps)
    z = (d * rstd[:, None, :, None]).reshape(n, l, c)
    gamma = np.asarray(gamma, np.float64)
    beta = np.asarray(beta, np.float64) if ln else np.zeros(c)
    q = z * gamma + beta
    spread = ((np.abs(xg) + np.abs(mean)[:, None, :, None]) * rstd[:, None, :, None])
    mag = spread.reshape(n, l, c) * np.abs(gamma) + np.abs(beta)
    return dict(y=q * sigmoid(q) if act == "silu" else q, mean=mean, rstd=rstd, mag=mag, z=z, q=q)


def group_norm_bwd(dy, x, gamma, beta, groups, eps, norm="layernorm", act="none"):
    """Returns dict(dx, dgamma, dbeta) and magnitudes mag_dx, mag_dgamma, mag_dbeta."""
    f = group_norm(x, gamma, beta, groups, eps, norm, act)
    x = np.asarray(x, np.float64)
    n, l, c = x.shape
    gamma = np.asarray(gamma, np.float64)
    shape = (n, l, groups, c // groups)
    dq = np.asarray(dy, np.float64)
    if act == "silu":
        s = sigmoid(f["q"])
        dq = dq * s * (1 + f["q"] * (1 - s))
    z = f["z"].reshape(shape)
    # the parts that rounding errors of z scale with (z holds x - mean)
    az = ((np.abs(x).reshape(shape) + np.abs(f["mean"])[:, None, :, None])
          * f["rstd"][:, None, :, None])
    adq = np.abs(np.asarray(dy, np.float64)) * 1.1 * (1 + (f["mag"] if act == "silu" else 0))
    dz, adz = (dq * gamma).reshape(shape), (adq * np.abs(gamma)).reshape(shape)
    m2, am2 = ((dz * z).mean((1, 3), keepdims=True), (adz * az).mean((1, 3), keepdims=True))
    dx, adx = dz - z * m2, adz + az * am2
    if norm == "layernorm":
        dx = dx - dz.mean((1, 3), keepdims=True)
        adx = adx + adz.mean((1, 3), keepdims=True)
    r = f["rstd"][:, None, :, None]
    return dict(dx=(dx * r).reshape(n, l, c), mag_dx=(adx * r).reshape(n, l, c),
                dgamma=(dq * f["z"]).sum((0, 1)), dbeta=dq.sum((0, 1)),
                mag_dgamma=(adq * az.reshape(n, l, c)).sum((0, 1)), mag_dbeta=adq.sum((0, 1)))
