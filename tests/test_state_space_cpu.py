"""Host side of rotary positions with several axes and of the state space layer: the
table, and every refusal before anything reaches a GPU (fake addresses that are never
dereferenced; no call here launches work)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import state_space as orc
from sp_boundary_norm_gb300 import binding as sp

FAKE = 0x7F0000000000
STEP = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    yield


def _ptrs(t, at, off=0):
    return (ctypes.c_void_p * t)(*[FAKE + (at * 16 + r) * STEP + off for r in range(t)])


# ------------------------------------------------------------ several axes --

@pytest.mark.parametrize("sections,kw", [
    ([1], {}), ([16, 24, 24], dict(base=1e6)), ([20, 20], dict(frequencies="own")),
    ([3, 1, 7], dict(order="cyclic")), ([1, 250, 5], dict(order="cyclic", frequencies="own")),
    ([8, 12, 12], dict(factors=[2.0, 1.0, 1.5], mscale=1.25)), ([1] * 8, dict(order="cyclic"))])
def test_axes_table_holds_the_frequencies(sections, kw):
    tab = sp.sp_rope_axes_table(sections, **kw)
    axis, want = orc.axes_table(sections, **{k: v for k, v in kw.items() if k != "mscale"})
    n = sum(sections)
    got = np.array([tab.turns[i] for i in range(n)], np.float64) * 2.0 ** -64 * 2 * np.pi
    assert (tab.pairs, tab.axes) == (n, len(sections)) and tab.mscale == kw.get("mscale", 1.0)
    assert [tab.axis[i] for i in range(n)] == axis.tolist()
    # pow and the division: a few steps of 2^-53 each; turns in whole units of 2^-64
    assert np.allclose(got, want, rtol=1e-14, atol=2 * np.pi * 2.0 ** -64)


@pytest.mark.parametrize("sections,kw", [
    ([], {}), ([1] * 9, {}), ([0, 4], {}), ([4, -1], {}), ([200, 57], {}),
    ([4], dict(base=0.5)), ([4], dict(base=float("inf"))), ([4], dict(base=float("nan"))),
    ([4], dict(mscale=float("inf"))), ([4, 4], dict(factors=[1.0, 0.5])),
    ([4, 4], dict(factors=[float("nan"), 1.0]))])
def test_axes_table_refuses(sections, kw):
    with pytest.raises(sp.SpError) as e:
        sp.sp_rope_axes_table(sections, **kw)
    assert e.value.name == "SP_ERR_INVALID_ARG"


def test_axes_unknown_choices():
    for kw in (dict(order="rows"), dict(frequencies="mine"), dict(factors=[1.0])):
        with pytest.raises(ValueError):
            sp.sp_rope_axes_table([4, 4], **kw)
    x = [torch.zeros(1, 2, 1, 16, dtype=torch.bfloat16)]
    tab = sp.sp_rope_axes_table([4, 4])
    pos = torch.zeros(2, 1, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="layout"):
        sp.sp_rope_axes_fwd(x, tab, layout="other", positions=pos, y=x)
    for bad in (pos[:1], pos.int(), pos.transpose(0, 1)):
        with pytest.raises(ValueError, match="positions"):
            sp.sp_rope_axes_fwd(x, tab, positions=bad, y=x)
    for bad in (None, 3):
        with pytest.raises(TypeError):
            sp.sp_rope_axes_fwd(x, tab, positions=bad, y=x)
    with pytest.raises(TypeError):
        sp.sp_rope_axes_fwd(x, sp.sp_rope_table(8), positions=pos, y=x)


def _axes(back=False, **kw):
    t, b, s, heads, d = (kw.get(k, v) for k, v in dict(t=2, b=1, s=8, heads=3, d=64).items())
    tab = kw.get("table", sp.sp_rope_axes_table([16, 8, 8]))
    head, ld = kw.get("head", d), kw.get("ld", heads * d)
    n = max(1, min(t, 16))
    fn = sp.load().sp_rope_axes_bwd if back else sp.load().sp_rope_axes_fwd
    return fn(kw.get("x", _ptrs(n, 0)), ld, head, b, s, heads, d, t, kw.get("dtype", 0),
              ctypes.byref(tab) if tab is not None else None, kw.get("layout", 0),
              kw.get("positions", FAKE + 15 * 16 * STEP), kw.get("y", _ptrs(n, 1)),
              kw.get("y_ld", ld), kw.get("y_head", head), None)


def _broken_table():
    tab = sp.sp_rope_axes_table([4, 4])
    tab.axis[3] = 2
    return tab


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(b=-1), 1), (dict(s=-1), 1), (dict(dtype=3), 1),
    (dict(heads=0), 1), (dict(heads=4097), 1), (dict(d=62), 1), (dict(layout=2), 1),
    (dict(table=None), 1), (dict(table=sp.RopeAxesTable()), 1), (dict(table="broken"), 1),
    (dict(head=32), 1), (dict(ld=100), 1), (dict(positions=None), 1), (dict(positions=FAKE + 4), 2),
    (dict(x=None), 1), (dict(x=_ptrs(2, 0, 8)), 2), (dict(y=(ctypes.c_void_p * 2)(FAKE, 0)), 1),
    (dict(y=_ptrs(2, 0, 384)), 7), (dict(y=_ptrs(2, 0), y_ld=256), 7),
    # the last axis' coordinates inside the output
    (dict(positions=FAKE + 16 * STEP - 2 * 8 * 8), 7)])
def test_axes_refuses(kw, code, back):
    if kw.get("table") == "broken":
        kw = dict(table=_broken_table())
    assert _axes(back, **kw) == code, sp.load().sp_last_error()


def test_no_token_needs_nothing():
    assert _axes(s=0, x=None, y=None, positions=None) == 0
    assert _conv(False, b=0, x=None, y=None, weight=None) == 0
    assert _ssm(False, b=0, u=None, y=None, A=None) == 0
    assert _conv(True, b=0, x=None, y=None, weight=None, dweight=None, dbias=None) == 0
    assert _ssm(True, b=0, u=None, y=None, A=None, dA=None, dD=None, ddt_bias=None) == 0


# ----------------------------------------------------- causal convolution --

ONE = FAKE + 14 * 16 * STEP           # parameters and scratch


def _conv(back, **kw):
    t, b, s, c, w = (kw.get(k, v) for k, v in dict(t=2, b=2, s=40, c=64, width=4).items())
    ld = kw.get("ld", c)
    n = max(1, min(t, 16))
    a = lambda name, at: kw[name] if name in kw else _ptrs(n, at)
    lib = sp.load()
    head = (a("x", 0), ld, kw.get("weight", ONE), kw.get("bias", ONE + STEP), kw.get("x0"))
    shape = (b, s, c, w, t, kw.get("dtype", 0), kw.get("act", 1), kw.get("cu"), kw.get("n_seqs", 0))
    if not back:
        return lib.sp_causal_conv_fwd(*head, *shape, a("y", 1), kw.get("y_ld", ld), kw.get("xT"),
                                      kw.get("status"), None)
    size = kw.get("bytes", 1 << 30)
    return lib.sp_causal_conv_bwd(*head, a("dy", 2), ld, kw.get("dxT"), *shape, a("y", 1),
                                  kw.get("y_ld", ld), kw.get("dx0"), kw.get("dweight", ONE + 2 * STEP),
                                  kw.get("dbias", ONE + 3 * STEP), kw.get("workspace", ONE + 4 * STEP),
                                  size, kw.get("status"), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(dtype=3), 1), (dict(b=-1), 1), (dict(s=-3), 1),
    (dict(c=0), 1), (dict(c=12), 1), (dict(c=16392), 3), (dict(b=1 << 20), 3),
    (dict(b=1 << 30, s=1 << 30), 1), (dict(b=1, s=1 << 47), 3), (dict(width=1), 3), (dict(width=5), 3),
    (dict(act=2), 1), (dict(ld=56), 1), (dict(ld=68), 1), (dict(ld=1 << 29), 3),
    (dict(cu=FAKE, n_seqs=2), 1), (dict(cu=FAKE, n_seqs=0, b=1), 1),
    (dict(cu=FAKE + 1, n_seqs=1, b=1), 2), (dict(x=None), 1), (dict(x=_ptrs(2, 0, 8)), 2),
    (dict(y=None), 1), (dict(y=(ctypes.c_void_p * 2)(FAKE, 0)), 1), (dict(weight=None), 1),
    (dict(weight=ONE + 8), 2), (dict(bias=ONE + 4), 2), (dict(x0=_ptrs(2, 7, 8)), 2),
    (dict(y=_ptrs(2, 0)), 7), (dict(weight=FAKE + 16 * STEP), 7), (dict(status=FAKE + 2), 2)])
def test_conv_refuses(kw, code, back):
    assert _conv(back, **kw) == code, sp.load().sp_last_error()


def test_conv_refuses_states_and_scratch():
    assert _conv(False, xT=_ptrs(2, 1)) == 7                      # xT over y
    assert _conv(False, xT=_ptrs(2, 9, 16), x0=_ptrs(2, 9)) == 7  # in place, but shifted
    assert _conv(True, dx0=_ptrs(2, 9), dxT=_ptrs(2, 9)) == 7
    assert _conv(True, dx0=_ptrs(2, 9), x0=_ptrs(2, 9)) == 7
    assert _conv(True, dy=None) == 1
    assert _conv(True, workspace=None) == 1 and b"workspace" in sp.load().sp_last_error()
    assert _conv(True, bytes=8) == 1
    assert _conv(True, workspace=ONE + 4 * STEP + 8) == 2
    assert _conv(True, workspace=ONE + 2 * STEP) == 7             # over dweight
    assert _conv(True, dweight=ONE + 4) == 2
    assert sp.sp_causal_conv_bwd_workspace_bytes(1, 64, 12, 4, 2) == 0
    assert sp.sp_causal_conv_bwd_workspace_bytes(1, 0, 64, 4, 2) == 0
    n = sp.sp_causal_conv_bwd_workspace_bytes(1, 640, 64, 4, 2)
    assert n > 0 and n % (2 * 64 * 5 * 4) == 0


# --------------------------------------------------------- selective scan --

def _ssm(back, **kw):
    t, b, s, c, n, g = (kw.get(k, v) for k, v in
                        dict(t=2, b=2, s=40, c=64, n=16, groups=2).items())
    ld, ldb = kw.get("ld", c), kw.get("ldb", g * n)
    m = max(1, min(t, 16))
    a = lambda name, at: kw[name] if name in kw else _ptrs(m, at)
    lib = sp.load()
    z = kw.get("z", _ptrs(m, 4))
    head = (a("u", 0), ld, a("dt", 1), ld, kw.get("A", ONE), a("B", 2), ldb, a("C", 3), ldb,
            kw.get("D", ONE + STEP), z, ld, kw.get("dt_bias", ONE + 2 * STEP), 1, kw.get("h0"))
    shape = (b, s, c, n, g, t, kw.get("dtype", 0), kw.get("cu"), kw.get("n_seqs", 0))
    ws = (kw.get("workspace", ONE + 9 * STEP), kw.get("bytes", 1 << 40), kw.get("status"), None)
    if not back:
        return lib.sp_selective_scan_fwd(*head, *shape, a("y", 5), kw.get("y_ld", ld), kw.get("hT"),
                                         kw.get("states"), *ws)
    return lib.sp_selective_scan_bwd(
        *head, a("states", 6), a("dy", 7), ld, kw.get("dhT"), *shape, a("y", 5), kw.get("y_ld", ld),
        a("ddt", 8), ld, a("dB", 9), ldb, a("dC", 10), ldb, a("dz", 11), ld, kw.get("dA", ONE + 3 * STEP),
        kw.get("dD", ONE + 4 * STEP), kw.get("ddt_bias", ONE + 5 * STEP), kw.get("dh0"), *ws)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(dtype=-1), 1), (dict(b=-1), 1), (dict(s=-3), 1),
    (dict(c=0), 1), (dict(c=12), 1), (dict(c=16392), 3), (dict(b=1 << 20), 3),
    (dict(b=1 << 30, s=1 << 30), 1), (dict(b=1, s=1 << 47), 3), (dict(n=4), 3), (dict(n=24), 3),
    (dict(n=128), 3), (dict(groups=0), 1), (dict(groups=3), 1), (dict(groups=16), 1),
    (dict(ld=56), 1), (dict(ld=68), 1), (dict(ldb=24), 1), (dict(ldb=36), 1), (dict(ld=1 << 29), 3),
    (dict(cu=FAKE, n_seqs=2), 1), (dict(cu=FAKE, n_seqs=0, b=1), 1),
    (dict(cu=FAKE + 1, n_seqs=1, b=1), 2), (dict(u=None), 1), (dict(dt=_ptrs(2, 1, 4)), 2),
    (dict(B=None), 1), (dict(C=(ctypes.c_void_p * 2)(FAKE, 0)), 1), (dict(z=_ptrs(2, 4, 2)), 2),
    (dict(A=None), 1), (dict(A=ONE + 4), 2), (dict(D=ONE + 8), 2), (dict(dt_bias=ONE + 2), 2),
    (dict(y=None), 1), (dict(y=_ptrs(2, 0)), 7), (dict(y=_ptrs(2, 4)), 7), (dict(y=_ptrs(2, 3)), 7),
    (dict(A=FAKE + 5 * 16 * STEP), 7), (dict(h0=_ptrs(2, 12, 8)), 2), (dict(status=FAKE + 2), 2)])
def test_ssm_refuses(kw, code, back):
    assert _ssm(back, **kw) == code, sp.load().sp_last_error()


def test_ssm_refuses_states_and_scratch():
    assert _ssm(False, hT=_ptrs(2, 5)) == 7                       # hT over y
    assert _ssm(False, hT=_ptrs(2, 12, 16), h0=_ptrs(2, 12)) == 7   # in place, but shifted
    assert _ssm(False, states=_ptrs(2, 4)) == 7
    assert _ssm(True, states=None) == 1 and _ssm(True, dy=None) == 1
    assert _ssm(True, dz=None) == 1 and _ssm(True, dB=None) == 1
    assert _ssm(True, dB=_ptrs(2, 10)) == 7                       # dB over dC
    assert _ssm(True, dh0=_ptrs(2, 12), dhT=_ptrs(2, 12)) == 7
    assert _ssm(True, dh0=_ptrs(2, 12), h0=_ptrs(2, 12)) == 7
    assert _ssm(True, workspace=None) == 1 and b"workspace" in sp.load().sp_last_error()
    assert _ssm(True, bytes=64) == 1
    assert _ssm(True, workspace=ONE + 9 * STEP + 8) == 2
    assert _ssm(True, workspace=ONE + 3 * STEP) == 7              # over dA
    for fn in (sp.sp_selective_scan_fwd_workspace_bytes, sp.sp_selective_scan_bwd_workspace_bytes):
        assert fn(1, 64, 12, 16, 1, 2) == 0 and fn(1, 0, 64, 16, 1, 2) == 0
        assert fn(1, 64, 64, 17, 1, 2) == 0 and fn(1, 64, 64, 16, 3, 2) == 0
    # a decoding step needs none
    assert sp.sp_selective_scan_fwd_workspace_bytes(64, 1, 1024, 16, 1, 8) == 0
    assert sp.sp_selective_scan_bwd_workspace_bytes(1, 640, 64, 16, 1, 2) > 0
    assert sp.sp_selective_scan_states_shape(2, 33, 64, 16) == (2, 3, 64, 16)


def test_widest_call_counts_all_buffers():
    """16 ranks with every tensor there is fit the list of checked buffers."""
    lib = sp.load()
    p = lambda at: _ptrs(16, at)
    same = dict(t=16, h0=p(12), dhT=p(13))
    # (dh0 over dhT is found, so the list held all of them)
    assert _ssm(True, dh0=p(13), cu=FAKE + 15 * 16 * STEP, n_seqs=3, b=1, **same) == 7
    assert b"dh0" in lib.sp_last_error() or b"dhT" in lib.sp_last_error()


def test_binding_says_what_is_wrong():
    f = lambda *shape: torch.zeros(*shape)
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
    x, w = [bf(1, 4, 16)], bf(16, 4)
    call = lambda **kw: sp.sp_causal_conv_fwd(kw.get("x", x), kw.get("w", w), kw.get("bias"), y=kw.get("y", x),
                                              x0=kw.get("x0"), act=kw.get("act", "none"))
    for kw, error in ((dict(w=w[:8]), ValueError), (dict(w=w.float()), ValueError), (dict(w=None), TypeError),
                      (dict(bias=bf(15)), ValueError), (dict(x0=[bf(1, 4, 16)]), ValueError),
                      (dict(x0=[f(1, 3, 16)]), ValueError), (dict(act="gelu"), ValueError),
                      (dict(y=[bf(1, 4, 8)]), ValueError), (dict(x=x + x), ValueError),
                      ({}, ValueError)):                          # (CPU tensors)
        with pytest.raises(error):
            call(**kw)
    A, B = f(16, 8), [bf(1, 4, 8)]
    scan = lambda **kw: sp.sp_selective_scan_fwd(x, kw.get("dt", x), kw.get("A", A), kw.get("B", B), kw.get("C", B),
                                                 D=kw.get("D"), y=x, hT=kw.get("hT"))
    for kw, error in ((dict(A=A[:8]), ValueError), (dict(A=A.bfloat16()), ValueError), (dict(A=None), TypeError),
                      (dict(B=[bf(1, 4, 12)]), ValueError), (dict(C=[bf(1, 4, 16)]), ValueError),
                      (dict(D=f(8)), ValueError), (dict(hT=[f(1, 16, 4)]), ValueError),
                      (dict(dt=[f(1, 4, 16)]), ValueError), ({}, ValueError)):
        with pytest.raises(error):
            scan(**kw)
    with pytest.raises(ValueError, match="dz"):
        sp.sp_selective_scan_bwd(x, x, A, B, B, [f(1, 1, 16, 8)], x, z=x, du=x, ddt=x, dB=B, dC=B)


def test_short_way_takes_only_cuda_tensors():
    """Whatever is not lists of equal CUDA tensors gives None, never an exception."""
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    quick, table = sp._quick(), sp.sp_rope_axes_table([2, 2])
    at = ctypes.addressof(table)
    f = torch.zeros(8, 8)
    for xs in ([x], [], [None], [3], "a", None, [x] * 17, (x,), [x[0]], [x.int()], 7):
        assert quick.rope_axes(False, xs, at, 0, None, 2, xs) is None
        assert quick.conv_fwd(xs, f, None, 0, None, None, xs, None, None) is None
        assert quick.conv_bwd(xs, f, None, 0, None, None, xs, None, xs, None, None, None, None, None) is None
        assert quick.ssm_fwd(xs, xs, f, xs, xs, None, None, None, True, None, None, xs, None, None, None,
                             None) is None
        assert quick.ssm_bwd(xs, xs, f, xs, xs, [f], xs, None, None, None, True, None, None, None, xs, xs, xs,
                             xs, None, None, None, None, None, None, None) is None
    for name in ("rope_axes", "conv_fwd", "conv_bwd", "ssm_fwd", "ssm_bwd"):
        for n in (0, 1, 7, 9, 14, 16, 25, 30):
            assert getattr(quick, name)(*[None] * n) is None
    for wrong in ((), ((1, 2), None, None), ((0,) * 12, None, None), ("ab", None, None)):
        with pytest.raises((TypeError, ValueError)):
            quick.setup(*wrong)
