"""Host side of the operators between g and the next g*: the rotary table, and
every refusal before anything reaches a GPU (fake addresses that are never
dereferenced; no call here launches work)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import region as orc
from sp_boundary_norm_gb300 import binding as sp

FAKE = 0x7F0000000000
STEP = 1 << 32


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    yield


def _ptrs(t, at, off=0):
    return (ctypes.c_void_p * t)(*[FAKE + (at * 16 + r) * STEP + off for r in range(t)])


# ------------------------------------------------------------------ table --

@pytest.mark.parametrize("rot,kw", [
    (2, {}), (20, {}), (128, dict(base=500000.0)), (512, {}),
    (64, dict(scaling="linear", factor=4.0)), (64, dict(scaling="base", factor=8.0)),
    (128, dict(base=500000.0, scaling="parts", factor=8.0, original_len=8192, low_turns=1.0,
               high_turns=4.0, mscale=1.25))])
def test_rope_table_holds_the_frequencies(rot, kw):
    tab = sp.sp_rope_table(rot, **kw)
    want = orc.frequencies(rot, **{k: v for k, v in kw.items() if k != "mscale"})
    got = np.array([tab.turns[i] for i in range(rot // 2)], np.float64) * 2.0 ** -64 * 2 * np.pi
    assert tab.pairs == rot // 2 and tab.mscale == kw.get("mscale", 1.0)
    # pow and the divisions: a few steps of 2^-53 each; the table holds turns in
    # whole units of 2^-64, off by at most one unit of 2 pi 2^-64 radians
    assert np.allclose(got, want, rtol=1e-14, atol=2 * np.pi * 2.0 ** -64)


@pytest.mark.parametrize("rot,kw", [
    (0, {}), (3, {}), (514, {}), (-2, {}), (64, dict(base=0.5)), (64, dict(base=float("nan"))),
    (64, dict(base=float("inf"))), (64, dict(mscale=float("nan"))),
    (64, dict(scaling="linear", factor=0.5)), (64, dict(scaling="base", factor=float("inf"))),
    (2, dict(scaling="base", factor=2.0)), (4, dict(scaling="base", base=1e300, factor=1e200)),
    (64, dict(scaling="parts", factor=2.0)),
    (64, dict(scaling="parts", factor=2.0, original_len=8, low_turns=4.0, high_turns=4.0))])
def test_rope_table_refuses(rot, kw):
    with pytest.raises(sp.SpError) as e:
        sp.sp_rope_table(rot, **kw)
    assert e.value.name == "SP_ERR_INVALID_ARG"


def test_unknown_choices():
    with pytest.raises(ValueError):
        sp.sp_rope_table(64, scaling="dynamic")
    x = [torch.zeros(1, 2, 1, 8, dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="layout"):
        sp.sp_rope_fwd(x, sp.sp_rope_table(8), layout="other", y=x)


# ---------------------------------------------------------------- refusals --

def _rope(**kw):
    t, b, s, heads, d = (kw.get(k, v) for k, v in dict(t=2, b=1, s=8, heads=3, d=64).items())
    tab = kw.get("table", sp.sp_rope_table(kw.get("rot", 64)))
    head, ld = kw.get("head", d), kw.get("ld", heads * d)
    n = max(1, min(t, 16))
    fn = sp.load().sp_rope_bwd if kw.get("back") else sp.load().sp_rope_fwd
    return fn(kw.get("x", _ptrs(n, 0)), ld, head, b, s, heads, d, t, kw.get("dtype", 0),
              ctypes.byref(tab) if tab is not None else None, kw.get("layout", 0),
              kw.get("positions"), 0, kw.get("cu"), kw.get("n_seqs", 0), kw.get("y", _ptrs(n, 1)),
              kw.get("y_ld", ld), kw.get("y_head", head), kw.get("status"), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(b=-1), 1), (dict(s=-1), 1), (dict(dtype=3), 1),
    (dict(heads=0), 1), (dict(heads=4097), 1), (dict(d=62), 1), (dict(d=16392, rot=8), 1),
    (dict(layout=2), 1), (dict(table=None), 1), (dict(table=sp.RopeTable()), 1),
    (dict(head=32), 1), (dict(ld=100), 1), (dict(b=1 << 40, s=1 << 40), 1),
    (dict(ld=1 << 50), 1), (dict(head=1 << 60), 1),
    (dict(cu=FAKE, n_seqs=0), 1), (dict(cu=FAKE, n_seqs=2, b=2), 1), (dict(cu=FAKE + 2, n_seqs=2), 2),
    (dict(cu=FAKE, n_seqs=2, positions=FAKE), 1), (dict(positions=FAKE + 4), 2),
    (dict(x=None), 1), (dict(x=_ptrs(2, 0, 8)), 2), (dict(y=_ptrs(2, 1, 2)), 2),
    (dict(y=(ctypes.c_void_p * 2)(FAKE, 0)), 1), (dict(status=FAKE + 1), 2),
    # the input shifted by one row, in place with other strides, one output for two ranks
    (dict(y=_ptrs(2, 0, 384)), 7), (dict(y=_ptrs(2, 0), y_ld=256), 7),
    (dict(y=(ctypes.c_void_p * 2)(FAKE + 99 * STEP, FAKE + 99 * STEP)), 7),
    # positions inside the output
    (dict(positions=FAKE + 16 * STEP), 7)])
def test_rope_refuses(kw, code, back):
    assert _rope(back=back, **kw) == code, sp.load().sp_last_error()


def _scan(back, **kw):
    t, b, s, c = (kw.get(k, v) for k, v in dict(t=2, b=2, s=40, c=64).items())
    ld = kw.get("ld", c)
    n = max(1, min(t, 16))
    a = lambda name, at: kw[name] if name in kw else _ptrs(n, at)
    lib = sp.load()
    tail = (kw.get("status"), None)
    if not back:
        return lib.sp_gated_scan_fwd(a("gate", 0), ld, a("value", 1), ld, kw.get("h0"), b, s, c, t,
                                     kw.get("dtype", 0), 1, kw.get("cu"), kw.get("n_seqs", 0),
                                     a("y", 2), kw.get("y_ld", ld), kw.get("hT"), kw.get("states"),
                                     *tail)
    return lib.sp_gated_scan_bwd(a("gate", 0), ld, a("value", 1), ld, kw.get("h0"),
                                 a("states", 3), a("dy", 4), ld, kw.get("dhT"), b, s, c, t,
                                 kw.get("dtype", 0), 1, kw.get("cu"), kw.get("n_seqs", 0),
                                 a("y", 2), kw.get("y_ld", ld), a("dvalue", 5), ld, kw.get("dh0"),
                                 *tail)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(dtype=-1), 1), (dict(b=-1), 1), (dict(s=-3), 1),
    (dict(c=0), 1), (dict(c=12), 1), (dict(c=16392), 3), (dict(b=1 << 20), 3),
    (dict(b=1 << 30, s=1 << 30), 1), (dict(ld=56), 1), (dict(ld=68), 1), (dict(ld=1 << 46), 1),
    (dict(cu=FAKE, n_seqs=2), 1), (dict(cu=FAKE, n_seqs=0, b=1), 1),
    (dict(cu=FAKE + 1, n_seqs=1, b=1), 2), (dict(cu=FAKE, n_seqs=1, b=1, s=1 << 31), 1),
    (dict(gate=None), 1), (dict(value=_ptrs(2, 1, 4)), 2), (dict(y=None), 1),
    (dict(y=(ctypes.c_void_p * 2)(FAKE, 0)), 1), (dict(h0=_ptrs(2, 7, 8)), 2),
    (dict(y=_ptrs(2, 0)), 7), (dict(y=_ptrs(2, 1, 16)), 7), (dict(status=FAKE + 2), 2)])
def test_scan_refuses(kw, code, back):
    assert _scan(back, **kw) == code, sp.load().sp_last_error()


def test_scan_refuses_overlapping_states():
    assert _scan(False, hT=_ptrs(2, 2)) == 7                    # hT over y
    assert _scan(False, hT=_ptrs(2, 9, 16), h0=_ptrs(2, 9)) == 7   # in place, but shifted
    assert _scan(False, states=_ptrs(2, 1)) == 7
    assert _scan(True, states=None) == 1
    assert _scan(True, dvalue=_ptrs(2, 2)) == 7                 # dvalue over dgate
    assert _scan(True, dvalue=_ptrs(2, 2, 64)) == 7             # beside it, rows too narrow
    assert _scan(True, dh0=_ptrs(2, 9), h0=_ptrs(2, 9)) == 7
    assert _scan(True, dh0=_ptrs(2, 9), dhT=_ptrs(2, 9)) == 7
    # slices of one buffer whose rows overlap by eight elements
    assert _scan(True, ld=120, dvalue=_ptrs(2, 2, 112)) == 7


def _norm(back, **kw):
    t, n, l, c, groups = (kw.get(k, v) for k, v in dict(t=2, n=3, l=5, c=64, groups=4).items())
    ld = kw.get("ld", c)
    m = max(1, min(t, 16))
    a = lambda name, at: kw[name] if name in kw else _ptrs(m, at)
    one = lambda name, at: kw[name] if name in kw else FAKE + at * 16 * STEP
    lib = sp.load()
    if not back:
        return lib.sp_group_norm_fwd(a("x", 0), ld, one("gamma", 10), one("beta", 11), n, l, c,
                                     groups, t, kw.get("dtype", 0), kw.get("eps", 1e-5),
                                     kw.get("norm", 0), kw.get("act", 1), a("y", 1), ld,
                                     a("mean", 2), a("rstd", 3), None)
    return lib.sp_group_norm_bwd(a("dy", 4), ld, a("x", 0), ld, a("mean", 2), a("rstd", 3),
                                 one("gamma", 10), one("beta", 11), n, l, c, groups, t,
                                 kw.get("dtype", 0), kw.get("norm", 0), kw.get("act", 1),
                                 a("y", 1), ld, kw.get("dgamma"), kw.get("dbeta"),
                                 kw.get("ws"), kw.get("ws_bytes", 0), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(t=0), 1), (dict(t=17), 1), (dict(dtype=9), 1), (dict(n=-1), 1), (dict(l=-1), 1),
    (dict(c=60), 1), (dict(c=0), 1), (dict(c=16392, groups=1), 1), (dict(groups=0), 1),
    (dict(groups=3), 1), (dict(groups=16), 1), (dict(c=8192, groups=1), 3),
    (dict(n=1 << 40, l=1 << 40), 1), (dict(l=1 << 30), 3), (dict(ld=56), 1), (dict(ld=70), 1),
    (dict(norm=2), 1), (dict(act=2), 1), (dict(x=None), 1), (dict(rstd=None), 1),
    (dict(mean=None), 1), (dict(gamma=None), 1), (dict(beta=None), 1),
    (dict(gamma=FAKE + 8), 2), (dict(x=_ptrs(2, 0, 8)), 2), (dict(rstd=_ptrs(2, 3, 2)), 2),
    (dict(y=_ptrs(2, 0)), 7)])
def test_group_norm_refuses(kw, code, back):
    assert _norm(back, **kw) == code, sp.load().sp_last_error()


def test_group_norm_refuses_its_own_arguments():
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _norm(False, eps=eps) == 1
    assert _norm(False, rstd=_ptrs(2, 2)) == 7                  # rstd over mean
    assert _norm(True, dgamma=FAKE + 900 * STEP) == 1 and b"workspace" in sp.load().sp_last_error()
    assert _norm(True, dgamma=FAKE + 4) == 2
    assert _norm(True, dgamma=FAKE + 900 * STEP, ws=FAKE + 901 * STEP, ws_bytes=8) == 1
    assert _norm(True, dgamma=FAKE + 900 * STEP, ws=FAKE + 901 * STEP + 4, ws_bytes=1 << 30) == 2
    assert _norm(True, dgamma=FAKE + 900 * STEP, ws=FAKE + 900 * STEP, ws_bytes=1 << 30) == 7
    assert _norm(True, dgamma=FAKE + 900 * STEP, dbeta=FAKE + 900 * STEP, ws=FAKE + 901 * STEP,
                 ws_bytes=1 << 30) == 7


def test_group_norm_workspace_bytes():
    ok = sp.sp_group_norm_bwd_workspace_bytes(8, 64, 64, 4, 2)
    assert ok > 0 and ok % (2 * 2 * 64 * 4) == 0
    assert sp.sp_group_norm_bwd_workspace_bytes(0, 64, 64, 4, 2) == 0
    assert sp.sp_group_norm_bwd_workspace_bytes(8, 64, 60, 4, 2) == 0


def test_calls_without_tokens_need_no_pointers():
    lib = sp.load()
    tab = sp.sp_rope_table(64)
    assert lib.sp_rope_fwd(None, 64, 64, 0, 8, 1, 64, 1, 0, ctypes.byref(tab), 0, None, 0, None, 0,
                           None, 64, 64, None, None) == 0
    assert lib.sp_gated_scan_fwd(None, 64, None, 64, None, 3, 0, 64, 1, 0, 1, None, 0, None, 64,
                                 None, None, None, None) == 0
    assert lib.sp_group_norm_fwd(None, 64, None, None, 0, 4, 64, 2, 1, 0, 1e-5, 0, 0, None, 64,
                                 None, None, None) == 0
    assert lib.sp_group_norm_bwd(None, 64, None, 64, None, None, None, None, 4, 0, 64, 2, 1, 0, 0,
                                 0, None, 64, None, None, None, 0, None) == 0


def test_injected_failure_reaches_the_new_entry_points():
    lib = sp.load()
    for call in (_rope, lambda: _scan(False), lambda: _scan(True), lambda: _norm(False),
                 lambda: _norm(True)):
        assert lib.sp_debug_inject(5) == 0
        assert call() == 5 and b"injected" in lib.sp_last_error()


# ------------------------------------------------------- the binding's checks --

def test_binding_refuses_before_the_library():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.zeros(s)
    x = [bf(2, 4, 16), bf(2, 4, 16)]
    with pytest.raises(ValueError, match="shape"):
        sp.sp_gated_scan_fwd(x, [bf(2, 4, 16), bf(2, 4, 8)], y=x)
    with pytest.raises(ValueError, match="dtype"):
        sp.sp_gated_scan_fwd(x, [bf(2, 4, 16), f32(2, 4, 16)], y=x)
    with pytest.raises(ValueError, match="ranks"):
        sp.sp_gated_scan_fwd(x, x[:1], y=x)
    with pytest.raises(ValueError, match="dtype"):
        sp.sp_gated_scan_fwd([torch.zeros(2, 4, 16, dtype=torch.float64)], x, y=x)
    with pytest.raises(ValueError, match="contiguous"):
        sp.sp_gated_scan_fwd([q.transpose(1, 2) for q in [bf(2, 16, 4)] * 2], x, y=x)
    with pytest.raises(ValueError, match="follow"):
        sp.sp_gated_scan_fwd([bf(2, 8, 16)[:, :4]] * 2, x, y=x)
    with pytest.raises(ValueError, match="row stride"):
        sp.sp_gated_scan_fwd([bf(2, 4, 16), bf(2, 4, 24)[..., :16]], x, y=x)
    with pytest.raises(ValueError, match="h0"):
        sp.sp_gated_scan_fwd(x, x, y=x, h0=[f32(3, 16)] * 2)
    with pytest.raises(ValueError, match="b == 1"):
        sp.sp_gated_scan_fwd(x, x, y=x, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        sp.sp_gated_scan_fwd(x, x, y=x, status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        sp.sp_group_norm_fwd([bf(4, 16)], bf(16), bf(16), groups=2, eps=1e-5, y=x, rstd=x)
    with pytest.raises(ValueError, match="mean"):
        sp.sp_group_norm_fwd(x, bf(32), bf(32), groups=2, eps=1e-5, y=x, rstd=[f32(2, 2)] * 2)
    with pytest.raises(ValueError, match="gamma"):
        sp.sp_group_norm_fwd(x, bf(16), bf(32), groups=2, eps=1e-5, y=x, mean=[f32(2, 2)] * 2,
                             rstd=[f32(2, 2)] * 2)
    with pytest.raises(TypeError, match="sp_rope_table"):
        sp.sp_rope_fwd([bf(1, 4, 2, 16)], None, y=[bf(1, 4, 2, 16)])
    with pytest.raises(ValueError, match="positions"):
        sp.sp_rope_fwd([bf(1, 4, 2, 16)], sp.sp_rope_table(16), y=[bf(1, 4, 2, 16)],
                       positions=torch.zeros(1, 3, dtype=torch.int64))
    with pytest.raises(ValueError, match="batch rows"):
        sp.sp_rope_fwd([bf(2, 8, 2, 16)[:, :4]], sp.sp_rope_table(16), y=[bf(2, 4, 2, 16)])


def test_row_strides():
    x = torch.zeros(3, 5, 48)
    row = lambda y: sp._row_stride(y.shape, y.stride(), "x")
    assert row(x) == 48
    assert row(x[..., :16]) == 48
    assert row(x[:, :1, 16:32]) == 240       # one row a sample: the samples' stride
    assert row(x[:1, :1, :16]) == 16
    assert row(x[:1, ::2, :16]) == 96
    with pytest.raises(ValueError):
        row(x[:, ::2, :16])


def test_short_way_takes_only_cuda_tensors():
    """Whatever is not lists of equal CUDA tensors gives None (the binding then goes
    through it and says what is wrong), never an exception."""
    x = torch.zeros(2, 3, 8, dtype=torch.bfloat16)
    quick, table = sp._quick(), sp.sp_rope_table(4)
    at = ctypes.addressof(table)
    f = torch.zeros(2, 1)
    for xs in ([x], [], [None], [3], "a", None, [x] * 17, (x,), [x[0]], [x.int()], 7):
        assert quick.rope(False, xs, at, 0, None, 0, None, xs, None) is None
        assert quick.scan_fwd(xs, xs, None, True, None, xs, None, None, None) is None
        assert quick.scan_bwd(xs, xs, None, 1, None, xs, xs, None, xs, xs, None, None) is None
        assert quick.norm_fwd(xs, x[0, 0], x[0, 0], 1, 1e-5, 0, 0, xs, [f], [f]) is None
        assert quick.norm_bwd(xs, xs, [f], [f], x[0, 0], None, 1, 1, 0, xs, None, None, None) is None
    for name in ("rope", "scan_fwd", "scan_bwd", "norm_fwd", "norm_bwd"):
        for n in (0, 1, 9, 12, 20):
            assert getattr(quick, name)(*[None] * n) is None
    for wrong in ((), ((1, 2), None, None), ((0,) * 6, None, None), ("ab", None, None)):
        with pytest.raises((TypeError, ValueError)):
            quick.setup(*wrong)
