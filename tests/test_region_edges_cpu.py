"""Host rules of the operators between g and the next g* over their whole range."""
import ctypes

import pytest
import torch

from sp_boundary_norm_gb300 import binding as sp

BF, F32 = torch.bfloat16, torch.float32
ROWS, TILES, HELD, UNITS = range(4)


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    yield


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_group_norm_splits_fit_their_kernels(dtype, backward):
    """Every width of a group (8 to 4096 channels), one to as many groups as a row holds,
    samples of 1 to 32,771 rows: blocks within their kernels' threads and shared memory,
    slabs of whole groups that cover a row, samples that fit a block's registers."""
    hold = (3 if dtype is F32 else 6) if backward else (6 if dtype is F32 else 12)
    tile = 2 if backward else 4
    for q in range(1, 513):
        most = 16384 // (8 * q)
        for groups in {1, 2, 3, min(5, most), most}:
            if groups > most:
                continue
            for n, l, t in ((1, 1, 1), (64, 1, 8), (3, 2, 1), (2, 3, 2), (1, 5, 1), (700, 5, 2),
                            (5, 17, 1), (40, 100, 1), (1, 700, 2), (8, 4096, 1), (1, 32771, 2)):
                s = sp.sp_debug_group_norm_shape(n, l, 8 * q * groups, groups, t, dtype, backward)
                what = (q, groups, n, l, t, s)
                # teams of whole warps in the rows form, one thread a vector else
                limit = {ROWS: 256 if q <= 32 else 512, TILES: 512, HELD: 256, UNITS: 512}[s["form"]]
                assert 32 <= s["threads"] <= limit and s["threads"] % 32 == 0, what
                assert s["cols"] % q == 0 and (s["slabs"] - 1) * s["cols"] < q * groups, what
                assert s["slabs"] * s["cols"] >= q * groups, what
                assert s["rows"] * s["cols"] <= s["threads"] or s["form"] == ROWS, what
                assert s["smem"] <= 48 << 10 and s["parts"] >= 1, what
                assert (s["form"] == ROWS) == (l == 1), what
                assert s["cluster"] == 1 or s["form"] == UNITS, what
                if s["form"] == TILES:
                    assert l <= s["rows"] * tile, what
                if s["form"] == HELD:
                    assert l <= s["rows"] * hold, what


def test_group_norm_split_refuses():
    for bad in (dict(c=12), dict(n=0), dict(l=-1), dict(groups=3), dict(t=17)):
        how = dict(n=2, l=3, c=64, groups=2, t=1)
        how.update(bad)
        with pytest.raises(sp.SpError):
            sp.sp_debug_group_norm_shape(**how)


def test_rope_refuses_heads_outside_tokens():
    """(b, heads, s, d) memory seen as (b, s, heads, d): the stride between tokens is one
    head's, below the extent of a token's heads."""
    lib, tab = sp.load(), sp.sp_rope_table(64)
    x, y = ((ctypes.c_void_p * 1)(at) for at in (0x7F0000000000, 0x7F1000000000))
    for x_ld, x_head, y_ld, y_head in ((64, 8 * 64, 3 * 64, 64), (3 * 64, 64, 64, 8 * 64),
                                       (2 * 80 + 63, 80, 3 * 64, 64)):
        assert lib.sp_rope_fwd(x, x_ld, x_head, 1, 8, 3, 64, 1, 0, ctypes.byref(tab), 0, None, 0,
                               None, 0, y, y_ld, y_head, None, None) == 1
        assert b"strides" in lib.sp_last_error()
