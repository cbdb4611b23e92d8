"""The comparison in norm finds what is planted in an oracle's outputs: tokens left out of
a parameter's gradient, a chunk that began from a wrong state, ranks and sequences mixed up,
a decay that is off to one side."""
import numpy as np
import pytest
import torch

from _scan_norms import HALF_STEP, PARAMS, in_norm, oracle

BF, F32 = torch.bfloat16, torch.float32
LENS = [1, 700, 0, 15, 17, 1276]
S, C = 2009, 8


def inputs(m, n, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *shape, dt=dtype: torch.randn(shape, generator=gen).to(dt)
    step = torch.exp(torch.rand((C,), generator=gen) * np.log(300.0)) * 1e-3
    return dict(u=[mk(1, S, C)], dt=[mk(1, S, C).mul(0.5).clamp(-1, 1)], B=[mk(1, S, n)], C=[mk(1, S, n)],
                z=[mk(1, S, C)], dy=[mk(1, S, C)], D=mk(C, dt=F32),
                dt_bias=step + torch.log(-torch.expm1(-step)),
                A=-torch.exp(mk(C, n, dt=F32).mul(0.8).clamp(-2.5, 2.5)) * 2,
                h0=[mk(m, C, n, dt=F32)], dhT=[mk(m, C, n, dt=F32)])


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


@pytest.mark.parametrize("lens", [None, LENS], ids=["dense", "packed"])
@pytest.mark.parametrize("n", [8, 64])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_what_is_planted_is_found(lens, n, dtype):
    i = inputs(1 if lens is None else len(lens), n, dtype, 3)
    w = oracle(i, 0, lens)
    of = lambda k: F32 if k in PARAMS or k in ("hT", "dh0") else dtype
    for k, v in w.items():
        assert in_norm(rounded(v, of(k)), v, of(k)), k
    # the last 1000 tokens left out of a sum over tokens
    left = w["ddt_bias"] - w["ddt"][:, -1000:].sum((0, 1))
    assert not in_norm(left, w["ddt_bias"], F32)
    e = w["dz"] * 0 + np.where(np.arange(S)[:, None] < S - 1000, 1.0, 0.0)
    assert not in_norm(w["ddt"] * e, w["ddt"], dtype)
    for k, v in w.items():
        assert not in_norm(np.zeros_like(v), v, of(k)), k
        assert not in_norm(v * (1 + 2.0 ** -15 + HALF_STEP[of(k)]), v, of(k)), k
        # a run of 16 tokens, or one channel's parameters, are another's
        bad = v.copy()
        if k in PARAMS:
            bad[3] = v[4]
        elif k in ("hT", "dh0"):
            bad[-1] = bad[-1][::-1]
        else:
            bad[:, 800:816] = v[:, 816:832]
        assert not in_norm(bad, v, of(k)), k
    # parameters' gradients without a chunk of 128 tokens
    short = inputs(1 if lens is None else len(lens), n, dtype, 3)
    short["dy"][0][:, 1024:1152] = 0
    x = oracle(short, 0, lens)
    for k in PARAMS:
        assert not in_norm(x[k], w[k], F32), k
    # decays off to one side by 2^-22.8 of themselves
    slow = dict(i, A=i["A"] - 2.0 ** -22.8 / 0.01)
    assert not in_norm(oracle(slow, 0, lens)["dA"], w["dA"], F32)
