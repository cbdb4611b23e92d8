"""What the convolution's parameter gradients keep of their digits over many tokens.

A float32 sum of n terms of about the same size is off by sqrt(n / 3) 0.36 2^-23 of itself
in the rms: its k-th addition by a rounding of a sum of k terms, 0.72 2^-23 k / sqrt(12) on
the mean.  In 128 tokens at a time, 32 times: their own errors are of no pattern and lose
sqrt(128 / 3 / 32) 0.21 2^-23 together, adding them up sqrt(32 / 3) 0.21 2^-23; the sums of
four threads half of both, and adding these two roundings: 0.9 2^-23.  Allowed are 2^-22.
One sum of 4096 terms a thread, four threads a channel, is off by sqrt(4096 / 3) / 2 0.21
2^-23 = 3.9 2^-23.
"""
import pytest
import torch

from sp_boundary_norm_gb300 import binding as sp
from test_gpu_state_space import BF, DEV, F32, NAN, nans, scratch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


@pytest.mark.parametrize("w", [2, 4])
def test_sums_over_many_tokens(w):
    """8 ranks of 9728 channels: so many that a channel has four threads in all, 4096 of
    the 16,384 tokens each."""
    t, s, c = 8, 16384, 9728
    gen = torch.Generator(device=DEV).manual_seed(61)
    draw = lambda shape: torch.rand(shape, generator=gen, device=DEV).add_(0.5).to(BF)
    x, dy = ([draw((1, s, c)) for _ in range(t)] for _ in range(2))
    weight = draw((t * c, w))
    dweight, dbias = (torch.full(n, NAN, dtype=F32, device=DEV) for n in ((t * c, w), (t * c,)))
    sp.sp_causal_conv_bwd(x, weight, None, dy, dx=nans(t, (1, s, c), BF), dweight=dweight, dbias=dbias,
                          workspace=scratch(sp.sp_causal_conv_bwd_workspace_bytes(1, s, c, w, t)))
    for r in (0, t - 1):
        p = slice(r * c, (r + 1) * c)
        g = dy[r][0].double()
        v = torch.cat((torch.zeros(w - 1, c, device=DEV), x[r][0])).double()
        want = torch.stack([(g * v[j:j + s]).sum(0) for j in range(w)], 1)
        for got, exact in ((dweight[p], want), (dbias[p], g.sum(0))):
            assert (got.double() - exact).norm() <= 2.0 ** -22 * exact.norm(), r
