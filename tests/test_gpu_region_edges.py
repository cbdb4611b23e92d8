"""The operators between g and the next g* where digits are easily lost, against
float64: gates that shut or stay open, values that are not finite, groups without
spread, widths and counts at a rule's edge.

Units of rounding: an output of type T is its exact value rounded once (STEP), and
what float32 arithmetic does before is counted in 2^-24 per operation.  For the
recurrence, with e = exp(-gate), a = 1 / (1 + e) and k = e a:
- e is off by DELTA: the power of two by 2^-22; for 16-bit types its argument
  gate * log2(e) by 2^-24 |gate| (the product) and 2^-26 |gate| (the constant), for
  float32 that rest is multiplied in, which leaves 2^-24;
- a is off by k DELTA and by RHO = 2^-23 + 2^-24 (the reciprocal, 1 + e);
- k is off by a DELTA, RHO and a rounding.
"""
import numpy as np
import pytest
import torch

from sp_boundary_norm_gb300 import binding as sp
from test_gpu_region import BF, DEV, F32, FP, LEAST, STEP, f64, rand

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RHO = 3 * U


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    sp.check_device_status(DEV)


def delta(gate, dtype):
    """Relative error of exp(-gate)."""
    return 4 * U + (U if dtype is F32 else 1.25 * U * np.abs(gate))


def within(got, want, bound, what):
    """Elementwise: got is `want` rounded once, off before by at most `bound`."""
    dtype, got = got.dtype, f64(got)
    tol = STEP[dtype] * (np.abs(want) + bound) + LEAST[dtype] + bound
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, the worst by "
                           f"{np.nanmax(np.abs(got - want) / tol):.3g} tolerances")


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def empties(like, n):
    return [torch.full_like(like, float("nan")) for _ in range(n)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tied", [True, False])
def test_scan_gradient_of_saturated_gates(dtype, tied):
    """dgate = dy a k (h0 - v): one token a sequence, gates up to 80 either way, where
    a k is 1e-35 and still a normal number."""
    gate = torch.linspace(-80, 80, 512).view(8, 1, 64).to(dtype).to(DEV)
    value, dy = torch.zeros_like(gate), torch.ones_like(gate)
    h0 = torch.ones((8, 64), device=DEV)
    y, dgate, dvalue = empties(gate, 3)
    st = torch.empty(sp.sp_gated_scan_states_shape(8, 1, 64), device=DEV)
    sp.sp_gated_scan_fwd([gate], [value], h0=[h0], tied=tied, y=[y], states=[st])
    sp.sp_gated_scan_bwd([gate], [value], [st], [dy], h0=[h0], tied=tied, dgate=[dgate],
                         dvalue=[dvalue])
    g = f64(gate)
    want = sigmoid(g) * sigmoid(-g)
    # a and k each once, two products, the difference h0 - v is exact
    within(dgate, want, want * (delta(g, dtype) + 2 * RHO + 3 * U), "dgate")
