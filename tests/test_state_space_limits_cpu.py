"""Counts that the state space operators' kernels could not hold are refused (fake
addresses; nothing is launched)."""
import pytest

from sp_boundary_norm_gb300 import binding as sp
from test_state_space_cpu import FAKE, STEP, _conv, _ssm

CU = FAKE + 15 * 16 * STEP


@pytest.fixture(scope="module", autouse=True)
def _built(lib):
    yield


@pytest.mark.parametrize("call", [_conv, _ssm])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n_seqs", [(1 << 30) + 1, (1 << 31) - 1])
def test_more_sequences_than_a_search_can_halve(call, back, n_seqs):
    assert call(back, b=1, cu=CU, n_seqs=n_seqs) == 3
    assert b"n_seqs" in sp.load().sp_last_error()
