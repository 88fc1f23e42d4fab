"""Host-side limits of the operators around the experts' step that their arithmetic sets."""
import pytest

from test_block_abi import _add, _norm, m  # noqa: F401


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.17e-38, 2e37, 3.4e38])
def test_eps_that_no_sum_of_squares_can_stand_beside(m, eps):  # noqa: F811
    """1e-21 squared is 714 steps of the least 32-bit number, half a step of which is 7e-4 of it: beside an eps as small, the
    norm would be off by as much."""
    assert _norm(m, eps=eps) == m.EINVAL and _norm(m, eps=eps, t=0) == m.EINVAL
    assert _add(m, eps=eps) == m.EINVAL


@pytest.mark.parametrize("eps", [1.1754944e-38, 1e-30, 1.0, 1e37])
def test_eps_at_its_limits(m, eps):  # noqa: F811
    assert _norm(m, eps=eps, t=0) == 0 and _add(m, eps=eps, t=0) == 0
