"""The norm's eps on the CPU: what binary32 does not hold is refused."""
import pytest

from group_dft_structured_amd import EqlinearError, NormPlan


@pytest.mark.parametrize("eps", [1e-46, 1e-60, 4e38, 1e300])
def test_eps_outside_binary32_is_refused(eps):
    # they would be zero (NaN for rows of equal values) and infinity
    with pytest.raises(EqlinearError, match="EQL_ERR_INVALID_ARG"):
        NormPlan(8, eps=eps)


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-5, 3e38])
def test_eps_inside_binary32(eps):
    assert NormPlan(8, eps=eps).handle
