"""CPU: a temperature whose reciprocal fp32 cannot hold (every exponential would
be 0 * inf) is refused."""
import pytest

import sparse_gradient_backward_amd as sgb
from sparse_gradient_backward_amd import lm


@pytest.mark.parametrize("T", [1e-45, 1e-40, 4.2e-39])
def test_reciprocal_overflows(T):
    with pytest.raises(sgb.SgbError) as e:
        lm.TopkDistill(10, 4, temperature=T)
    assert e.value.name == "SGB_ERR_INVALID_ARGUMENT"


@pytest.mark.parametrize("T", [4.3e-39, 1e-30, 1e30, 3e38])
def test_the_ends_are_taken(T):
    lm.TopkDistill(10, 4, temperature=T)
