"""Host side of the log probabilities: what the gradient reads only together with another operand."""
import pytest

from tests.test_fp4_cpu import lib, logprobs_bwd  # noqa: F401


@pytest.mark.parametrize("k", [0, 5, 65, 101, 1 << 40, -1])
def test_k_counts_with_the_listed_columns_gradient_alone(lib, k):  # noqa: F811
    assert logprobs_bwd(lib, rows=0, k=k, gt=None) == 0
    assert logprobs_bwd(lib, rows=0, k=k, gt=None, ti=None) == 0
    assert logprobs_bwd(lib, rows=0, k=k) == (0 if k in (0, 5) else 2 if k == 65 else 1)
    # what is behind the check of k: an unaligned gradient, alone among the operands
    assert logprobs_bwd(lib, k=k, gt=None, ti=2, dx=1) == 1
