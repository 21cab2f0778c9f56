"""A short run of the drawn cases of sampling and sequence extension."""
import pytest

from tests import drawn_cases

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [1, 2])
def test_drawn_cases(seed):
    cases, rows, borders = drawn_cases.compare(seed, 60)
    assert min(cases.values()) >= 10 and rows > 1000
    # (the bound of 2^-28 + V 2^-42 would leave about as many open; the weights are far closer)
    assert borders * 1000 <= rows
