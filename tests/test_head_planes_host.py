"""The tolerances of the fp32 products' tests tell six products from five, on the CPU."""
import numpy as np
import pytest

from tests import head_planes as hp


def test_three_planes_are_the_number():
    x = hp.mantissas(np.random.default_rng(1), 100_000)
    assert np.abs(sum(hp.planes(x)) / x.astype(np.float64) - 1).max() <= 2.0 ** -26


@pytest.mark.parametrize("tolerance", [hp.PRODUCT, hp.gradient_error(np.log(1000))])
@pytest.mark.parametrize("without", (None,) + hp.PAIRS)
def test_a_product_less_is_out_of_tolerance(without, tolerance):
    rng = np.random.default_rng(2)
    x, y = hp.mantissas(rng, 200), hp.mantissas(rng, 200)
    exact = x.astype(np.float64) * y.astype(np.float64)
    off = np.abs(hp.product(x, y, without) / exact - 1)
    if without is None:
        assert off.max() <= 2.0 ** -25
    else:
        assert (off > tolerance).mean() > 0.3
