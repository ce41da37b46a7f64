"""Calls of the selected-block operators at the edges of what their documentation
allows: scales and queries that are not finite where nothing counts them, sizes at
the ends of the number formats, shapes that other variants of the kernels take.

Tolerances: the chosen blocks, ranges, tables and rows are equal to the oracle's;
attention's are derived at each test."""
import numpy as np
import pytest

from tests.test_gpu_blocks import Select

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# choice

@pytest.mark.parametrize("width", [None, 5000])
@pytest.mark.parametrize("d", [64, 128])
def test_select_scales_of_minus_infinity(cuda_lib, d, width):
    """A scale that is not finite makes its block's score +infinity whatever its sign and the sum it would multiply, 0 among
    them; in one launch and in two."""
    c = Select(8, 2, d, [16 * 90, 16 * 200], 20, 1, 2, seed=9, width=width)
    rng = np.random.default_rng(5)
    odd = rng.random(c.scales.shape) < 0.1
    c.scales[odd] = rng.choice([np.inf, -np.inf, np.nan], odd.sum())
    c.check()
    c.codes[odd] = 0                                                 # sums of 0
    c.check()
    c.scales[:] = -np.inf
    c.check()
    c.codes[:] = 0
    c.check()
