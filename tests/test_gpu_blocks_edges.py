"""Calls of the selected-block operators at the edges of what their documentation
allows: scales and queries that are not finite where nothing counts them, sizes at
the ends of the number formats, shapes that other variants of the kernels take.

Tolerances: the chosen blocks, ranges, tables and rows are equal to the oracle's;
attention's are derived at each test."""
import numpy as np
import pytest

from memory_bound_transformer_gb300 import capi
from oracle.numerics import bf16_decode, round_bf16
from tests.test_gpu_blocks import ALL, Attend, Select

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


# ---------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("nq,d", [(8, 64), (14, 128), (8, 128), (14, 64)])
@pytest.mark.parametrize("n,k", [(6, 40), (6, 3), (400, 3)])
def test_attention_rows_without_a_token(cuda_lib, kind, nq, d, n, k):
    """They are 0 (the tolerance there is 0 too) whatever the query, in CTAs and in clusters: empty lists, rows outside the
    table, and, flagged as well, lists of blocks behind the context."""
    c = Attend(kind, nq, 2, d, [700, 20, 333], k, seed=50, rows=[(i % 3, (699, 19, 332)[i % 3]) for i in range(n)])
    bad = (np.nan, np.inf, -np.inf, np.nan, np.inf)
    for i in range(5):
        c.q[i, i % nq::2, 7] = bad[i]
    c.q[4] = np.nan
    c.sel[0] = -1
    c.sel[1], c.sel[3] = 0, 0
    c.seq[1], c.pos[1] = 3, 0                                        # a padding row
    c.sel[2] = 44
    c.pos[3] = -1
    c.sel[4, 0], c.sel[4, 1] = -7, 2 ** 31 - 1
    got = c.check(capi.DEV_POS_RANGE | capi.DEV_BLOCK_RANGE)
    assert not got[:5].any() and got[5].any()


@pytest.mark.parametrize("nq", [8, 14])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,k,scale", [(-60, 124, -64), (-124, 124, 0), (-118, 118, 0), (-41, 105, -64), (-90, 120, -30), (-140, 124, 16),
                                       (-100, 124, -64), (-140, 124, -64), (-60, 124, 0), (-100, 124, 30), (-45, 110, 0), (-140, 124, 64)])
def test_attention_tiny_queries_and_huge_keys(cuda_lib, nq, d, q, k, scale):
    """BF16 queries, keys and k_scale of 2^q, 2^k and 2^scale: the sums in between stay in range too. Scores of ordinary size
    or smaller are as exact as ordinary ones, which 2e-5 * max |V| allows for. Where they are far larger, one channel
    alone counts: keys that differ do by 2^-8 of a score beyond 2^40, so that all but the largest ones' shares are 0."""
    c = Attend("bf16", nq, 2, d, [700, 20, 333], 40, seed=51, kg=2.0 ** scale)
    c.kp = round_bf16((bf16_decode(c.kp) * 2.0 ** k).astype(np.float32))
    if q + k + scale > 0:
        keep = np.zeros_like(c.q)
        keep[..., 3] = c.q[..., 3]
        c.q = keep
    c.q[:, 1::2] = (c.q[:, 1::2].astype(np.float64) * 2.0 ** q).astype(np.float32)
    c.q[:, ::2] = (c.q[:, ::2].astype(np.float64) * 2.0 ** (q - 3)).astype(np.float32)
    c.check()
