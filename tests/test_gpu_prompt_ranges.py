"""Prompt attention where values of very different sizes meet: queries of zero,
of the smallest and the largest magnitudes, cached values that differ by many
powers of two, infinities and NaN in single channels, extreme scales.

Tolerance: 2e-5 of the largest |V| among the tokens a row attends to (queries and
probabilities as FP16 high and low parts, 2^-22 relative; BF16 caches as FP16
with an exponent per 16 tokens, 2^-30 of the largest)."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle.kv_fp4 import pool_values, prompt_positions, rows_attention
from oracle.numerics import bf16_decode, round_bf16
from tests.test_gpu_kv_fp4 import Decode
from tests.test_gpu_prompt_attention import KINDS, Prompt

pytestmark = pytest.mark.gpu


def check_rows(c, rows=None):
    """Rows (all, or those of the mask) against the oracle, each within 2e-5 of the largest |V| it attends to."""
    got, err = c.run()
    assert err == 0
    seq, pos = prompt_positions(c.cu, c.ctx, c.n)
    k, v = pool_values(c.kp, c.kind, c.d, c.kg), pool_values(c.vp, c.kind, c.d, c.vg)
    pick = np.flatnonzero((seq >= 0) & (pos >= 0) & (True if rows is None else rows))
    ref = rows_attention(c.q[pick], k, v, c.bt, seq[pick], pos[pick]).reshape(len(pick), c.nq, c.d)
    got = got.reshape(c.n, c.nq, c.d)[pick]
    for i, at in enumerate(pick):
        seen = v[c.bt[seq[at], :pos[at] // 16 + 1]].transpose(1, 0, 2, 3).reshape(c.nkv, -1, c.d)[:, :pos[at] + 1]
        most = np.abs(seen).max((1, 2)).repeat(c.nq // c.nkv)[:, None]
        # (a V of zeros reads as up to 2^-126 of either sign: FP16's smallest normal at the lowest exponent)
        assert np.all(np.abs(got[i] - ref[i]) <= 2e-5 * most + c.vg * 2.0 ** -126), (at, np.abs(got[i] - ref[i]).max(), most.max())
    return got


# --- scales at their limits --------------------------------------------------

@pytest.mark.parametrize("kind,vg,up", [(k, vg, 0) for k in KINDS for vg in (2.0 ** -64, 2.0 ** 64)] +
                         [("bf16", 2.0 ** -64, -20), ("bf16", 2.0 ** -64, -60), ("bf16", 2.0 ** 64, -80), ("bf16", 2.0 ** 64, 50)])
def test_extreme_value_scales(cuda_lib, kind, vg, up):
    """Outputs in fp32's normal range are right for every v_scale that is taken."""
    c = Prompt(kind, 4, 2, 64, [40], [30], seed=90, vg=1.0)
    if up:
        c.vp[...] = round_bf16(bf16_decode(c.vp) * 2.0 ** up)
    c.vg = vg
    check_rows(c)


# --- queries that are not finite --------------------------------------------

@pytest.mark.parametrize("kind", list(KINDS))
def test_queries_that_are_not_finite(cuda_lib, kind):
    """A row whose query is not finite is NaN in that head; before position 0 a row is 0 whatever its query."""
    c = Prompt(kind, 4, 2, 64, [60], [0], seed=89)
    c.ctx[0] = 50                                           # the first 10 rows lie before position 0
    want = c.ref().reshape(c.n, 4, 64)
    for row in (0, 3, 20, 41):
        c.q[row, 1, 7] = np.nan
        c.q[row + 1, 2, 0] = np.inf
    got, err = c.run()
    got = got.reshape(c.n, 4, 64)
    assert err == 0 and not got[:10].any()
    bad = np.zeros((c.n, 4), bool)
    bad[[20, 41], 1] = bad[[21, 42], 2] = True
    assert np.isnan(got[bad]).all() and np.abs(got - want)[~bad].max() <= 2e-5 * c.vmax


# --- small and zero queries -------------------------------------------------

@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("kg", [0.75, 2.0 ** -30, 2.0 ** -64])
@pytest.mark.parametrize("lens,prefix", [([37], [0]), ([5, 150], [40, 3])])
def test_small_and_zero_queries(cuda_lib, kind, kg, lens, prefix):
    """Scores of 0, or as good as: those rows are the mean of their V."""
    c = Prompt(kind, 4, 2, 64, lens, prefix, seed=80, kg=kg)
    for i, scale in enumerate((0.0, 2.0 ** -20, 2.0 ** -30, 2.0 ** -60, 2.0 ** -100, 2.0 ** -126, 1.0)):
        c.q[i::7] *= np.float32(scale)
    check_rows(c)


def test_small_and_zero_queries_of_single_tokens(cuda_lib):
    for kg in (0.75, 2.0 ** -64):
        c = Decode(8, 2, 64, [37, 1, 300, 64, 16, 5, 90], seed=81, kg=kg)
        for i, scale in enumerate((0.0, 2.0 ** -20, 2.0 ** -30, 2.0 ** -60, 2.0 ** -100, 2.0 ** -126, 1.0)):
            c.q[i] *= np.float32(scale)
        c.check()


@pytest.mark.parametrize("up", [40, 80, 110])
def test_small_queries_meet_large_keys(cuda_lib, up):
    """Queries of 2^-up over BF16 keys of 2^up, and the other way round: ordinary scores."""
    for q, k in ((-up, up), (up, -up)):
        c = Prompt("bf16", 4, 2, 64, [70], [100], seed=82, kg=1.0)
        c.kp[...] = round_bf16(bf16_decode(c.kp) * 2.0 ** k)
        c.q *= np.float32(2.0 ** q)
        check_rows(c)


# --- single values that are not finite --------------------------------------

def one_bad_channel(tok, ch, bits):
    """(output with V's channel `ch` of token `tok` in KV head 1 replaced, output without, where it counts, tolerance)."""
    c = Prompt("bf16", 4, 2, 128, [90], [100], seed=86, kg=1.0, vg=1.0)
    want = c.ref().reshape(c.n, c.nq, c.d)
    c.vp[c.bt[0, tok // 16], 1, tok % 16, ch] = bits
    got, err = c.run()
    assert err == 0
    at = np.zeros(want.shape, bool)
    at[max(0, tok - 100):, 2:, ch] = True
    return got.reshape(want.shape), want, at, 2e-5 * c.vmax


@pytest.mark.parametrize("tok", [3, 99, 100, 131, 180])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_neighbours_of_a_value_that_is_not_finite(cuda_lib, tok, bits):
    """An infinity or a NaN in one channel of one token's V leaves the other channels, and the rows before it, alone."""
    for ch in (6, 7, 64, 127):
        got, want, at, tol = one_bad_channel(tok, ch, bits)
        assert np.abs(got - want)[~at].max() <= tol and not np.isfinite(got[at]).any()


@pytest.mark.parametrize("tok", [3, 99, 100, 131, 180])
@pytest.mark.parametrize("bits,what", [(0x7F80, np.inf), (0xFF80, -np.inf), (0x7FC0, np.nan)])
def test_one_channel_that_is_not_finite(cuda_lib, tok, bits, what):
    """The rows that attend to an infinity have it, wherever it lies: it is added with a weight above 0."""
    got, _, at, _ = one_bad_channel(tok, 6, bits)
    assert np.all(np.isnan(got[at])) if np.isnan(what) else np.all(got[at] == what)


@pytest.mark.parametrize("tok", [20, 120])
def test_infinities_of_both_signs_are_nan(cuda_lib, tok):
    c = Prompt("bf16", 4, 2, 64, [50], [100], seed=87)
    c.vp[c.bt[0, tok // 16], 0, tok % 16, 5] = 0x7F80
    c.vp[c.bt[0, 135 // 16], 0, 135 % 16, 5] = 0xFF80
    got = c.run()[0].reshape(c.n, 4, 64)[:, :2, 5]
    first = max(0, tok - 100)
    assert np.all(np.isfinite(got[:first])) and np.all(got[first:35] == np.inf) and np.isnan(got[35:]).all()


def test_large_finite_values_beside_a_nan(cuda_lib):
    """BF16 values above 3.0e38 are finite, also where the slow path for values that are not finite runs."""
    c = Prompt("bf16", 4, 2, 64, [60], [100], seed=88, kg=1.0, vg=1.0)
    c.ref()                                                 # sets vmax, of the ordinary values
    c.vp[c.bt[0, 130 // 16], :, 130 % 16, 3] = 0x7F7F       # 3.39e38
    c.vp[c.bt[0, 120 // 16], :, 120 % 16, 9] = 0x7FC0
    got, err = c.run()
    got = got.reshape(c.n, 4, 64)
    v = pool_values(c.vp, "bf16", 64, 1.0)
    v[c.bt[0, 120 // 16], :, 120 % 16, 9] = 0.0
    seq, pos = prompt_positions(c.cu, c.ctx, c.n)
    ref = rows_attention(c.q, pool_values(c.kp, "bf16", 64, 1.0), v, c.bt, seq, pos).reshape(c.n, 4, 64)
    assert err == 0 and np.isnan(got[20:, :, 9]).all()
    assert np.abs(got - ref)[30:, :, 3].max() <= 2e-5 * 3.39e38
    assert np.abs(got - ref)[:20].max() <= 2e-5 * c.vmax


# --- later tokens of a finite, much larger value ----------------------------

@pytest.mark.parametrize("nq,nkv,d", [(4, 2, 64), (2, 2, 128), (16, 1, 128)])
@pytest.mark.parametrize("up", [10, 14, 18, 26, 30, 60, 120])
@pytest.mark.parametrize("what", ["k", "v", "kv"])
def test_later_finite_values_never_reach_a_row(cuda_lib, nq, nkv, d, up, what):
    """2^up in one token of a BF16 cache: the rows before it are as they would be without it, whether it lies in the same
    block, in the same tile of 128 or in the next one; rows from it on see it."""
    for tok in (101, 110, 127, 128, 150, 229):
        c = Prompt("bf16", nq, nkv, d, [130], [100], seed=83, kg=1.0, vg=1.0)
        for name, pool in (("k", c.kp), ("v", c.vp)):
            if name in what:
                pool[c.bt[0, tok // 16], :, tok % 16] = round_bf16(np.float64(2.0 ** up))
        check_rows(c, np.arange(c.n) + 100 < tok if "k" in what else None)


def test_values_grow_and_shrink_along_the_context(cuda_lib):
    """V and K of every token on a scale of its own, tokens of zeros among them, from the first on."""
    rng = np.random.default_rng(84)
    for lens, prefix in (([200], [0]), ([60, 33, 1], [0, 100, 17])):
        c = Prompt("bf16", 4, 2, 64, lens, prefix, seed=85, kg=1.0, vg=1.0)
        for pool, spread in ((c.kp, 6), (c.vp, 40)):
            f = 2.0 ** rng.integers(-spread, spread if spread > 6 else 1, pool.shape[:1] + (1, 16, 1))
            f[rng.random(f.shape) < 0.2] = 0.0
            f[c.bt[:, 0], :, 0] = 0.0
            pool[...] = round_bf16(bf16_decode(pool) * f)
        check_rows(c)


# --- infinities far before the prompt ----------------------------------------

@pytest.mark.parametrize("d", [64, 128])
def test_infinities_far_before_the_prompt(cuda_lib, d):
    """In key tiles that every row sees whole, beside others in the last tiles: as such in their channels, NaN where both
    signs meet, and nothing else changes."""
    c = Prompt("bf16", 4, 2, d, [90, 30], [400, 0], seed=91, kg=1.0, vg=1.0)
    want = c.ref().reshape(c.n, 4, d)
    for tok, head, ch, bits in ((5, 0, 6, 0x7F80), (5, 0, 7, 0xFF80), (200, 1, 8, 0x7F80), (210, 1, 8, 0xFF80),
                                (300, 0, 6, 0x7F80), (383, 1, d - 1, 0x7FC0), (430, 0, 7, 0x7F80), (430, 0, 9, 0x7F80)):
        c.vp[c.bt[0, tok // 16], head, tok % 16, ch] = bits
    got, err = c.run()
    got = got.reshape(want.shape)
    assert err == 0
    assert np.all(got[:90, :2, 6] == np.inf)
    assert np.all(got[:30, :2, 7] == -np.inf) and np.isnan(got[30:90, :2, 7]).all()
    assert np.isnan(got[:90, 2:, 8]).all() and np.isnan(got[:90, 2:, d - 1]).all()
    assert np.isfinite(got[:30, :2, 9]).all() and np.all(got[30:90, :2, 9] == np.inf)
    ok = np.ones(got.shape, bool)
    ok[:90, :2, [6, 7, 9]] = ok[:90, 2:, 8] = ok[:90, 2:, d - 1] = False
    ok[:30, :2, 9] = True
    assert np.abs(got - want)[ok].max() <= 2e-5 * c.vmax


@pytest.mark.parametrize("tok", [7, 250, 399, 400, 431, 489])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_keys_that_are_not_finite(cuda_lib, tok, bits):
    """One channel of one token's K: the rows that attend to it are NaN in its KV head, the others as they were."""
    for ch in (0, 63):
        c = Prompt("bf16", 4, 2, 64, [90, 30], [400, 0], seed=92, kg=1.0, vg=1.0)
        want = c.ref().reshape(c.n, 4, 64)
        c.kp[c.bt[0, tok // 16], 1, tok % 16, ch] = bits
        got, err = c.run()
        got = got.reshape(want.shape)
        bad = np.zeros(want.shape, bool)
        bad[max(0, tok - 400):90, 2:] = True
        assert err == 0 and np.isnan(got[bad]).all() and np.abs(got - want)[~bad].max() <= 2e-5 * c.vmax


def test_a_cache_full_of_infinities(cuda_lib):
    c = Prompt("bf16", 4, 2, 64, [40], [4000], seed=93)
    c.vp[...] = 0x7F80
    got, err = c.run()
    assert err == 0 and np.all(got == np.inf)
