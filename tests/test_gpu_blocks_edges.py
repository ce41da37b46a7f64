"""Calls of the selected-block operators at the edges of what their documentation
allows: scales and queries that are not finite where nothing counts them, sizes at
the ends of the number formats, shapes that other variants of the kernels take.

Tolerances: the chosen blocks, ranges, tables and rows are equal to the oracle's;
attention's are derived at each test."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle import blocks as ob
from oracle.kv_fp4 import pool_values
from oracle.numerics import bf16_decode, round_bf16
from tests.test_gpu_blocks import ALL, KINDS, Attend, Select, dev

pytestmark = pytest.mark.gpu
DEV = "cuda"


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


# ---------------------------------------------------------------------------
# together

@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_steps_over_the_wider_caches(cuda_lib, kind):
    """The BF16 and e4m3 caches through the whole chain: steps in which sequences get none, one or many tokens, written by the
    caller at `slots`, padding rows in the null block; then steps of one token each, written by op_rope_kv_write. Every step
    against the oracle. k_scale and v_scale are powers of two, so the caller's rounding is the write's."""
    nq, nkv, d, kg, vg, k, width, nseq, theta = 8, 2, 64, 0.5, 2.0, 4, 16, 3, 10000.0
    rng = np.random.default_rng(60)
    nb = nseq * width
    free = rng.permutation(nb).astype(np.int32)
    bt_ref, held, at = np.full((nseq, width), -1, np.int32), np.zeros(nseq, int), 0
    bt = dev(np.concatenate((bt_ref, np.full((1, width), nb, np.int32))))
    kind_t = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    pools = torch.zeros((2, nb + 1, nkv, 16, d), device=DEV).to(kind_t)
    codes = torch.zeros((nb + 1, nkv, 2, d), dtype=torch.int8, device=DEV)
    scales = torch.zeros((nb + 1, nkv), device=DEV)
    ctx, free_d, free_at, err = dev(held), dev(free), dev([0]), dev([0])
    table = torch.empty((256, d // 2, 2), device=DEV)
    capi.op_rope_table(256, d, theta, table)
    for new, pad in (([40, 0, 100], 5), ([1, 70, 0], 0), ([0, 1, 2], 2), ([1, 1, 1], 0), ([0, 0, 1], 1), ([1, 1, 1], 0)):
        rows = sum(new)
        n = rows + pad
        qkv = rng.standard_normal((n, nq + 2 * nkv, d)).astype(np.float32)
        pos, seq, slots, cu = dev(np.zeros(n)), dev(np.zeros(n)), dev(np.zeros(n), torch.int64), dev(np.zeros(nseq + 1))
        capi.op_kv_extend(ctx, dev(new), bt[:nseq], nb, free_d, free_at, ctx, cu, pos, seq, slots, free_at, err=err)
        x, q = dev(qkv, torch.float32), torch.empty((n, nq, d), device=DEV)
        if new == [1, 1, 1]:
            capi.op_rope_kv_write(x.view(n, -1), nq, nkv, d, pos, bt[:nseq], 256, theta, pools[0], pools[1], nb, KINDS[kind], kg, vg, q,
                                  err=err)
        else:
            c, s = table[pos.long()].unsqueeze(1).unbind(-1)
            a, b = x[:, :nq + nkv, :d // 2], x[:, :nq + nkv, d // 2:]
            y = torch.cat((a * c - b * s, b * c + a * s), -1)
            q = y[:, :nq].contiguous()
            blk, tok = slots // 16, slots % 16
            pools[0].view(torch.uint8).view(nb + 1, nkv, 16, -1)[blk, :, tok] = (y[:, nq:] / kg).to(kind_t).view(torch.uint8)
            pools[1].view(torch.uint8).view(nb + 1, nkv, 16, -1)[blk, :, tok] = (x[:, nq + nkv:] / vg).to(kind_t).view(torch.uint8)
        sel, out = dev(np.zeros((n, nkv, k))), torch.empty((n, nq * d), device=DEV)
        capi.op_key_bounds(pos, bt, pools[0], nkv, d, KINDS[kind], nb, codes, scales, row_seq=seq, err=err)
        capi.op_block_select(q, nkv, codes, scales, pos, bt, nb, 1, 1, sel, row_seq=seq, err=err)
        capi.op_block_attention(q, nkv, pools[0], pools[1], KINDS[kind], kg, vg, pos, bt, sel, nb, out, row_seq=seq, err=err)
        torch.cuda.synchronize()
        want, bits = ob.extend(held, new, bt_ref, nb, free, at, n)
        bt_ref, held, at = want["bt"], want["held"], want["free_next"]
        assert bits == 0 and int(err) == 0 and np.array_equal(slots.cpu().numpy(), want["slots"])
        # what the cache holds: every token of this step where its table says, as the write rounds it
        raw = pools.view(torch.uint8).cpu().numpy().view(np.uint16 if kind == "bf16" else np.uint8)
        kv = pool_values(raw[0], kind, d, kg), pool_values(raw[1], kind, d, vg)
        step = 2.0 ** -8 if kind == "bf16" else 2.0 ** -4             # half a step; e4m3's smallest numbers are 2^-9 apart
        least = 0.0 if kind == "bf16" else 2.0 ** -10
        p, sq = want["positions"][:rows], want["row_seq"][:rows]
        cs = table.double().cpu().numpy()[p][:, None]
        a, b = qkv[:rows, :nq + nkv, :d // 2].astype(float), qkv[:rows, :nq + nkv, d // 2:].astype(float)
        y = np.concatenate((a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]), -1)
        got = kv[0][bt_ref[sq, p // 16], :, p % 16], kv[1][bt_ref[sq, p // 16], :, p % 16]
        # the rotation in fp32 is within 1e-6 here
        assert np.all(np.abs(got[0] - y[:, nq:]) <= np.maximum(step * np.abs(y[:, nq:]), least * kg) + 2e-6)
        v = qkv[:rows, nq + nkv:].astype(float)
        assert np.all(np.abs(got[1] - v) <= np.maximum(step * np.abs(v), least * vg))
        chosen = np.full((rows, nkv, k), -1)
        qs = q.cpu().numpy()
        for i in range(rows):
            ids = bt_ref[sq[i], :p[i] // 16 + 1]
            for h in range(nkv):
                r = [ob.key_range(kv[0][z, h, :min(16, held[sq[i]] - 16 * j)] / kg) for j, z in enumerate(ids)]
                best = ob.select(ob.scores(qs[i, 4 * h:4 * h + 4], np.array([z[0] for z in r]), np.array([z[1] for z in r])), 1, 1, k)
                chosen[i, h, :len(best)] = best
        assert np.array_equal(sel[:rows].cpu().numpy(), chosen)
        ref, most = ob.attention(qs[:rows], kv[0], kv[1], bt_ref, sq, p, chosen)
        assert np.all(np.abs(out[:rows].double().cpu().numpy() - ref) <= 2e-5 * most)
