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
from tests.test_gpu_blocks import ALL, KINDS, Attend, Select, check_bounds, dev, pool_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------------------
# key ranges

@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_long_prompts(cuda_lib, kind, d):
    """Windows of many rows per CTA: runs that end in the middle of one, cross its edge or fill several."""
    lens, prefix = [1, 9001, 15, 16, 17, 33, 8000, 5, 4400], [4, 7, 0, 16, 31, 1, 160, 27, 0]
    held = np.add(lens, prefix)
    at = np.cumsum([0] + [-(-h // 16) for h in held])
    nb = int(at[-1])
    ids = np.random.default_rng(61).permutation(nb)
    bt = np.full((len(held), int(max(held)) // 16 + 1), -1, np.int32)
    for s in range(len(held)):
        bt[s, :at[s + 1] - at[s]] = ids[at[s]:at[s + 1]]
    x = np.random.default_rng(62).standard_normal((nb + 1, 1, 16, d)) * 3.0
    check_bounds(x, kind, bt, nb, [(s, p) for s in range(len(held)) for p in range(prefix[s], held[s])])


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("nkv,n", [(1, 20000), (3, 5003)])
def test_bounds_of_many_blocks_in_a_window(cuda_lib, kind, nkv, n):
    """Rows in no order, each in a block of its own: every row of a window counts, more of them than warps; some rows are
    outside their table, some blocks outside the pool."""
    rng = np.random.default_rng(63)
    width = 70
    bt = rng.permutation(-(-n // width) * width).astype(np.int32).reshape(-1, width)
    nb = bt.size - 4                                                 # the last three ids are none, and the null block is one
    rows = [(int(i) // width, int(i) % width * 16 + int(t)) for i, t in zip(rng.permutation(bt.size)[:n], rng.integers(0, 16, n))]
    for i in range(0, n, 997):
        rows[i] = [(bt.shape[0], 5), (3, 16 * width), (-1, 0), (2, -1)][i // 997 % 4]
    rows += [(int(s), int(c) * 16) for s, c in zip(*np.where(bt >= nb - 1)) if (int(s), int(c)) not in {(a, b // 16) for a, b in rows}]
    x = rng.standard_normal((nb + 1, nkv, 16, 64))
    check_bounds(x, kind, bt, nb, rows, bits=capi.DEV_POS_RANGE | capi.DEV_BLOCK_RANGE)


@pytest.mark.parametrize("n", [40000, 160001])
def test_bounds_of_the_largest_windows(cuda_lib, n):
    """A CTA looks through up to 256 rows; three sequences."""
    edges = [0, n // 3 + 5, n // 3 + 6, n]
    held = np.diff(edges)
    width = -(-int(held.max()) // 16)
    bt, nb = np.arange(3 * width, dtype=np.int32).reshape(3, width)[:, ::-1].copy(), 3 * width
    x = np.random.default_rng(64).standard_normal((nb + 1, 1, 16, 64)).astype(np.float32)
    check_bounds(x, "fp8", bt, nb, [(s, p) for s in range(3) for p in range(int(held[s]))])


# ---------------------------------------------------------------------------
# choice

@pytest.mark.parametrize("spread", [0, 100])
@pytest.mark.parametrize("nq,nkv", [(16, 2), (16, 1), (2, 1)])
@pytest.mark.parametrize("held,k", [(70000, 2000), (70000, 3), (130000, 256)])
def test_select_long_of_wide_heads(cuda_lib, nq, nkv, held, k, spread):
    """Tables of two launches with 128 channels; scores within one binade, or over most of fp32's range."""
    Select(nq, nkv, 128, [held, held - 16 * 7, 40], k, 1, 2, seed=held + k, spread=spread).check()


@pytest.mark.parametrize("held,k", [(4096, 7), (4097, 4090), (5000, 1), (9000, 700), (40000, 33), (40000, 39999)])
def test_select_tables_of_two_launches_of_wide_heads(cuda_lib, held, k):
    c = Select(24, 3, 128, [16 * held - 3, 16 * (held // 3) + 1, 40, 1], k, 0, 1, seed=held + k)
    want = c.want()
    assert np.array_equal(c.run()[0], want)
    t = (dev(c.q, torch.float32), dev(c.codes, torch.int8), dev(c.scales, torch.float32), dev(c.pos), dev(c.bt))
    sel = dev(np.zeros(want.shape))
    own = torch.zeros(max(1, capi.op_block_select_scratch(4, 3, c.bt.shape[1], k)), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        capi.op_block_select(t[0], 3, *t[1:], c.nb, 0, 1, sel, scratch=own)
    for _ in range(2):
        sel.zero_()
        own.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("k", [5000, 60000])
def test_select_widest_table_of_wide_heads(cuda_lib, k):
    c = Select(16, 1, 128, [16 * 40], k, 2, 3, seed=3)
    ids = np.random.default_rng(4).integers(0, 40, 1 << 18)
    c.bt, c.pos = ids[None].astype(np.int32), np.array([(16 << 18) - 1])
    c.check()


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


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d,per_sm", [(64, 3.9), (64, 7.9), (64, 15.5), (64, 20), (128, 2.9), (128, 4.9), (128, 8.9), (128, 20)])
@pytest.mark.parametrize("G", [2, 6, 16])
def test_attention_of_every_shape_of_cta(cuda_lib, kind, d, per_sm, G):
    """So many (row, KV head, group of eight heads) per SM that CTAs have four, two and one warps, and two again in several
    waves; few heads, more than four, more than eight. Over a BF16 cache with infinities in some rows' values."""
    n = round(per_sm * torch.cuda.get_device_properties(0).multi_processor_count / 8 / (2 if G > 8 else 1) - 0.5)
    c = Attend(kind, 8 * G, 8, d, np.random.default_rng(n).integers(1, 41, n), 3, seed=n + G)
    for i in range(0, n, 13):
        c.sel[i, i % 8] = -1
    got = c.check()
    if kind == "bf16":
        for i in range(0, n, 7):
            c.vp[c.bt[i, c.pos[i] // 16], i % 8, 0, i % d] = 0x7F80
        odd = np.zeros((n, 8, G, d), bool)
        for i in range(0, n, 7):
            if (c.sel[i, i % 8] == c.pos[i] // 16).any():
                odd[i, i % 8, :, i % d] = True
        odd, again = odd.reshape(n, -1), c.run()[0]
        assert odd.any() and np.all(again[odd] == np.inf) and np.array_equal(again[~odd], got[~odd])


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 6, 16])
@pytest.mark.parametrize("n", [1, 150])
def test_attention_keeps_the_bits_of_probabilities(cuda_lib, kind, d, G, n):
    """Values +A and -A under scores of one channel within [-0.52, 0.52], over 64 tokens. In steps of 2^-22: a score is off by
    0.52 (the query's parts), so a difference of two by 1.04; the argument's own roundings take 1.5 per factor of e, of which
    there are up to 1.04; the exponential 1, the probability's parts 1: 4.6 of the probability. A mean of values within
    [-A, A] moves by twice that, 9.2 A. Products truncate at 2 per value (aligned with the largest), 128 A over a sum of
    probabilities of at least 64 / e^1.04 = 22: 5.8 A; the sum's and the merge's additions 1 A. 16 A 2^-22 together. A
    probability without its low part would be off by 2^-12 or 2^-9."""
    c = Attend(kind, 2 * G, 2, d, [64] * n, 4, seed=65, kg=1.0, vg=1.0)
    rng = np.random.default_rng(66)
    key = np.zeros((c.nb + 1, 2, 16, d))
    key[..., 5] = rng.choice([-1.0, -0.75, -0.5, 0.5, 0.75, 1.0], key.shape[:3])
    c.kp = pool_of(key, kind)
    c.vp = pool_of(rng.choice([-6.0, 6.0], key.shape), kind)
    q = np.zeros_like(c.q)
    q[..., 5] = rng.uniform(0.1, 0.5, q.shape[:2]) * np.sqrt(d)
    c.q = q
    got, err = c.run()
    want, most = c.want()
    assert err == 0 and np.all(most == 6.0)
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -22 * most), np.abs(got - want).max() / 6.0 * 2 ** 22


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 6, 16])
def test_attention_keeps_the_bits_of_queries(cuda_lib, kind, d, G):
    """Scores that are left where the queries' high bits cancel: 128 (1 + 2^-9 + 2^-17 u) and -128 (1 + 2^-9) in neighbouring
    channels under equal keys of 192. Every product of the queries' parts is a multiple of 2^-6 and below 2^15, so the sums,
    below 2^17, are exact. Differences of up to D then cost 1.5 D in the argument, 1 in the exponential and 1 in the parts,
    in steps of 2^-22: twice that of A, and for the products and sums 2 * 64 A over the sum of probabilities, which is at
    least the number of tokens with the largest score, and 1 A."""
    c = Attend(kind, 2 * G, 2, d, [64] * 20, 4, seed=67, kg=1.0, vg=1.0)
    rng = np.random.default_rng(68)
    sign = rng.choice([-1.0, 0.0, 1.0], (c.nb + 1, 2, 16))
    sign[:, :, 3], sign[:, :, 11] = 1.0, 1.0
    c.kp = pool_of(np.broadcast_to(192.0 * sign[..., None], (c.nb + 1, 2, 16, d)), kind)
    c.vp = pool_of(rng.choice([-6.0, 6.0], (c.nb + 1, 2, 16, d)), kind)
    u = rng.integers(1, 8, (*c.q.shape[:2], d // 2)) / 4.0
    q = np.empty_like(c.q)
    q[..., ::2], q[..., 1::2] = 128.0 * (1.0 + 2.0 ** -9 + 2.0 ** -17 * u), -128.0 * (1.0 + 2.0 ** -9)
    c.q = q
    got, err = c.run()
    want, most = c.want()
    D = 2 * 192 * 128 * 2.0 ** -17 * u.sum(-1) / np.sqrt(d)
    assert err == 0 and D.min() > 0.5
    # two of each block's tokens at least have the largest score: eight in all
    steps = np.repeat(2 * (1.5 * D + 2) + 2 * 64 / 8 + 1, d, axis=-1).reshape(want.shape)
    assert np.all(np.abs(got - want) <= steps * 2.0 ** -22 * most), (np.abs(got - want) / steps).max() / 6.0 * 2 ** 22


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
