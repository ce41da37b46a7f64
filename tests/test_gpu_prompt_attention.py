"""Prompt attention over the paged cache (BF16, e4m3, 4-bit) against the float64
oracle.

Tolerance: 2e-5 * max |V|, as for single-token attention (queries and
probabilities enter the tensor cores as FP16 high + low parts, 2^-22 relative;
BF16 caches as FP16 with an exponent per block, 2^-30 of its largest; fp32
scores and sums)."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle.kv_fp4 import decode, encode, pack_pool, pool_values, prompt_positions, rows_attention, unit_bytes, unpack_pool
from oracle.numerics import bf16_decode, round_bf16, round_e4m3
from tests.test_gpu_kv_fp4 import Decode, dev, random_pool, rope_table, rotate, tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"bf16": capi.DTYPE_BF16, "fp8": capi.DTYPE_E4M3, "fp4": capi.DTYPE_E2M1}


def raw_pool(kind, nb, nkv, d, seed, g):
    if kind == "fp4":
        return random_pool(nb, nkv, d, seed, g)
    x = np.random.default_rng(seed).standard_normal((nb + 1, nkv, 16, d)) / g
    return round_bf16(x) if kind == "bf16" else round_e4m3(np.clip(x, -448, 448))


def to_gpu(raw):
    return torch.as_tensor(raw.view(np.int16) if raw.dtype == np.uint16 else raw, device=DEV)


class Prompt:
    def __init__(self, kind, nq, nkv, d, lens, prefix, seed, tail=0, qscale=0.6, kg=0.75, vg=1.25, width=None):
        self.kind, self.nq, self.nkv, self.d, self.kg, self.vg = kind, nq, nkv, d, kg, vg
        self.cu = np.r_[0, np.cumsum(lens)].astype(np.int32)
        self.ctx = (np.asarray(lens) + np.asarray(prefix)).astype(np.int32)
        self.n = int(self.cu[-1]) + tail
        self.bt, self.nb = tables(np.maximum(self.ctx, 0), seed, width=width)
        self.kp, self.vp = raw_pool(kind, self.nb, nkv, d, seed + 1, kg), raw_pool(kind, self.nb, nkv, d, seed + 2, vg)
        self.q = (np.random.default_rng(seed + 3).standard_normal((self.n, nq, d)) * qscale).astype(np.float32)

    def run(self, stream=None):
        out = torch.full((self.n, self.nq * self.d), 7.5, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        capi.op_prompt_attention(dev(self.q, torch.float32), self.nkv, dev(self.cu), dev(self.ctx), to_gpu(self.kp),
                                 to_gpu(self.vp), KINDS[self.kind], self.kg, self.vg, dev(self.bt), self.nb, out, err, stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), int(err.item())

    def ref(self):
        seq, pos = prompt_positions(self.cu, self.ctx, self.n)
        k, v = pool_values(self.kp, self.kind, self.d, self.kg), pool_values(self.vp, self.kind, self.d, self.vg)
        self.vmax = np.abs(np.where(np.isfinite(v), v, 0)).max()
        out = rows_attention(self.q, k, v, np.where(self.bt < 0, self.nb, self.bt), seq, pos)
        out[seq < 0] = 7.5
        return out

    def check(self, bits=0):
        got, err = self.run()
        assert err == bits
        ref = self.ref()
        assert np.abs(got - ref).max() <= 2e-5 * self.vmax, np.abs(got - ref).max() / self.vmax
        return got


HEADS = [(32, 8, 128), (8, 1, 64), (5, 1, 128), (16, 1, 64), (2, 2, 128), (11, 1, 128)]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("nq,nkv,d", HEADS)
@pytest.mark.parametrize("lens,prefix", [([1], [0]), ([33], [0]), ([16, 1, 0, 17], [0, 40, 3, 5])])
def test_short(cuda_lib, kind, nq, nkv, d, lens, prefix):
    Prompt(kind, nq, nkv, d, lens, prefix, seed=nq + len(lens), tail=len(lens) - 1).check()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("nq,nkv,d,lens,prefix", [
    (4, 1, 128, [300], [0]),
    (4, 2, 64, [128, 129, 127], [0, 128, 1]),
    (8, 1, 128, [1, 257, 0, 64], [511, 130, 9, 0]),
    (5, 1, 64, [77, 200], [300, 0]),
    (3, 3, 128, [260], [700]),
], ids=lambda x: str(x))
def test_longer(cuda_lib, kind, nq, nkv, d, lens, prefix):
    Prompt(kind, nq, nkv, d, lens, prefix, seed=sum(lens), tail=3).check()


def test_many_sequences(cuda_lib):
    """More sequences than a warp has lanes, some empty, some of one token."""
    rng = np.random.default_rng(0)
    lens = rng.choice([0, 1, 2, 5, 18], 75)
    Prompt("fp4", 4, 2, 64, lens, rng.choice([0, 7, 50], 75), seed=2, tail=2).check()


def test_rows_before_position_zero_attend_over_nothing(cuda_lib):
    c = Prompt("bf16", 4, 2, 64, [20, 10], [0, 0], seed=3)
    c.ctx = np.array([12, 0], np.int32)                  # the first 8 rows, and all of the second sequence
    got = c.check()
    assert not got[:8].any() and not got[20:].any()


@pytest.mark.parametrize("kind", list(KINDS))
def test_peaked_scores(cuda_lib, kind):
    """Large queries, and queries far beyond the range of FP16."""
    Prompt(kind, 4, 1, 128, [150], [30], seed=4, qscale=30.0).check()
    c = Prompt(kind, 4, 2, 64, [40], [100], seed=5, qscale=1e6)
    got, err = c.run()
    assert err == 0 and np.isfinite(got).all() and np.abs(got - c.ref()).max() <= 2e-5 * c.vmax


def poke(c, pool, tok, head, value):
    """Sets every value of one token's head (sequence 0) to `value` (NaN or inf where the format has it)."""
    blk = c.bt[0, tok // 16]
    if c.kind == "fp4":
        unpack_pool(pool, c.d)[1][blk, head, tok % 16] = 0x7F
    elif c.kind == "fp8":
        pool[blk, head, tok % 16] = 0x7F
    else:
        pool[blk, head, tok % 16] = 0x7F80 if value == np.inf else 0x7FC0


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("nq", [4, 2])
def test_later_tokens_never_reach_a_row(cuda_lib, kind, nq):
    """A NaN (infinity) in the K and V of one token: rows before it keep their values to the bit's tolerance, rows from it
    on have it."""
    for tok in (0, 70, 255, 299):
        for what in ("k", "v"):
            c = Prompt(kind, nq, 2, 64, [200], [100], seed=6)
            want = c.ref().reshape(-1, nq, 64)
            poke(c, c.kp if what == "k" else c.vp, tok, 1, np.nan if what == "k" else np.inf)
            got, err = c.run()
            got = got.reshape(-1, nq, 64)
            assert err == 0
            first = max(0, tok - 100)
            assert np.abs(got[:, :nq // 2] - want[:, :nq // 2]).max() <= 2e-5 * c.vmax        # the other KV head
            if first:
                assert np.abs(got[:first, nq // 2:] - want[:first, nq // 2:]).max() <= 2e-5 * c.vmax
            assert not np.isfinite(got[first:, nq // 2:]).any()


@pytest.mark.parametrize("kind", list(KINDS))
def test_cache_past_the_context_is_ignored(cuda_lib, kind):
    c = Prompt(kind, 4, 2, 128, [19], [18], seed=7)
    want, _ = c.run()
    for tok in range(37, 48):
        for h in range(2):
            poke(c, c.kp, tok, h, np.nan)
            poke(c, c.vp, tok, h, np.inf)
    got, err = c.run()
    assert err == 0 and np.array_equal(got, want)


def test_lengths_out_of_range(cuda_lib):
    c = Prompt("fp4", 4, 2, 64, [20, 30, 10], [0, 0, 0], seed=8)
    c.ctx = np.array([-1, 33, 10], np.int32)
    got, err = c.run()
    assert err == capi.DEV_SEQLEN_RANGE and not got[:50].any()
    c.ctx[:2] = 0
    assert np.abs(got[50:] - c.ref()[50:]).max() <= 2e-5 * c.vmax


@pytest.mark.parametrize("kind", list(KINDS))
def test_bad_block_reads_the_null_block(cuda_lib, kind):
    c = Prompt(kind, 4, 2, 64, [40], [30], seed=9)
    c.bt[0, 1], c.bt[0, 3] = -7, c.nb + 1
    got, err = c.run()
    assert err == capi.DEV_BLOCK_RANGE
    c.bt[0, 3] = c.nb
    assert np.abs(got - c.ref()).max() <= 2e-5 * c.vmax


def test_malformed_boundaries_stay_in_range(cuda_lib):
    """Row boundaries beyond n or decreasing are clamped: no row outside the call is touched, the others are finite."""
    c = Prompt("bf16", 4, 2, 64, [20, 30], [0, 0], seed=10, tail=6)
    for cu in ([0, 20, 80], [0, 60, 50], [-5, 20, 50], [0, 20, 20]):
        c.cu = np.array(cu, np.int32)
        got, _ = c.run()
        assert np.isfinite(got).all()


def test_one_row_prompts_equal_single_token_attention(cuda_lib):
    d = Decode(16, 2, 128, [40, 1, 700, 33], seed=14)
    c = Prompt("fp4", 16, 2, 128, [1] * 4, d.lens - 1, seed=14)
    c.kp, c.vp, c.bt, c.nb, c.q = d.kp, d.vp, d.bt, d.nb, d.q
    got, err = c.run()
    assert err == 0 and np.abs(got - d.run()[0]).max() <= 2e-5 * 6 * 1.25


def test_streams_and_graphs(cuda_lib):
    cases = [Prompt("fp4", 8, 1, 128, [300], [100], seed=15), Prompt("bf16", 8, 2, 64, [40, 130], [0, 7], seed=16)]
    want, graphs, outs, keep = [], [], [], []
    for c in cases:
        want.append(c.run()[0])
        a = (dev(c.q, torch.float32), dev(c.cu), dev(c.ctx), to_gpu(c.kp), to_gpu(c.vp), dev(c.bt))
        out = torch.zeros((c.n, c.nq * c.d), device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            capi.op_prompt_attention(a[0], c.nkv, a[1], a[2], a[3], a[4], KINDS[c.kind], c.kg, c.vg, a[5], c.nb, out)
        graphs.append(g), outs.append(out), keep.append(a)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w)
    assert np.array_equal(cases[1].run(stream=streams[1])[0], want[1])


def test_prompt_then_decode(cuda_lib):
    """A packed prompt is written to the 4-bit cache and attended over, then each sequence decodes two tokens; every
    output against the oracle's own cache."""
    nq, nkv, d, kg, vg = 8, 2, 64, 0.875, 1.25
    rng = np.random.default_rng(40)
    lens = np.array([37, 1, 150])
    bt, nb = tables(lens + 2, 41)
    pools = dev(rng.integers(0, 256, (2, nb + 1, nkv, unit_bytes(d))), torch.uint8)
    kv = np.zeros((2, nb + 1, nkv, 16, d))
    table = rope_table(256, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = np.r_[0, np.cumsum(lens)]
    for step in range(3):
        if step == 0:
            seq, pos = prompt_positions(cu, lens, int(cu[-1]))
        else:
            seq, pos = np.arange(3), lens + step - 1
        n = len(pos)
        qkv = rng.standard_normal((n, (nq + 2 * nkv) * d)).astype(np.float32)
        q, out = torch.zeros((n, nq, d), device=DEV), torch.zeros((n, nq * d), device=DEV)
        capi.op_rope_kv_write_fp4(dev(qkv, torch.float32), nq, nkv, d, dev(pos), dev(bt), table, pools[0], pools[1], nb, kg,
                                  vg, q, row_seq=dev(seq), err=err)
        if step == 0:
            capi.op_prompt_attention(q, nkv, dev(cu), dev(lens), pools[0], pools[1], capi.DTYPE_E2M1, kg, vg, dev(bt), nb,
                                     out, err)
        else:
            capi.op_paged_attention_fp4(q, nkv, pools[0], pools[1], kg, vg, dev(bt), dev(pos + 1), nb, out, err)
        x = qkv.reshape(n, nq + 2 * nkv, d)
        y, _ = rotate(x[:, :nq + nkv], pos, table)
        for i in range(n):
            at = bt[seq[i], pos[i] // 16], slice(None), pos[i] % 16
            kv[0][at] = decode(*encode(y[i, nq:], kg), kg)
            kv[1][at] = decode(*encode(x[i, nq + nkv:].astype(np.float64), vg), vg)
        ref = rows_attention(y[:, :nq], kv[0], kv[1], bt, seq, pos)
        assert np.abs(out.double().cpu().numpy() - ref).max() <= 2e-5 * np.abs(kv[1]).max()
    assert int(err.item()) == 0


@pytest.mark.parametrize("kind", list(KINDS))
def test_blocks_beyond_four_gigabytes(cuda_lib, kind):
    """The same prompt in a small pool and behind 2^32 bytes of a large one."""
    c = Prompt(kind, 16, 2, 128, [70], [20], seed=70)
    per_block = c.kp[0].nbytes
    far = 2 ** 32 // per_block + 3
    got = []
    for first in (0, far):
        pools = []
        for raw in (c.kp, c.vp):
            p = torch.empty((first + c.nb + 1) * per_block, dtype=torch.uint8, device=DEV)
            p[first * per_block:].copy_(torch.as_tensor(raw.reshape(-1).view(np.uint8), device=DEV))
            pools.append(p)
        out, err = torch.zeros((c.n, c.nq * c.d), device=DEV), dev([0])
        capi.op_prompt_attention(dev(c.q, torch.float32), c.nkv, dev(c.cu), dev(c.ctx), *pools, KINDS[kind], c.kg, c.vg,
                                 dev(c.bt + first), first + c.nb, out, err)
        assert int(err.item()) == 0
        got.append(out.cpu())
        del pools
    assert got[0].any() and torch.equal(*got)


def test_a_graph_follows_its_inputs(cuda_lib):
    """One captured call, replayed for other boundaries, lengths, tables, queries and cache contents."""
    cases = [Prompt("fp4", 8, 2, 64, [60, 0, 5], [0, 9, 30], seed=71, width=12), Prompt("fp4", 8, 2, 64, [1, 33, 31], [150, 0, 2], seed=72, width=12)]
    nb = max(c.nb for c in cases)
    sides = []
    for c in cases:
        pools = np.zeros((2, nb + 1, 2, unit_bytes(64)), np.uint8)
        pools[0, :c.nb + 1], pools[1, :c.nb + 1] = c.kp, c.vp
        sides.append((dev(c.q, torch.float32), dev(c.cu), dev(c.ctx), dev(pools, torch.uint8), dev(c.bt)))
    q, cu, ctx, pools, bt = live = [t.clone() for t in sides[0]]
    out = torch.zeros((65, 8 * 64), device=DEV)
    call = lambda: capi.op_prompt_attention(q, 2, cu, ctx, pools[0], pools[1], capi.DTYPE_E2M1, 0.75, 1.25, bt, nb, out)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for c, side in ((cases[1], sides[1]), (cases[0], sides[0])):
        for mine, new in zip(live, side):
            mine.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        ref = c.ref()
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 2e-5 * c.vmax)


def test_hundreds_of_sequences(cuda_lib):
    """Boundaries are searched 256 sequences at a time before 32."""
    rng = np.random.default_rng(73)
    lens = rng.integers(0, 4, 901)
    lens[[255, 256, 512, 900]] = 40, 0, 70, 3
    Prompt("fp8", 8, 2, 64, lens.tolist(), rng.integers(0, 30, 901).tolist(), seed=74, tail=2).check()
