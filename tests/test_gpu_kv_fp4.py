"""The 4-bit paged KV cache on the GPU: RoPE + write, read-back and single-token
attention, against the float64 oracle.

Tolerances, from the arithmetic:
* stored codes and scales: equal, byte for byte. The kernel decides every
  rounding for the exact value, and so does the oracle (whose float64 rotation is
  exact to 2^-53).
* rotated queries: two fp32 products and a sum, |err| <= 3 * 2^-24 (|q1 c| + |q2 s|).
* values read back: code * scale is exact in fp32 and is multiplied by g once:
  |err| <= 2^-24 |value|.
* attention: 2e-5 * max |V|, as for the BF16 and e4m3 caches (fp32 scores and
  sums; queries and probabilities as FP16 high + low parts, 2^-22 relative)."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle.kv_fp4 import decode, encode, pack_pool, pool_values, rows_attention, unit_bytes, unpack_pool
from oracle.numerics import E4M3_VALUES

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype, device=DEV)


def tables(held, seed, spare=2, width=None):
    """Scattered, distinct blocks for sequences of `held` tokens; unused entries -1. (table, number of blocks)."""
    need = [max(1, -(-int(h) // 16)) for h in held]
    nb = sum(need) + spare
    ids = np.random.default_rng(seed).permutation(nb)
    bt = np.full((len(need), width or max(need)), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = ids[at:at + k]
        at += k
    return bt, nb


def random_pool(nb, nkv, d, seed, g=1.0):
    x = np.random.default_rng(seed).standard_normal((nb + 1, nkv, 16, d))
    return pack_pool(*encode(x, g))


def rope_table(max_pos, d, theta=10000.0):
    t = torch.empty((max_pos, d // 2, 2), device=DEV)
    capi.op_rope_table(max_pos, d, theta, t)
    return t


def rotate(x, pos, table):
    """Exact rotation of fp32 rows by the fp32 table: x [n][heads][d] -> float64."""
    cs = table.double().cpu().numpy()[pos][:, None]
    h = x.shape[-1] // 2
    a, b = x[..., :h].astype(np.float64), x[..., h:].astype(np.float64)
    c, s = cs[..., 0], cs[..., 1]
    return np.concatenate([a * c - b * s, b * c + a * s], -1), np.concatenate(
        [np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)


class Write:
    """One op_rope_kv_write_fp4 call and the pool bytes the oracle expects after it."""

    def __init__(self, qkv, nq, nkv, d, pos, row_seq, bt, nb, kg=0.875, vg=1.25, max_pos=300, ld=None):
        n = len(pos)
        self.nq, self.nkv, self.d, self.pos, self.row_seq, self.bt, self.nb = nq, nkv, d, pos, row_seq, bt, nb
        self.kg, self.vg = kg, vg
        self.table = rope_table(max_pos, d)
        rng = np.random.default_rng(5)
        self.before = rng.integers(0, 256, (2, nb + 1, nkv, unit_bytes(d))).astype(np.uint8)
        self.pool = dev(self.before, torch.uint8)
        wide = torch.full((n, ld or qkv.shape[1]), float("nan"), device=DEV)
        wide[:, :qkv.shape[1]] = torch.tensor(qkv, device=DEV)
        self.q = torch.full((n, nq, d), float("nan"), device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        capi.op_rope_kv_write_fp4(wide, nq, nkv, d, dev(pos), dev(bt), self.table, self.pool[0], self.pool[1], nb, kg, vg,
                                  self.q, row_seq=None if row_seq is None else dev(row_seq), err=self.err)
        torch.cuda.synchronize()
        x = qkv.reshape(n, nq + 2 * nkv, d)
        ok = (np.asarray(pos) >= 0) & (np.asarray(pos) < max_pos)
        y, mag = rotate(x[:, :nq + nkv], np.where(ok, pos, 0), self.table)
        self.q_ref, self.q_mag = y[:, :nq], mag[:, :nq]
        want = self.before.copy()
        self.stored = np.zeros(n, bool)
        for w, vals, g in ((0, y[:, nq:], kg), (1, x[:, nq + nkv:].astype(np.float64), vg)):
            codes, sc = encode(vals, g)
            c2, s2 = unpack_pool(want[w], d)
            c2, s2 = c2.copy(), s2.copy()
            for i in range(n):
                s = i if row_seq is None else row_seq[i]
                if not ok[i] or not 0 <= s < len(bt) or pos[i] // 16 >= bt.shape[1]:
                    continue
                blk = bt[s, pos[i] // 16]
                if not 0 <= blk <= nb:
                    continue
                c2[blk, :, pos[i] % 16], s2[blk, :, pos[i] % 16] = codes[i], sc[i]
                self.stored[i] = True
            want[w] = pack_pool(c2, s2)
        self.want = want

    def check(self, bits=0):
        got = self.pool.cpu().numpy()
        assert int(self.err.item()) == bits
        fin = np.isfinite(self.q_ref)
        q = self.q.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            assert np.all((np.abs(q - self.q_ref) <= 3 * 2.0 ** -24 * self.q_mag)[fin])
        # a NaN group's codes and the sign of a zero code are free: compare those as values
        gc, gs = unpack_pool(got.reshape(-1, self.nkv, got.shape[-1]), self.d)
        wc, ws = unpack_pool(self.want.reshape(-1, self.nkv, got.shape[-1]), self.d)
        assert np.array_equal(gs, ws)
        nan = np.repeat((ws & 0x7F) == 0x7F, 16, -1)
        same = (gc == wc) | nan | (((gc | wc) & 7) == 0)
        assert same.all(), f"{(~same).sum()} codes differ"


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (4, 2, 64), (40, 8, 64), (1, 1, 128), (3, 3, 64)])
@pytest.mark.parametrize("n", [1, 3, 64, 257])
def test_write_codes_exact(cuda_lib, nq, nkv, d, n):
    """Rows of several sequences in scattered order, strided qkv rows; every stored byte, and no other, as the oracle has it."""
    rng = np.random.default_rng(n * d + nq)
    qkv = rng.standard_normal((n, (nq + 2 * nkv) * d)).astype(np.float32)
    nseq = min(n, 5)
    held = rng.integers(n // nseq + 1, 300, nseq)
    bt, nb = tables(held, n)
    row_seq = np.arange(n) % nseq
    pos = np.empty(n, int)
    for s in range(nseq):
        pos[row_seq == s] = rng.permutation(held[s])[:(row_seq == s).sum()]
    Write(qkv, nq, nkv, d, pos, row_seq, bt, nb, ld=qkv.shape[1] + 12).check()


def test_write_many_borders(cuda_lib):
    """Three million values drawn so that many lie within fp32 rounding of a border of either grid."""
    rng = np.random.default_rng(3)
    n, nq, nkv, d = 700, 1, 16, 128
    x = rng.standard_normal((n, nq + 2 * nkv, d)).astype(np.float32)
    # group maxima on the midpoints of the e4m3 grid times 6 g, other values on the midpoints of the e2m1 grid
    v = x[:, nq + nkv:].reshape(n, nkv, -1, 16)
    code = rng.integers(40, 90, v.shape[:-1])
    top = (E4M3_VALUES[code] + E4M3_VALUES[code + 1]) / 2 * 6 * 1.25
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v[...] = (mids[rng.integers(0, 7, v.shape)] * (E4M3_VALUES[code + (code & 1)] * 1.25)[..., None]).astype(np.float32)
    v *= rng.choice([-1.0, 1.0], v.shape).astype(np.float32)
    v[..., 5] = top
    nudge = rng.integers(-1, 2, v.shape)
    v[...] = np.where(nudge < 0, np.nextafter(v, np.float32(-np.inf)), np.where(nudge > 0, np.nextafter(v, np.float32(np.inf)), v))
    pos = rng.permutation(4096)[:n]
    bt, nb = tables([4096], 1)
    Write(x.reshape(n, -1), nq, nkv, d, pos, np.zeros(n, int), bt, nb, max_pos=4096).check()


def test_write_cancelling_rotations(cuda_lib):
    """Keys that the rotation cancels to almost nothing: the fp32 error is as large as the values."""
    rng = np.random.default_rng(4)
    n, nq, nkv, d = 200, 1, 2, 64
    x = rng.standard_normal((n, nq + 2 * nkv, d)).astype(np.float32)
    pos = rng.permutation(300)[:n]
    cs = rope_table(300, d).cpu().numpy()[pos][:, None]
    x[:, nq:nq + nkv, :d // 2] = x[:, nq:nq + nkv, d // 2:] * (cs[..., 1] / np.where(cs[..., 0] == 0, 1, cs[..., 0]))
    bt, nb = tables([300], 1)
    Write(x.reshape(n, -1), nq, nkv, d, pos, np.zeros(n, int), bt, nb).check()


def test_write_edges(cuda_lib):
    """Zeros, tiny and huge rows, a NaN, infinities."""
    n, nq, nkv, d = 6, 1, 1, 64
    x = np.random.default_rng(1).standard_normal((n, 3, d)).astype(np.float32)
    x[0] = 0
    x[1] *= np.float32(2.0 ** -12)
    x[2] *= np.float32(1e5)
    x[3, 2, 17] = np.nan
    x[4, 2, 33] = np.inf
    x[5, 2, :16] = -np.inf
    bt, nb = tables([16], 1)
    # at position 0 the rotation is the identity: K rows carry the same edges
    x[:, 1] = x[:, 2]
    for i in range(n):
        with np.errstate(invalid="ignore"):
            w = Write(x[i:i + 1].reshape(1, -1), nq, nkv, d, np.array([0]), None, bt, nb)
        got = unpack_pool(w.pool.cpu().numpy()[1], d)
        want = unpack_pool(w.want[1], d)
        blk = bt[0, 0]
        assert np.array_equal(got[1][blk, 0, 0], want[1][blk, 0, 0])
        a, b = decode(got[0][blk, 0, 0], got[1][blk, 0, 0], 1.25), decode(want[0][blk, 0, 0], want[1][blk, 0, 0], 1.25)
        assert np.array_equal(np.nan_to_num(a, nan=9e9), np.nan_to_num(b, nan=9e9))
        if i < 3:
            w.check()


def test_write_out_of_range_rows_are_skipped(cuda_lib):
    n, nq, nkv, d = 7, 2, 1, 128
    x = np.random.default_rng(2).standard_normal((n, (nq + 2 * nkv) * d)).astype(np.float32)
    bt, nb = tables([40, 40], 3)
    bt[1, 1], bt[1, 2] = nb + 1, nb                        # an invalid id, and the null block
    pos = np.array([-1, 300, 0, 17, 48, 33, 5])
    seq = np.array([0, 0, 2, 1, 0, 1, -1])
    w = Write(x, nq, nkv, d, pos, seq, bt, nb)
    assert w.stored.tolist() == [False] * 5 + [True, False]
    w.check(bits=capi.DEV_POS_RANGE | capi.DEV_BLOCK_RANGE)


@pytest.mark.parametrize("nkv,d,n", [(8, 128, 100), (1, 64, 1), (3, 64, 33)])
def test_read_back(cuda_lib, nkv, d, n):
    rng = np.random.default_rng(n)
    held = [200, 64]
    bt, nb = tables(held, 7, width=14)
    pool = np.stack([random_pool(nb, nkv, d, 1, 0.75), random_pool(nb, nkv, d, 2, 1.5)])
    seq = rng.integers(0, 2, n)
    pos = np.array([rng.integers(0, held[s]) for s in seq])
    bad = n > 40
    if bad:
        pos[3], seq[5], pos[9], seq[11], pos[11] = -1, 2, 14 * 16, 1, 200       # outside; an unused entry
    k = torch.full((n, nkv, d), float("nan"), device=DEV)
    v = torch.full_like(k, float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = dev(pool, torch.uint8)
    capi.op_kv_read_fp4(dev(pos), dev(bt), p[0], p[1], nkv, d, nb, 0.75, 1.5, k, v, row_seq=dev(seq), err=err)
    assert int(err.item()) == ((capi.DEV_POS_RANGE | capi.DEV_BLOCK_RANGE) if bad else 0)
    for w, got, g in ((0, k, 0.75), (1, v, 1.5)):
        vals = pool_values(pool[w], "fp4", d, g)
        for i in range(n):
            ok = 0 <= seq[i] < 2 and 0 <= pos[i] < 14 * 16 and bt[seq[i], pos[i] // 16] >= 0
            want = vals[bt[seq[i], pos[i] // 16], :, pos[i] % 16] if ok else np.zeros((nkv, d))
            assert np.all(np.abs(got[i].double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want))


# ---------------------------------------------------------------------------
# single-token attention

class Decode:
    def __init__(self, nq, nkv, d, lens, seed, kg=0.75, vg=1.25, width=None, qscale=0.6):
        self.nq, self.nkv, self.d, self.lens, self.kg, self.vg = nq, nkv, d, np.asarray(lens), kg, vg
        self.bt, self.nb = tables(lens, seed, width=width)
        self.kp, self.vp = random_pool(self.nb, nkv, d, seed + 1, kg), random_pool(self.nb, nkv, d, seed + 2, vg)
        self.q = (np.random.default_rng(seed + 3).standard_normal((len(lens), nq, d)) * qscale).astype(np.float32)

    def run(self, stream=None):
        out = torch.full((len(self.lens), self.nq * self.d), float("nan"), device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        capi.op_paged_attention_fp4(dev(self.q, torch.float32), self.nkv, dev(self.kp, torch.uint8), dev(self.vp, torch.uint8),
                                    self.kg, self.vg, dev(self.bt), dev(self.lens), self.nb, out, err, stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), int(err.item())

    def ref(self):
        limit = self.bt.shape[1] * 16
        last = np.where((self.lens >= 1) & (self.lens <= limit), self.lens - 1, -1)
        bt = np.where(self.bt < 0, self.nb, self.bt)
        k, v = pool_values(self.kp, "fp4", self.d, self.kg), pool_values(self.vp, "fp4", self.d, self.vg)
        self.vmax = np.nanmax(np.abs(np.where(np.isfinite(v), v, 0)))
        return rows_attention(self.q, k, v, bt, np.arange(len(last)), last)

    def check(self, bits=0):
        got, err = self.run()
        assert err == bits
        ref = self.ref()
        assert np.all(np.abs(got - ref) <= 2e-5 * self.vmax), np.abs(got - ref).max() / self.vmax


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (8, 1, 128), (5, 1, 64), (16, 1, 128), (11, 1, 64), (2, 2, 64), (40, 8, 128)])
@pytest.mark.parametrize("lens", [[1], [16, 17, 33], [15, 64, 65, 1, 130], [1000, 3, 511], [2049]])
def test_attention(cuda_lib, nq, nkv, d, lens):
    Decode(nq, nkv, d, lens, seed=len(lens) + nq).check()


@pytest.mark.parametrize("B,lo,hi", [(64, 1, 300), (200, 1, 40)])
def test_attention_batches(cuda_lib, B, lo, hi):
    Decode(8, 2, 64, np.random.default_rng(B).integers(lo, hi + 1, B), seed=B).check()


def test_attention_long_context_in_wide_table(cuda_lib):
    """A context that needs many splits, and short ones under a table that could hold far more."""
    Decode(8, 1, 128, [9001], seed=1).check()
    Decode(8, 2, 64, [40, 1, 700], seed=2, width=4096).check()


def test_attention_peaked_scores(cuda_lib):
    """Large queries: the running maximum moves, most probabilities vanish."""
    Decode(8, 2, 128, [300, 77], seed=5, qscale=30.0).check()
    # far beyond the FP16 range: still finite, one token takes all
    c = Decode(4, 1, 64, [50], seed=6, qscale=1e6)
    got, err = c.run()
    assert err == 0 and np.all(np.abs(got - c.ref()) <= 2e-5 * c.vmax)


def test_attention_lengths_out_of_range(cuda_lib):
    c = Decode(8, 2, 64, [20, 30, 16], seed=8)
    c.lens = np.array([0, 33, -5])
    c.check(bits=capi.DEV_SEQLEN_RANGE)
    assert not c.run()[0].any()


def test_attention_bad_block_reads_the_null_block(cuda_lib):
    c = Decode(8, 2, 64, [40, 33], seed=9)
    c.bt[0, 1], c.bt[1, 2] = -7, c.nb + 3
    got, err = c.run()
    assert err == capi.DEV_BLOCK_RANGE
    c.bt[1, 2] = c.nb
    assert np.all(np.abs(got - c.ref()) <= 2e-5 * c.vmax)


def test_attention_ignores_what_lies_past_the_context(cuda_lib):
    """NaN scales and every other byte past seq_len, in the last block and in others, leave the output as it is."""
    c = Decode(8, 2, 128, [37, 5, 64], seed=10)
    want, _ = c.run()
    for b, l in enumerate(c.lens):
        for pool in (c.kp, c.vp):
            codes, sc = unpack_pool(pool, c.d)
            blk = c.bt[b, (l - 1) // 16]
            if l % 16:
                sc[blk, :, l % 16:] = 0x7F
    used = set(c.bt[c.bt >= 0].tolist())
    for blk in set(range(c.nb + 1)) - used:
        unpack_pool(c.kp, c.d)[1][blk] = 0x7F
        unpack_pool(c.vp, c.d)[1][blk] = 0xFF
    got, err = c.run()
    assert err == 0 and np.array_equal(got, want)


def test_attention_nan_inside_the_context_stays_in_its_head(cuda_lib):
    c = Decode(8, 2, 64, [37, 20], seed=11)
    unpack_pool(c.vp, c.d)[1][c.bt[0, 1], 1, 2, 0] = 0x7F      # row 0, KV head 1, channels 0..15
    got, err = c.run()
    bad = np.isnan(got.reshape(2, 8, 64))
    assert err == 0 and bad[0, 4:, :16].all() and bad.sum() == 4 * 16


def test_attention_on_another_stream_and_in_a_graph(cuda_lib):
    """Two captured graphs of different shapes replayed at the same time on two streams equal the eager results."""
    cases = [Decode(8, 1, 128, [5000, 40], seed=12), Decode(16, 2, 64, [300] * 9, seed=13)]
    want, graphs, outs, keep = [], [], [], []
    for c in cases:
        want.append(c.run()[0])
        args = (dev(c.q, torch.float32), dev(c.kp, torch.uint8), dev(c.vp, torch.uint8), dev(c.bt), dev(c.lens))
        out = torch.zeros((len(c.lens), c.nq * c.d), device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            capi.op_paged_attention_fp4(args[0], c.nkv, args[1], args[2], c.kg, c.vg, args[3], args[4], c.nb, out)
        graphs.append(g), outs.append(out), keep.append(args)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w)
    got = cases[0].run(stream=streams[0])[0]
    assert np.array_equal(got, want[0])


def test_write_then_attend_as_a_serving_loop(cuda_lib):
    """Several steps of: rotate and append each sequence's row, attend over it; against the oracle's own cache."""
    nq, nkv, d, kg, vg = 8, 2, 128, 0.875, 1.25
    rng = np.random.default_rng(20)
    lens = np.array([15, 0, 31])
    bt, nb = tables(lens + 8, 21)
    pools = dev(np.zeros((2, nb + 1, nkv, unit_bytes(d))), torch.uint8)
    kv = np.zeros((2, nb + 1, nkv, 16, d))
    for w, g in ((0, kg), (1, vg)):
        raw = random_pool(nb, nkv, d, 30 + w, g)
        pools[w].copy_(dev(raw, torch.uint8))
        kv[w] = pool_values(raw, "fp4", d, g)
    table = rope_table(64, d)
    q = torch.zeros((3, nq, d), device=DEV)
    out = torch.zeros((3, nq * d), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for step in range(6):
        qkv = rng.standard_normal((3, (nq + 2 * nkv) * d)).astype(np.float32)
        pos = lens + step
        capi.op_rope_kv_write_fp4(dev(qkv, torch.float32), nq, nkv, d, dev(pos), dev(bt), table, pools[0], pools[1], nb, kg,
                                  vg, q, err=err)
        capi.op_paged_attention_fp4(q, nkv, pools[0], pools[1], kg, vg, dev(bt), dev(pos + 1), nb, out, err)
        x = qkv.reshape(3, nq + 2 * nkv, d)
        y, _ = rotate(x[:, :nq + nkv], pos, table)
        for i in range(3):
            at = bt[i, pos[i] // 16], slice(None), pos[i] % 16
            kv[0][at] = decode(*encode(y[i, nq:], kg), kg)
            kv[1][at] = decode(*encode(x[i, nq + nkv:].astype(np.float64), vg), vg)
        ref = rows_attention(y[:, :nq], kv[0], kv[1], bt, np.arange(3), pos)
        assert np.abs(out.double().cpu().numpy() - ref).max() <= 2e-5 * np.abs(kv[1]).max()
    assert int(err.item()) == 0


def test_blocks_beyond_four_gigabytes(cuda_lib):
    """The same rows in a small pool and behind 2^32 bytes of a large one: same bytes, values and outputs."""
    nq, nkv, d, n = 16, 8, 128, 40
    per_block = nkv * unit_bytes(d)
    far = 2 ** 32 // per_block + 3                                    # the large pool's first block past 2^32 bytes
    rng = np.random.default_rng(50)
    qkv, table = dev(rng.standard_normal((n, (nq + 2 * nkv) * d)), torch.float32), rope_table(64, d)
    bt, seq, lens = np.array([[2, 0, 1]], np.int32), dev(np.zeros(n)), dev([n])
    got = []
    for first in (0, far):
        nb = first + 3
        pools = [torch.empty((nb + 1) * per_block, dtype=torch.uint8, device=DEV) for _ in range(2)]
        for p in pools:
            p[first * per_block:].zero_()
        q, out = torch.zeros((n, nq, d), device=DEV), torch.zeros((1, nq * d), device=DEV)
        k, v, err = torch.zeros((n, nkv, d), device=DEV), torch.zeros((n, nkv, d), device=DEV), dev([0])
        at = dev(bt + first)
        capi.op_rope_kv_write_fp4(qkv, nq, nkv, d, dev(np.arange(n)), at, table, *pools, nb, 0.875, 1.25, q, row_seq=seq, err=err)
        capi.op_kv_read_fp4(dev(np.arange(n)), at, *pools, nkv, d, nb, 0.875, 1.25, k, v, row_seq=seq, err=err)
        capi.op_paged_attention_fp4(q[-1:], nkv, *pools, 0.875, 1.25, at, lens, nb, out, err)
        assert int(err.item()) == 0
        got.append([x.cpu() for x in (q, k, v, out, pools[0][first * per_block:], pools[1][first * per_block:])])
        del pools
    assert got[0][1].any() and got[0][3].any()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_graph_follows_its_inputs(cuda_lib):
    """A captured call reads lengths, tables, queries and pools when it is replayed."""
    first, then = Decode(16, 2, 128, [300, 40, 1], seed=60), Decode(16, 2, 128, [33, 300, 65], seed=61)
    width, nb = max(first.bt.shape[1], then.bt.shape[1]), max(first.nb, then.nb)
    sides = []
    for c in (first, then):
        bt = np.full((3, width), -1, np.int32)
        bt[:, :c.bt.shape[1]] = c.bt
        pools = np.zeros((2, nb + 1, 2, unit_bytes(128)), np.uint8)
        pools[0, :c.nb + 1], pools[1, :c.nb + 1] = c.kp, c.vp
        sides.append((dev(c.q, torch.float32), dev(pools, torch.uint8), dev(bt), dev(c.lens)))
    q, pools, bt, lens = (t.clone() for t in sides[0])
    out = torch.zeros((3, 16 * 128), device=DEV)
    call = lambda: capi.op_paged_attention_fp4(q, 2, pools[0], pools[1], 0.75, 1.25, bt, lens, nb, out)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for c, side in ((then, sides[1]), (first, sides[0])):
        for mine, new in zip((q, pools, bt, lens), side):
            mine.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        ref = c.ref()
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= 2e-5 * c.vmax)


def test_two_threads_at_once(cuda_lib):
    """Calls from two host threads on streams of their own."""
    from concurrent.futures import ThreadPoolExecutor
    cases = [Decode(8, 1, 128, [900, 40], seed=62), Decode(16, 2, 64, [300] * 5, seed=63)]
    want = [c.run()[0] for c in cases]

    def work(c):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            return [c.run()[0] for _ in range(10)]

    with ThreadPoolExecutor(2) as pool:
        for w, outs in zip(want, pool.map(work, cases)):
            assert all(np.array_equal(o, w) for o in outs)


def test_attention_many_uneven_rows_in_a_wide_table(cuda_lib):
    """More than a wave of CTAs and a table of 2048 tokens: rows are taken longest first. Equal, empty and too long
    lengths among them."""
    rng = np.random.default_rng(64)
    lens = rng.integers(1, 200, 128)
    lens[[3, 50, 127]] = 700, 1500, 1500
    lens[10:20] = 77
    c = Decode(8, 4, 64, lens, seed=65, width=128)
    c.check()
    c.lens = lens.copy()
    c.lens[[0, 64, 126]] = 0, 128 * 16 + 1, -5
    got, err = c.run()
    assert err == capi.DEV_SEQLEN_RANGE and not got[[0, 64, 126]].any()
    assert np.all(np.abs(got - c.ref()) <= 2e-5 * c.vmax)
