"""Attention over selected blocks of the paged cache on the GPU: tables and rows
from lengths, key ranges, the choice of blocks and the attention over them,
against the oracle.

Tolerances, from the arithmetic:
* tables, rows, slots, range codes, exponents and chosen blocks: equal. All are
  decided in exact integers, or by fp32 operations that round as IEEE says.
* attention: 2e-5 * max |V| over what the row may reach, as for the other paged
  attention kernels. A score off by e moves the output by at most e max |V|, and
  scores are exact to 2^-22 of sum |q k| / sqrt(d), the sums to 2^-20: with the
  largest queries here (10 times normal, or a single channel of 100 times) that
  is 2.4e-7 * 10 * 128 * 0.64 / 11.3 = 1.7e-5 if all errors had one sign."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle import blocks as ob
from oracle.kv_fp4 import decode, encode, pack_pool, pool_values, unit_bytes
from oracle.numerics import bf16_decode, round_bf16, round_e4m3

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"bf16": capi.DTYPE_BF16, "fp8": capi.DTYPE_E4M3, "fp4": capi.DTYPE_E2M1}


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


def pool_of(x, kind, g=1.0):
    """Raw pool of values x [blocks][nkv][16][d] (their units: what the cache holds)."""
    if kind == "fp4":
        return pack_pool(*encode(np.asarray(x, np.float64) * g, g))
    with np.errstate(invalid="ignore", over="ignore"):
        return round_bf16(x.astype(np.float32)) if kind == "bf16" else round_e4m3(x)


def raw_pool(raw):
    """Raw pool on the device as bytes."""
    return torch.as_tensor(np.ascontiguousarray(raw).view(np.uint8), device=DEV)


# ---------------------------------------------------------------------------
# tables and rows

class Extend:
    def __init__(self, ctx, new, width, nfree, n, at=0, seed=0, short=0, num_blocks=None):
        """short: so many entries of the free list too few."""
        self.ctx, self.new, self.n, self.at = np.asarray(ctx), np.asarray(new), n, at
        rng = np.random.default_rng(seed)
        self.nb = num_blocks or 50000
        ids = rng.permutation(self.nb)
        self.bt = np.full((len(ctx), width), -1, np.int32)
        used = 0
        for s, c in enumerate(self.ctx):
            k = min(width, max(0, -(-int(c) // 16)))
            self.bt[s, :k] = ids[used:used + k]
            used += k
        self.free = ids[used:used + nfree].astype(np.int32)

    def run(self, in_place=False, stream=None):
        a = dict(ctx=dev(self.ctx), new=dev(self.new), bt=dev(self.bt), free=dev(self.free), at=dev([self.at]),
                 cu=dev(np.full(len(self.ctx) + 1, -9)), positions=dev(np.full(self.n, -9)), row_seq=dev(np.full(self.n, -9)),
                 slots=dev(np.full(self.n, -9), torch.int64), err=dev([0]))
        a["held"] = a["ctx"] if in_place else dev(np.full(len(self.ctx), -9))
        a["next"] = a["at"] if in_place else dev([-9])
        capi.op_kv_extend(a["ctx"], a["new"], a["bt"], self.nb, a["free"], a["at"], a["held"], a["cu"], a["positions"],
                          a["row_seq"], a["slots"], a["next"], err=a["err"], stream=stream)
        torch.cuda.synchronize()
        return a

    def check(self, in_place=False):
        a = self.run(in_place)
        want, bits = ob.extend(self.ctx, self.new, self.bt, self.nb, self.free, self.at, self.n)
        for name in ("bt", "held", "cu", "positions", "row_seq", "slots"):
            assert np.array_equal(a[name].cpu().numpy(), want[name]), name
        assert int(a["next"]) == want["free_next"] and int(a["err"]) == bits
        if not in_place:
            assert np.array_equal(a["ctx"].cpu().numpy(), self.ctx) and int(a["at"]) == self.at
        return bits


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nseq,most", [(1, 1), (1, 17), (3, 40), (64, 1), (257, 33), (1024, 9), (1025, 5), (3001, 3)])
def test_extend(cuda_lib, nseq, most, in_place):
    rng = np.random.default_rng(nseq * most)
    ctx, new = rng.integers(0, 100, nseq), rng.integers(0, most + 1, nseq)
    new[0] = max(1, new[0])
    n = int(new.sum()) + int(rng.integers(0, 9))
    assert Extend(ctx, new, 10, 3100, n, at=3, seed=nseq).check(in_place) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [1, 15, 300, 4087, 4088, 70000])
def test_extend_prompts(cuda_lib, n, in_place):
    """One long prompt, then nothing new, then a sequence that begins on a block's edge; rows left over."""
    assert Extend([0, 33, 32], [n, 0, 1], n // 16 + 4, n // 16 + 5, n + 8, seed=n).check(in_place) == 0


@pytest.mark.parametrize("nseq", [4096, 4097, 9000])
def test_extend_many_sequences(cuda_lib, nseq):
    """More sequences than the rows' CTAs keep edges of, most of them without rows."""
    rng = np.random.default_rng(nseq)
    new = np.where(rng.random(nseq) < 0.3, rng.integers(1, 40, nseq), 0)
    e = Extend(rng.integers(0, 30, nseq), new, 5, 9000, int(new.sum()) + 100, seed=nseq)
    assert e.n > 4096 and e.check() == 0 and e.check(True) == 0


def test_extend_nothing(cuda_lib):
    e = Extend([0, 5, 16], [0, 0, 0], 2, 0, 4)
    assert e.check() == 0 and e.check(True) == 0


@pytest.mark.parametrize("seed", range(12))
def test_extend_when_something_runs_out(cuda_lib, seed):
    """Too few blocks, too few rows, bad lengths, ids outside the pool and a bad start of the list, several at once."""
    rng = np.random.default_rng(seed)
    nseq = int(rng.choice([5, 70, 1500]))
    ctx, new = rng.integers(0, 60, nseq), rng.integers(0, 40, nseq)
    bad = rng.random(nseq) < 0.1 * (seed % 3)
    new[bad] = rng.choice([-1, 200, 2 ** 31 - 1], bad.sum())
    ctx[rng.random(nseq) < 0.05 * (seed % 2)] = -7
    total = int(np.where((new > 0) & (new < 100), new, 0).sum())
    e = Extend(ctx, new, 6, int(rng.integers(0, total // 16 + 2)), max(1, int(rng.integers(total // 2, 2 * total + 2))),
               at=int(rng.integers(-1, 3)), seed=seed)
    if seed % 4 == 0 and len(e.free):
        e.free[rng.integers(0, len(e.free), 2)] = [-3, e.nb + 1]
        e.bt[0, 0] = 2 ** 31 - 1
    e.check(seed % 2 == 1)


@pytest.mark.parametrize("nseq,steps", [(70, 40), (4200, 5)])
def test_extend_replayed(cuda_lib, nseq, steps):
    """Captured in place: each replay adds a token to every sequence and goes on in the free list."""
    ctx = np.random.default_rng(1).integers(0, 50, nseq)
    e = Extend(ctx, np.ones(nseq), 8, 6 * nseq, nseq + 2, at=2)
    a = {k: dev(v) for k, v in dict(ctx=e.ctx, new=e.new, bt=e.bt, free=e.free, at=[2], cu=np.zeros(nseq + 1),
                                    positions=np.zeros(e.n), row_seq=np.zeros(e.n)).items()}
    slots, err = dev(np.zeros(e.n), torch.int64), dev([0])
    call = lambda: capi.op_kv_extend(a["ctx"], a["new"], a["bt"], e.nb, a["free"], a["at"], a["ctx"], a["cu"], a["positions"],
                                     a["row_seq"], slots, a["at"], err=err)
    call()                                                           # before the capture, as a program's first step
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    held, bt, at = e.ctx, e.bt, 2
    for i in range(steps):
        want, bits = ob.extend(held, e.new, bt, e.nb, e.free, at, e.n)
        held, bt, at = want["held"], want["bt"], want["free_next"]
        if i:
            g.replay()
    torch.cuda.synchronize()
    for name, key in (("bt", "bt"), ("held", "ctx"), ("cu", "cu"), ("positions", "positions"), ("row_seq", "row_seq")):
        assert np.array_equal(a[key].cpu().numpy(), want[name]), name
    assert np.array_equal(slots.cpu().numpy(), want["slots"]) and int(a["at"]) == at and int(err) == bits == 0


# ---------------------------------------------------------------------------
# key ranges

def check_bounds(x, kind, bt, nb, rows, bits=0, raw=None, nseq=None):
    """x [blocks][nkv][16][d]; rows (sequence, position). Every range, touched or not."""
    nkv, d = x.shape[1], x.shape[3]
    raw = pool_of(x, kind) if raw is None else raw
    vals = pool_values(raw, kind, d, 1.0)
    rng = np.random.default_rng(1)
    codes0 = rng.integers(-128, 128, (nb + 1, nkv, 2, d)).astype(np.int8)
    scales0 = rng.random((nb + 1, nkv)).astype(np.float32)
    codes, scales, err = dev(codes0, torch.int8), dev(scales0, torch.float32), dev([0])
    capi.op_key_bounds(dev([p for _, p in rows]), dev(bt), raw_pool(raw), nkv, d, KINDS[kind], nb, codes, scales,
                       row_seq=dev([s for s, _ in rows]), err=err)
    torch.cuda.synchronize()
    upto = {}
    for s, p in rows:
        if 0 <= s < len(bt) and 0 <= p < 16 * bt.shape[1] and 0 <= bt[s, p // 16] <= nb:
            upto[int(bt[s, p // 16])] = p % 16 + 1
    for b, t in upto.items():
        for h in range(nkv):
            codes0[b, h], scales0[b, h] = ob.key_range(vals[b, h, :t])
    assert np.array_equal(scales.cpu().numpy(), scales0)
    assert np.array_equal(codes.cpu().numpy(), codes0)
    assert int(err) == bits


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("nkv,d", [(1, 64), (8, 128), (3, 64), (2, 128), (9, 64)])
def test_bounds_of_decode_rows(cuda_lib, kind, nkv, d):
    """One row per sequence, every fill of the last block."""
    held = np.arange(1, 40)
    bt, nb = tables(held, 3)
    x = np.random.default_rng(nkv * d).standard_normal((nb + 1, nkv, 16, d)) * 2.0
    check_bounds(x, kind, bt, nb, [(s, h - 1) for s, h in enumerate(held)])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("lens,prefix", [([1], [0]), ([16, 16], [0, 16]), ([100, 1, 33, 700], [5, 31, 0, 17])])
def test_bounds_of_prompt_rows(cuda_lib, kind, lens, prefix):
    held = [a + b for a, b in zip(lens, prefix)]
    bt, nb = tables(held, 4)
    x = np.random.default_rng(len(lens)).standard_normal((nb + 1, 2, 16, 128)) * np.exp(
        np.random.default_rng(5).uniform(-3, 3, (nb + 1, 2, 1, 1)))
    check_bounds(x, kind, bt, nb, [(s, p) for s in range(len(lens)) for p in range(prefix[s], held[s])])


def test_bounds_of_every_size(cuda_lib):
    """BF16 keys over the whole range of exponents, subnormal ones too; borders of the exponent; zeros."""
    rng = np.random.default_rng(6)
    n = 300
    x = rng.standard_normal((n + 1, 2, 16, 64)) * 2.0 ** rng.integers(-134, 125, (n + 1, 2, 1, 1))
    x[:40] = 0.0
    x[10:20, 0, :, 3] = [[127.0], [127.5], [128.0], [63.5], [64.0], [-127.0], [-127.5], [2.0 ** -133], [-(2.0 ** -133)], [1.0]]
    x[20:30, 1, 5, 7] = -(2.0 ** -120)
    x[30:40] = np.where(rng.random((10, 2, 16, 64)) < 0.5, -0.0, 0.0)
    x[40:60, :, :, :32] *= 1e-30                                     # channels far below the block's largest
    check_bounds(x, "bf16", np.arange(n)[None].astype(np.int32), n, [(0, 16 * j + 15) for j in range(n)])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_bounds_of_keys_that_are_not_finite(cuda_lib, kind):
    """They mark their block and head, but not from behind the row's position."""
    n = 9
    x = np.random.default_rng(7).standard_normal((n + 1, 2, 16, 64))
    raw = pool_of(x, kind)
    nan, inf = {"bf16": (0x7FC1, 0xFF80), "fp8": (0x7F, 0xFF), "fp4": (0x7F, 0xFF)}[kind]
    for blk, tok, what in ((0, 0, nan), (1, 15, inf), (2, 7, nan), (3, 8, inf), (4, 8, nan)):
        if kind == "fp4":
            raw.reshape(n + 1, 2, -1)[blk, 1, 16 * 32 + tok * 4 + 2] = what
        else:
            raw[blk, 1, tok, 33] = what
    check_bounds(x, kind, np.arange(n)[None].astype(np.int32), n, [(0, 15), (0, 31), (0, 32 + 7), (0, 48 + 7), (0, 64 + 8)], raw=raw)


def test_bounds_errors(cuda_lib):
    x = np.random.default_rng(8).standard_normal((7, 2, 16, 64))
    bt = np.array([[0, 6, -1], [9, 5, 4]], np.int32)
    check_bounds(x, "bf16", bt, 6, [(0, 3), (0, 48), (0, -1), (2, 5), (-1, 5), (1, 31)], bits=capi.DEV_POS_RANGE)
    check_bounds(x, "bf16", bt, 6, [(0, 33), (1, 3), (1, 40), (0, 20)], bits=capi.DEV_BLOCK_RANGE)


# ---------------------------------------------------------------------------
# choice of blocks

class Select:
    def __init__(self, nq, nkv, d, held, k, first=0, last=1, seed=0, width=None, spread=8):
        self.nq, self.nkv, self.d, self.k, self.first, self.last = nq, nkv, d, k, first, last
        rng = np.random.default_rng(seed)
        self.bt, self.nb = tables(held, seed, width=width)
        self.pos, self.seq = np.asarray(held) - 1, np.arange(len(held))
        a, b = rng.integers(-127, 128, (2, self.nb + 1, nkv, d))
        self.codes = np.stack((np.minimum(a, b), np.maximum(a, b)), 2)
        self.scales = (2.0 ** rng.integers(-spread, spread + 1, (self.nb + 1, nkv))).astype(np.float32)
        self.q = rng.standard_normal((len(held), nq, d)).astype(np.float32)

    def run(self, stream=None):
        sel, err = dev(np.full((len(self.q), self.nkv, self.k), -9)), dev([0])
        capi.op_block_select(dev(self.q, torch.float32), self.nkv, dev(self.codes, torch.int8), dev(self.scales, torch.float32),
                             dev(self.pos), dev(self.bt), self.nb, self.first, self.last, sel, row_seq=dev(self.seq), err=err,
                             stream=stream)
        torch.cuda.synchronize()
        return sel.cpu().numpy(), int(err)

    def want(self):
        out = np.full((len(self.q), self.nkv, self.k), -1)
        G = self.nq // self.nkv
        for i, (s, p) in enumerate(zip(self.seq, self.pos)):
            if not (0 <= s < len(self.bt) and 0 <= p < 16 * self.bt.shape[1]):
                continue
            ids = self.bt[s, :p // 16 + 1]
            ids = np.where((ids < 0) | (ids > self.nb), self.nb, ids)
            for h in range(self.nkv):
                sc = ob.scores(self.q[i, h * G:(h + 1) * G], self.codes[ids, h], self.scales[ids, h])
                got = ob.select(sc, self.first, self.last, self.k)
                out[i, h, :len(got)] = got
        return out

    def check(self, bits=0):
        got, err = self.run()
        assert err == bits
        assert np.array_equal(got, self.want())


@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (4, 2, 64), (5, 1, 64), (16, 1, 128), (3, 3, 128), (27, 3, 64)])
@pytest.mark.parametrize("k,first,last", [(1, 0, 1), (8, 1, 2), (33, 4, 5), (64, 0, 1)])
def test_select(cuda_lib, nq, nkv, d, k, first, last):
    """Contexts from one token to a few thousand, around k blocks among them."""
    held = [1, 15, 16, 17, 16 * k - 1, 16 * k, 16 * k + 1, 16 * (k + 1), 16 * (k + 2) + 5, 700, 2048, 5000]
    Select(nq, nkv, d, held, k, first, last, seed=nq + k).check()


@pytest.mark.parametrize("spread", [0, 100])
@pytest.mark.parametrize("held,k", [(4097, 100), (70000, 2000), (70000, 3), (20000, 1249)])
def test_select_long(cuda_lib, held, k, spread):
    """Scores within one binade, or over most of fp32's range."""
    Select(4, 2, 64, [held, held - 16 * 7], k, 1, 2, seed=held + k, spread=spread).check()


@pytest.mark.parametrize("kinds", [1, 2, 5])
def test_select_ties(cuda_lib, kinds):
    """Tables that repeat a few blocks: whole runs of equal scores, cut at every place."""
    for k in (3, 50, 333, 700):
        c = Select(8, 2, 128, [16 * 800, 16 * 701 + 3], k, 0, 1, seed=kinds)
        c.bt[:] = np.where(c.bt >= 0, c.bt % kinds, c.bt)
        c.check()


@pytest.mark.parametrize("held,k", [(4096, 7), (4097, 4090), (5000, 1), (9000, 700), (40000, 33), (40000, 39999)])
def test_select_tables_of_two_launches(cuda_lib, held, k):
    """Contexts shorter than their wide tables, scratch of the caller's and of the allocator's, in a graph too; scratch that is
    too small is refused."""
    c = Select(8, 2, 64, [16 * held - 3, 16 * (held // 3) + 1, 40, 1], k, 0, 1, seed=held + k)
    want, (got, err) = c.want(), c.run()
    assert err == 0 and np.array_equal(got, want)
    t = (dev(c.q, torch.float32), dev(c.codes, torch.int8), dev(c.scales, torch.float32), dev(c.pos), dev(c.bt))
    size = capi.op_block_select_scratch(4, 2, c.bt.shape[1], k)
    assert (size > 0) == (c.bt.shape[1] > 4096)
    own, sel = torch.zeros(max(size, 1), dtype=torch.uint8, device=DEV), dev(np.zeros(want.shape))
    call = lambda scratch: capi.op_block_select(*t[:1], 2, *t[1:], c.nb, 0, 1, sel, scratch=scratch)
    call(own)
    assert np.array_equal(sel.cpu().numpy(), want)
    for stream in (torch.cuda.Stream(), torch.cuda.current_stream().cuda_stream):      # as an object and as a handle
        sel.zero_()
        torch.cuda.synchronize()
        capi.op_block_select(*t[:1], 2, *t[1:], c.nb, 0, 1, sel, stream=stream)
        torch.cuda.synchronize()
        assert np.array_equal(sel.cpu().numpy(), want)
    if size:
        with pytest.raises(capi.MbtError) as e:
            call(own[:size - 1])
        assert e.value.code == -8
    args = (4, *(capi._ptr(x) for x in t[:1]), 8, 2, 64, *(capi._ptr(x) for x in t[1:4]), None, 4, capi._ptr(t[4]), c.bt.shape[1],
            c.nb, 0, 1, k, capi._ptr(sel), None, 0, None, None)
    sel.zero_()
    torch.cuda.synchronize()
    assert cuda_lib.op_block_select(*args) == 0                      # the stream-ordered allocator's, on the default stream
    torch.cuda.synchronize()
    assert np.array_equal(sel.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(None)
    for _ in range(3):
        sel.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(sel.cpu().numpy(), want)


def test_select_scratch_of_any_size(cuda_lib):
    """A serving program's scratch may pass 2^31 bytes; sizes that no call takes need none."""
    c = Select(8, 2, 64, [16 * 5000 - 3, 40], 20, 0, 1, seed=4)
    t = (dev(c.q, torch.float32), dev(c.codes, torch.int8), dev(c.scales, torch.float32), dev(c.pos), dev(c.bt))
    want = c.want()
    sel = dev(np.zeros(want.shape))
    capi.op_block_select(*t[:1], 2, *t[1:], c.nb, 0, 1, sel, scratch=torch.empty(2 ** 31 + 512, dtype=torch.uint8, device=DEV))
    assert np.array_equal(sel.cpu().numpy(), want)
    assert capi.op_block_select_scratch(1, 1, 5000, 1) > 0
    for n, nkv, width, k in ((2 ** 30 + 1, 1, 5000, 1), (1, 2 ** 16 + 1, 5000, 1), (1, 1, 2 ** 26 + 1, 1), (1, 1, 5000, 2 ** 26 + 1),
                             (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 26, 2 ** 26), (0, 1, 5000, 1), (1, 0, 5000, 1), (1, 1, 0, 1), (1, 1, 5000, 0)):
        assert capi.op_block_select_scratch(n, nkv, width, k) == 0


def test_select_widest_table(cuda_lib):
    """A quarter of a million blocks, few different ones, so most scores are equal."""
    c = Select(2, 1, 64, [16 * 40], 5000, 2, 3, seed=3)
    ids = np.random.default_rng(4).integers(0, 40, 1 << 18)
    c.bt, c.pos = ids[None].astype(np.int32), np.array([(16 << 18) - 1])
    c.check()
    c.k = 60000
    c.check()


def test_select_scores_that_are_not_finite(cuda_lib):
    """Ranges with an infinite scale come first, in order; kept blocks before them."""
    c = Select(8, 2, 64, [16 * 90, 16 * 200], 20, 1, 2, seed=9)
    c.scales[np.random.default_rng(5).random(c.scales.shape) < 0.05] = np.inf
    c.check()
    c.scales[:] = np.inf
    c.check()
    c.scales[:] = 2.0 ** 120                                         # products beyond fp32's range
    c.codes[:, :, 1] = np.maximum(c.codes[:, :, 1], 0)
    c.check()
    c.codes[:], c.scales[::2], c.scales[1::2] = 0, 0.0, 1.0          # nothing but zeros
    c.check()
    c.codes[::3, :, :, :5] = -3                                      # below zero times zero
    c.check()


@pytest.mark.parametrize("what", ["zero", "nan", "inf", "tiny", "huge", "one"])
def test_select_queries_of_every_size(cuda_lib, what):
    c = Select(8, 2, 64, [16 * 90, 16 * 33, 16 * 300], 20, 1, 1, seed=10)
    if what in ("zero", "nan", "inf"):
        c.q[1] = 0.0
        c.q[0, 5, 7] = {"zero": 0.0, "nan": np.nan, "inf": -np.inf}[what]
    else:
        c.q *= np.float32({"tiny": 1e-44, "huge": 3e37, "one": 0.0}[what])
        if what == "one":
            c.q[:, 3, 9] = -2.0 ** -149
    c.check()


def test_select_rows_of_one_sequence(cuda_lib):
    """Rows of a prompt's piece and of other sequences, in any order, each with its own context; null row_seq."""
    c = Select(8, 4, 128, [5000, 900], 12, 1, 2, seed=11)
    rng = np.random.default_rng(12)
    c.seq = rng.integers(0, 2, 70)
    c.pos = np.where(c.seq == 0, rng.integers(0, 5000, 70), rng.integers(0, 900, 70))
    c.q = rng.standard_normal((70, 8, 128)).astype(np.float32)
    c.check()
    c.seq, c.pos, c.q = np.arange(2), c.pos[:2] % 900, c.q[:2]
    want = c.want()
    sel = dev(np.zeros(want.shape))
    capi.op_block_select(dev(c.q, torch.float32), 4, dev(c.codes, torch.int8), dev(c.scales, torch.float32), dev(c.pos), dev(c.bt),
                         c.nb, 1, 2, sel)
    assert np.array_equal(sel.cpu().numpy(), want)


def test_select_errors(cuda_lib):
    c = Select(8, 2, 64, [16 * 90, 16 * 33, 16 * 300], 20, 1, 1, seed=13)
    c.bt[2, 5], c.bt[0, 3] = c.nb + 1, -1
    c.check(capi.DEV_BLOCK_RANGE)
    c.bt[2, 5], c.bt[0, 3] = 0, 0
    c.seq, c.pos = np.array([0, 3, 1, -1, 2]), np.array([16 * 300, 5, -1, 5, 77])
    c.q = np.repeat(c.q, 2, 0)[:5]
    c.check(capi.DEV_POS_RANGE)
    c.seq, c.pos = np.array([0, 0, 0, 0, 0]), np.array([5, 50, 17, 5, 77])       # all of a context with a bad id
    c.bt[0, 1] = c.nb + 7
    c.check(capi.DEV_BLOCK_RANGE)


def test_select_follows_its_inputs_in_a_graph(cuda_lib):
    a, b = Select(8, 2, 64, [16 * 90, 16 * 300], 20, 1, 1, seed=14), Select(8, 2, 64, [16 * 300, 16 * 7], 20, 1, 1, seed=15)
    nb, width = max(a.nb, b.nb), 300
    sides = []
    for c in (a, b):
        codes, scales, bt = np.zeros((nb + 1, 2, 2, 64)), np.zeros((nb + 1, 2)), np.full((2, width), -1)
        codes[:c.nb + 1], scales[:c.nb + 1], bt[:, :c.bt.shape[1]] = c.codes, c.scales, c.bt
        sides.append((dev(c.q, torch.float32), dev(codes, torch.int8), dev(scales, torch.float32), dev(c.pos), dev(bt)))
    q, codes, scales, pos, bt = (t.clone() for t in sides[0])
    sel = dev(np.zeros((2, 2, 20)))
    call = lambda: capi.op_block_select(q, 2, codes, scales, pos, bt, nb, 1, 1, sel)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for c, side in ((b, sides[1]), (a, sides[0])):
        for mine, new in zip((q, codes, scales, pos, bt), side):
            mine.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(sel.cpu().numpy(), c.want())


# ---------------------------------------------------------------------------
# attention

class Attend:
    def __init__(self, kind, nq, nkv, d, held, k, seed=0, rows=None, kg=0.75, vg=1.25, scale=1.0):
        """rows: (sequence, position) pairs, or one row per sequence at its end."""
        self.kind, self.nq, self.nkv, self.d, self.k, self.kg, self.vg = kind, nq, nkv, d, k, kg, vg
        rng = np.random.default_rng(seed)
        self.bt, self.nb = tables(held, seed)
        rows = [(s, h - 1) for s, h in enumerate(held)] if rows is None else rows
        self.seq, self.pos = np.array([s for s, _ in rows]), np.array([p for _, p in rows])
        self.kp, self.vp = (pool_of(rng.standard_normal((self.nb + 1, nkv, 16, d)), kind, g) for g in (kg, vg))
        self.q = (rng.standard_normal((len(rows), nq, d)) * scale).astype(np.float32)
        self.sel = np.full((len(rows), nkv, k), -1)
        for i, p in enumerate(self.pos):
            for h in range(nkv):
                pick = rng.permutation(p // 16 + 1)[:k]
                if p // 16 not in pick:
                    pick[0] = p // 16
                self.sel[i, h, :len(pick)] = np.sort(pick)

    def values(self):
        return pool_values(self.kp, self.kind, self.d, self.kg), pool_values(self.vp, self.kind, self.d, self.vg)

    def run(self, stream=None):
        out, err = torch.full((len(self.q), self.nq * self.d), float("nan"), device=DEV), dev([0])
        capi.op_block_attention(dev(self.q, torch.float32), self.nkv, raw_pool(self.kp), raw_pool(self.vp), KINDS[self.kind],
                                self.kg, self.vg, dev(self.pos), dev(self.bt), dev(self.sel), self.nb, out,
                                row_seq=dev(self.seq), err=err, stream=stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), int(err)

    def want(self):
        k, v = self.values()
        ok = (self.seq >= 0) & (self.seq < len(self.bt)) & (self.pos >= 0) & (self.pos < 16 * self.bt.shape[1])
        bt = np.where((self.bt < 0) | (self.bt > self.nb), self.nb, self.bt)
        return ob.attention(self.q, k, v, bt, np.where(ok, self.seq, -1), self.pos, self.sel)

    def check(self, bits=0):
        got, err = self.run()
        want, most = self.want()
        assert err == bits
        assert np.all(np.abs(got - want) <= 2e-5 * most), np.nanmax(np.abs(got - want))
        return got


ALL = ["bf16", "fp8", "fp4"]


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 128), (1, 1, 64), (4, 2, 64), (3, 1, 128), (5, 1, 128), (16, 1, 128), (9, 1, 64),
                                      (40, 8, 64), (12, 4, 64), (39, 3, 128)])
def test_attention(cuda_lib, kind, nq, nkv, d):
    """Contexts from one token on, all or a few of their blocks."""
    Attend(kind, nq, nkv, d, [1, 2, 15, 16, 17, 31, 33, 100, 160, 161, 700], 10, seed=nq + d).check()


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("k", [1, 2, 3, 5, 8, 31, 64, 257, 1000])
def test_attention_every_number_of_blocks(cuda_lib, kind, k):
    for n in (1, 3):
        Attend(kind, 8, 2, 128 if n == 1 else 64, [16 * k + 5, 16 * k - 3, 16 * 1200][:n], k, seed=k).check()


@pytest.mark.parametrize("kind", ALL)
def test_attention_rows_of_a_prompt(cuda_lib, kind):
    """Many rows of few sequences, every row with blocks and a position of its own."""
    rng = np.random.default_rng(21)
    rows = [(int(s), int(rng.integers(0, (900, 260, 16)[s]))) for s in rng.integers(0, 3, 300)]
    Attend(kind, 8, 4, 128, [900, 260, 16], 9, seed=22, rows=rows).check()


@pytest.mark.parametrize("kind", ALL)
def test_attention_lists_of_any_form(cuda_lib, kind):
    """Entries out of order, gaps, blocks twice, rows with one or no block; entries beyond the context are flagged."""
    c = Attend(kind, 8, 2, 64, [900] * 8, 12, seed=23)
    rng = np.random.default_rng(24)
    c.sel = rng.permuted(c.sel, axis=2)
    c.sel[1][rng.random((2, 12)) < 0.5] = -1
    c.sel[2] = -1
    c.sel[3, 0], c.sel[3, 1, 1:] = -1, -(2 ** 31)
    c.sel[4, :, 3:] = c.sel[4, :, :9]
    c.sel[5] = 56
    c.check()
    c.sel[6, 0, 4], c.sel[7, 1, 11] = 57, 2 ** 31 - 1
    c.check(capi.DEV_BLOCK_RANGE)


@pytest.mark.parametrize("kind", ALL)
def test_attention_never_sees_past_a_position(cuda_lib, kind):
    """NaN and infinities in the block's later tokens and in blocks not chosen change nothing."""
    c = Attend(kind, 16, 2, 128, [37, 16, 1, 730], 5, seed=25)
    want = c.run()[0]
    nan, inf = {"bf16": (0x7FC1, 0xFF80), "fp8": (0x7F, 0xFF), "fp4": (0x7F, 0xFF)}[kind]
    for pool in (c.kp, c.vp):
        used = np.zeros((c.nb + 1, c.nkv, 16), bool)
        for i, p in enumerate(c.pos):
            for h in range(c.nkv):
                for j in c.sel[i, h][c.sel[i, h] >= 0]:
                    used[c.bt[i, j], h, :min(16, p - 16 * j + 1)] = True
        if kind == "fp4":
            sc = pool[..., 16 * 64:].reshape(c.nb + 1, c.nkv, 16, 8)
            sc[~used] = nan
            pool[..., 16 * 64:] = sc.reshape(c.nb + 1, c.nkv, -1)
        else:
            pool[~used] = nan
            pool[..., ::2][~used] = inf
    got, err = c.run()
    assert err == 0 and np.array_equal(got, want)


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("nq", [8, 14])
def test_attention_values_that_are_not_finite(cuda_lib, kind, nq):
    """A key: its rows. A value: its channel of the rows that see it, an infinity as such. Others keep every bit."""
    h = nq // 2                                                      # heads of the second KV head from here on
    c = Attend(kind, nq, 2, 64, [700, 700, 700], 8, seed=26)
    c.sel[1] = c.sel[0]
    want = c.run()[0].reshape(3, nq, 64)
    nan = {"bf16": 0x7FC1, "fp8": 0x7F, "fp4": 0x7F}[kind]
    blk = c.bt[0, c.sel[0, 1, 2]]
    raw = c.vp.copy()
    if kind == "fp4":
        raw.reshape(c.nb + 1, 2, -1)[blk, 1, 16 * 32 + 5 * 4 + 2] = nan
        hit = np.arange(64) // 16 == 2
    else:
        raw[blk, 1, 5, 33] = nan
        hit = np.arange(64) == 33
    c.vp, keep = raw, c.vp
    got = c.run()[0].reshape(3, nq, 64)
    assert np.isnan(got[0, h:][:, hit]).all()
    got[0, h:][:, hit] = want[0, h:][:, hit]
    assert np.array_equal(got, want)
    if kind == "bf16":
        raw[blk, 1, 5, 33], raw[blk, 1, 6, 40], raw[blk, 1, 7, 40], raw[blk, 1, 15, 63] = 0x7F80, 0x7F80, 0xFF80, 0xFF80
        got = c.run()[0].reshape(3, nq, 64)
        assert np.all(got[0, h:, 33] == np.inf) and np.isnan(got[0, h:, 40]).all() and np.all(got[0, h:, 63] == -np.inf)
        got[0, h:][:, [33, 40, 63]] = want[0, h:][:, [33, 40, 63]]
        assert np.array_equal(got, want)
    c.vp, raw = keep, c.kp.copy()
    for bad in ((nan, 0x7F80, 0xFF80) if kind == "bf16" else (nan,)):
        c.kp = raw.copy()
        if kind == "fp4":
            c.kp.reshape(c.nb + 1, 2, -1)[blk, 1, 16 * 32 + 5 * 4 + 2] = bad
        else:
            c.kp[blk, 1, 5, 33] = bad
        got = c.run()[0].reshape(3, nq, 64)
        assert np.isnan(got[0, h:]).all()
        got[0, h:] = want[0, h:]
        assert np.array_equal(got, want)


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("n", [40, 64, 110, 300])
def test_attention_many_rows(cuda_lib, kind, n):
    """CTAs of four, two and one warps, one wave and several; over a BF16 cache with infinities in some rows' values."""
    rng = np.random.default_rng(n)
    c = Attend(kind, 16, 8, 128, rng.integers(1, 90, n), 3, seed=n)
    for i in range(0, n, 13):
        c.sel[i, i % 8] = -1
    got, (want, most) = c.run()[0], c.want()
    assert np.all(np.abs(got - want) <= 2e-5 * most)
    if kind == "bf16":
        for i in range(0, n, 7):
            c.vp[c.bt[i, c.pos[i] // 16], i % 8, 0, i % 128] = 0x7F80
        odd = np.zeros((n, 8, 2, 128), bool)
        for i in range(0, n, 7):
            if (c.sel[i, i % 8] == c.pos[i] // 16).any():
                odd[i, i % 8, :, i % 128] = True
        odd, again = odd.reshape(n, -1), c.run()[0]
        assert odd.any() and np.all(again[odd] == np.inf) and np.array_equal(again[~odd], got[~odd])


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("nq", [8, 14])
def test_attention_queries_that_are_not_finite(cuda_lib, kind, bad, nq):
    c = Attend(kind, nq, 2, 64, [700, 20], 8, seed=27)
    want = c.run()[0].reshape(2, nq, 64)
    c.q[1, 5, 9] = bad
    got = c.run()[0].reshape(2, nq, 64)
    assert np.isnan(got[1, 5]).all()
    got[1, 5] = want[1, 5]
    assert np.array_equal(got, want)


@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("scale", [0.0, 1e-44, 1e-30, 10.0, 100.0, 1e30])
@pytest.mark.parametrize("nq", [8, 14])
def test_attention_queries_of_every_size(cuda_lib, kind, scale, nq):
    """Even and one-hot softmaxes; heads of very different size in one group."""
    c = Attend(kind, nq, 2, 128, [700, 20, 333], 40, seed=28)
    c.q[:, 1::2] *= np.float32(scale)
    if scale >= 100:                                                 # scores that fp32's own rounding does not reorder
        keep = np.zeros_like(c.q[:, 1::2])
        keep[..., 3] = c.q[:, 1::2, 3]
        c.q[:, 1::2] = keep
    c.check()


@pytest.mark.parametrize("nq", [8, 14])
def test_attention_bf16_values_of_every_size(cuda_lib, nq):
    """Keys and values from the smallest to the largest BF16 numbers, in one block and over blocks."""
    c = Attend("bf16", nq, 2, 64, [900] * 3, 30, seed=29, kg=1.0, vg=1.0)
    rng = np.random.default_rng(30)
    v = bf16_decode(c.vp) * 2.0 ** rng.integers(-120, 100, c.vp.shape[:3] + (1,))
    c.vp = round_bf16(v.astype(np.float32))
    k = bf16_decode(c.kp) * 2.0 ** rng.integers(-130, 2, c.kp.shape[:3] + (1,))
    c.kp = round_bf16(k.astype(np.float32))
    c.check()


@pytest.mark.parametrize("kind", ALL)
def test_attention_small_probabilities_behind_a_dominant_one(cuda_lib, kind):
    """One token takes nearly all; many small shares still count."""
    c = Attend(kind, 4, 1, 64, [16 * 600], 600, seed=31, kg=1.0, vg=1.0)
    x, y = np.zeros((c.nb + 1, 1, 16, 64)), np.ones((c.nb + 1, 1, 16, 64))
    x[c.bt[0, 0], 0, 0, :16] = 4.0
    y[c.bt[0, 0], 0, 0] = 0.0
    c.kp, c.vp = pool_of(x, kind), pool_of(y, kind)
    for lead in (6.0, 9.0, 12.0):
        c.q[:] = 0.0
        c.q[..., :16] = lead * 8 / 64
        c.check()


def test_attention_errors(cuda_lib):
    c = Attend("bf16", 8, 2, 64, [100, 40], 3, seed=32)
    c.bt[0, 6], c.sel[0, 0], c.sel[0, 1] = -4, [0, 1, 6], [0, 1, 2]
    c.check(capi.DEV_BLOCK_RANGE)
    c.bt[0, 6] = 1
    c.seq, c.pos = np.array([0, 2, 1, -1, 0]), np.array([112, 5, -1, 5, 77])
    c.q, c.sel = np.repeat(c.q, 3, 0)[:5], np.zeros((5, 2, 3), int)
    got = c.check(capi.DEV_POS_RANGE)
    assert not got[:4].any() and got[4].any()


@pytest.mark.parametrize("kind", ALL)
def test_attention_blocks_beyond_four_gigabytes(cuda_lib, kind):
    """The same blocks at a pool's start and behind 2^32 bytes of a large one."""
    c = Attend(kind, 8, 8, 128, [100], 4, seed=33)
    per = c.kp.nbytes // (c.nb + 1)
    far = 2 ** 32 // per + 3
    want = c.run()[0]
    pools = [torch.empty((far + c.nb + 1) * per, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for p, raw in zip(pools, (c.kp, c.vp)):
        p[far * per:] = raw_pool(raw).reshape(-1)
    out = torch.zeros((1, 8 * 128), device=DEV)
    capi.op_block_attention(dev(c.q, torch.float32), 8, *pools, KINDS[kind], c.kg, c.vg, dev(c.pos),
                            dev(np.where(c.bt >= 0, c.bt + far, -1)), dev(c.sel), far + c.nb, out, row_seq=dev(c.seq))
    assert np.array_equal(out.double().cpu().numpy(), want)
    codes = [torch.zeros((n + 1, 8, 2, 128), dtype=torch.int8, device=DEV) for n in (c.nb, far + c.nb)]
    scales = [torch.zeros((n + 1, 8), device=DEV) for n in (c.nb, far + c.nb)]
    rows, seq = dev(np.arange(100)), dev(np.zeros(100))
    capi.op_key_bounds(rows, dev(c.bt), raw_pool(c.kp), 8, 128, KINDS[kind], c.nb, codes[0], scales[0], row_seq=seq)
    capi.op_key_bounds(rows, dev(np.where(c.bt >= 0, c.bt + far, -1)), pools[0], 8, 128, KINDS[kind], far + c.nb, codes[1],
                       scales[1], row_seq=seq)
    assert torch.equal(codes[0], codes[1][far:]) and torch.equal(scales[0], scales[1][far:]) and scales[0].any()


def test_attention_in_graphs_at_once(cuda_lib):
    """Two captured calls of different shapes replayed on two streams at the same time equal the eager results."""
    cases = [Attend("bf16", 8, 1, 128, [5000, 40], 100, seed=34), Attend("fp8", 16, 2, 64, [300] * 9, 7, seed=35)]
    want, graphs, outs, keep = [], [], [], []
    for c in cases:
        want.append(c.run()[0])
        t = (dev(c.q, torch.float32), raw_pool(c.kp), raw_pool(c.vp), dev(c.pos), dev(c.bt), dev(c.sel))
        out = torch.zeros((len(c.q), c.nq * c.d), device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            capi.op_block_attention(t[0], c.nkv, t[1], t[2], KINDS[c.kind], c.kg, c.vg, t[3], t[4], t[5], c.nb, out)
        graphs.append(g), outs.append(out), keep.append(t)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.double().cpu().numpy(), w)
    assert np.array_equal(cases[0].run(stream=streams[0])[0], want[0])


# ---------------------------------------------------------------------------
# together

@pytest.mark.parametrize("graph", [False, True])
def test_a_serving_loop(cuda_lib, graph):
    """Prompts, then single tokens: blocks from the free list, the 4-bit write, ranges, choice, attention; every step's
    outputs against the oracle's own tables and cache. Captured: the same step replayed with new inputs, padding rows in
    the null block."""
    nq, nkv, d, kg, vg, k, width, nseq = 8, 2, 64, 0.875, 1.25, 4, 16, 3
    rng = np.random.default_rng(40)
    nb = nseq * width
    free = rng.permutation(nb).astype(np.int32)
    bt_ref, held, at = np.full((nseq, width), -1, np.int32), np.zeros(nseq, int), 0
    bt = dev(np.concatenate((bt_ref, np.full((1, width), nb, np.int32))))       # one more row: the null block
    pools = torch.zeros((2, nb + 1, nkv, unit_bytes(d)), dtype=torch.uint8, device=DEV)
    kv = np.zeros((2, nb + 1, nkv, 16, d))
    codes = torch.zeros((nb + 1, nkv, 2, d), dtype=torch.int8, device=DEV)
    scales = torch.zeros((nb + 1, nkv), device=DEV)
    ctx, free_d, free_at, err = dev(held), dev(free), dev([0]), dev([0])
    table = torch.empty((256, d // 2, 2), device=DEV)
    capi.op_rope_table(256, d, 10000.0, table)
    cs = table.double().cpu().numpy()

    def buffers(n):
        return dict(qkv=torch.zeros((n, (nq + 2 * nkv) * d), device=DEV), new=dev(np.zeros(nseq)), cu=dev(np.zeros(nseq + 1)),
                    pos=dev(np.zeros(n)), seq=dev(np.zeros(n)), slots=dev(np.zeros(n), torch.int64),
                    q=torch.zeros((n, nq, d), device=DEV), sel=dev(np.zeros((n, nkv, k))), out=torch.zeros((n, nq * d), device=DEV))

    def step(b):
        capi.op_kv_extend(ctx, b["new"], bt[:nseq], nb, free_d, free_at, ctx, b["cu"], b["pos"], b["seq"], b["slots"], free_at, err=err)
        capi.op_rope_kv_write_fp4(b["qkv"], nq, nkv, d, b["pos"], bt, table, pools[0], pools[1], nb, kg, vg, b["q"],
                                  row_seq=b["seq"], err=err)
        capi.op_key_bounds(b["pos"], bt, pools[0], nkv, d, capi.DTYPE_E2M1, nb, codes, scales, row_seq=b["seq"], err=err)
        capi.op_block_select(b["q"], nkv, codes, scales, b["pos"], bt, nb, 1, 1, b["sel"], row_seq=b["seq"], err=err)
        capi.op_block_attention(b["q"], nkv, pools[0], pools[1], capi.DTYPE_E2M1, kg, vg, b["pos"], bt, b["sel"], nb, b["out"],
                                row_seq=b["seq"], err=err)

    small, g = buffers(8), None
    for new in ([40, 0, 100], [1, 70, 1], [1, 1, 1], [1, 0, 1], [0, 1, 1], [2, 2, 2], [1, 1, 1], [1, 1, 1], [1, 1, 1]):
        rows = sum(new)
        b = small if rows <= 8 else buffers(rows + 3)
        x = rng.standard_normal((len(b["pos"]), nq + 2 * nkv, d)).astype(np.float32)
        b["qkv"].copy_(dev(x.reshape(len(x), -1), torch.float32))
        b["new"].copy_(dev(new))
        if graph and b is small:
            if g is None:
                saved = [t.clone() for t in (ctx, free_at, bt, pools, codes, scales)]
                step(b)                                              # warm-up, then back to where it was
                torch.cuda.synchronize()
                for t, old in zip((ctx, free_at, bt, pools, codes, scales), saved):
                    t.copy_(old)
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step(b)
            g.replay()
        else:
            step(b)
        torch.cuda.synchronize()
        want, bits = ob.extend(held, new, bt_ref, nb, free, at, len(b["pos"]))
        bt_ref, held, at = want["bt"], want["held"], want["free_next"]
        assert bits == 0 and int(err) == 0 and int(free_at) == at
        assert np.array_equal(bt[:nseq].cpu().numpy(), bt_ref) and np.array_equal(b["slots"].cpu().numpy(), want["slots"])
        pos, seq = want["positions"][:rows], want["row_seq"][:rows]
        h = d // 2
        c, s = cs[pos, :, 0][:, None], cs[pos, :, 1][:, None]
        p1, p2 = x[:rows, :nq + nkv, :h].astype(np.float64), x[:rows, :nq + nkv, h:].astype(np.float64)
        y = np.concatenate((p1 * c - p2 * s, p2 * c + p1 * s), -1)
        for i in range(rows):
            slot = bt_ref[seq[i], pos[i] // 16], slice(None), pos[i] % 16
            kv[0][slot] = decode(*encode(y[i, nq:], kg), kg)
            kv[1][slot] = decode(*encode(x[i, nq + nkv:].astype(np.float64), vg), vg)
        q = b["q"][:rows].cpu().numpy()
        assert np.all(np.abs(q - y[:, :nq]) <= 1e-5)
        ranges = {}
        for i in range(rows):                                        # what the cache holds after this step
            for j in range(int(pos[i]) // 16 + 1):
                blk = int(bt_ref[seq[i], j])
                if blk not in ranges:
                    t = min(16, int(held[seq[i]]) - 16 * j)
                    ranges[blk] = [ob.key_range(kv[0][blk, hh, :t] / kg) for hh in range(nkv)]
        sel = np.full((rows, nkv, k), -1)
        for i in range(rows):
            ids = [int(bt_ref[seq[i], j]) for j in range(int(pos[i]) // 16 + 1)]
            for hh in range(nkv):
                sc = ob.scores(q[i, hh * 4:hh * 4 + 4], np.array([ranges[z][hh][0] for z in ids]),
                               np.array([ranges[z][hh][1] for z in ids]))
                got = ob.select(sc, 1, 1, k)
                sel[i, hh, :len(got)] = got
        assert np.array_equal(b["sel"][:rows].cpu().numpy(), sel)
        ref, most = ob.attention(q, kv[0], kv[1], bt_ref, seq, pos, sel)
        assert np.all(np.abs(b["out"][:rows].double().cpu().numpy() - ref) <= 2e-5 * most)


def test_captured_between_other_work(cuda_lib):
    """Behind copies, fills and another stream's work, and before what overwrites its inputs, many times over."""
    att, sel = Attend("bf16", 8, 2, 128, [900, 40], 20, seed=45), Select(8, 2, 64, [16 * 300, 16 * 90], 20, 1, 1, seed=46)
    ext = Extend([3, 40], [20, 1], 5, 40, 24, seed=47)
    e, want = ext.run(), (att.run()[0], sel.run()[0])
    a = (dev(att.q, torch.float32), raw_pool(att.kp), raw_pool(att.vp), dev(att.pos), dev(att.bt), dev(att.sel))
    b = (dev(sel.q, torch.float32), dev(sel.codes, torch.int8), dev(sel.scales, torch.float32), dev(sel.pos), dev(sel.bt))
    c = (dev(ext.ctx), dev(ext.new), dev(ext.bt), dev(ext.free), dev([0]))
    mine = [[torch.zeros_like(t) for t in x] for x in (a, b, c)]
    out, chosen = torch.zeros((2, 8 * 128), device=DEV), dev(np.zeros((2, 2, 20)))
    held, cu, pos, seq, nxt = dev([0, 0]), dev([0] * 3), dev(np.zeros(24)), dev(np.zeros(24)), dev([0])
    slots, side = dev(np.zeros(24), torch.int64), torch.cuda.Stream()
    codes, scales = torch.zeros((att.nb + 1, 2, 2, 128), dtype=torch.int8, device=DEV), torch.zeros((att.nb + 1, 2), device=DEV)

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for m, t in zip(mine[0] + mine[1], a + b):
                m.copy_(t)
        for m, t in zip(mine[2], c):
            m.copy_(t)
        out.fill_(float("nan"))
        capi.op_kv_extend(*mine[2][:3], ext.nb, *mine[2][3:], held, cu, pos, seq, slots, nxt)
        torch.cuda.current_stream().wait_stream(side)
        capi.op_key_bounds(mine[0][3], mine[0][4], mine[0][1], 2, 128, capi.DTYPE_BF16, att.nb, codes, scales)
        capi.op_block_select(mine[1][0], 2, *mine[1][1:], sel.nb, 1, 1, chosen)
        capi.op_block_attention(mine[0][0], 2, *mine[0][1:3], capi.DTYPE_BF16, att.kg, att.vg, *mine[0][3:], att.nb, out)
        for m in mine[0] + mine[1] + mine[2]:                        # the next step's copies do not wait for more than this
            m.fill_(0)

    step()
    torch.cuda.synchronize()
    first = codes.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            step()
    for _ in range(5):
        for t in (out, chosen, slots, codes):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(chosen.cpu().numpy(), want[1])
        assert torch.equal(slots, e["slots"]) and torch.equal(held, e["held"]) and torch.equal(codes, first) and first.any()


def test_two_threads_at_once(cuda_lib):
    """Calls from two host threads on streams of their own."""
    from concurrent.futures import ThreadPoolExecutor
    att = [Attend("bf16", 8, 1, 128, [900, 40], 20, seed=41), Attend("fp4", 16, 2, 64, [300] * 5, 6, seed=42)]
    sel = [Select(8, 2, 64, [16 * 300, 16 * 90], 20, 1, 1, seed=43), Select(8, 1, 128, [16 * 60], 10, 1, 1, seed=44)]
    want = [(a.run()[0], s.run()[0]) for a, s in zip(att, sel)]

    def work(i):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            return [(att[i].run()[0], sel[i].run()[0]) for _ in range(10)]

    with ThreadPoolExecutor(2) as pool:
        for w, outs in zip(want, pool.map(work, (0, 1))):
            assert all(np.array_equal(o[0], w[0]) and np.array_equal(o[1], w[1]) for o in outs)


@pytest.mark.parametrize("what", ["dtype", "shape", "strided", "host"])
def test_binding_refuses(cuda_lib, what):
    def bad(t):
        if what == "dtype":
            return t.to(torch.float64)
        if what == "shape":
            return torch.cat((t, t[:1]))
        if what == "host":
            return t.cpu()
        wide = torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=DEV)
        return wide[..., ::2]

    i, pos, one = dev(np.zeros((4, 3))), dev(np.zeros(4)), dev([0])
    p = torch.zeros(6 * 2 * 576, dtype=torch.uint8, device=DEV)
    codes, sc = torch.zeros((6, 2, 2, 64), dtype=torch.int8, device=DEV), torch.zeros((6, 2), device=DEV)
    q, out, sel = torch.zeros((4, 4, 64), device=DEV), torch.zeros((4, 256), device=DEV), dev(np.zeros((4, 2, 3)))
    calls = [
        (capi.op_kv_extend, [pos, pos.clone(), i, 5, pos.clone(), one, pos.clone(), dev(np.zeros(5)), pos.clone(), pos.clone(),
                             dev(np.zeros(4), torch.int64), one.clone()], (0, 1, 2, 5, 6, 7, 9, 10, 11)),
        (capi.op_key_bounds, [pos, i, p, 2, 64, 3, 5, codes, sc], (7, 8)),
        (capi.op_block_select, [q, 2, codes, sc, pos, i, 5, 1, 1, sel], (2, 3, 4, 9)),
        (capi.op_block_attention, [q, 2, p, p, 3, 1.0, 1.0, pos, i, sel, 5, out], (7, 9, 11)),
    ]
    for fn, args, where in calls:
        fn(*args)
        for w in where:
            if what == "strided" and args[w].numel() == 1:
                continue
            wrong = list(args)
            wrong[w] = bad(args[w])
            with pytest.raises(ValueError):
                fn(*wrong)
    torch.cuda.synchronize()


@pytest.mark.parametrize("first,last,k", [(2 ** 32, 1, 3), (0, 2 ** 32 + 1, 3), (-1, 1, 3), (0, 0, 3), (2, 2, 3), (2 ** 80, 1, 3)])
def test_kept_blocks_beyond_k(cuda_lib, first, last, k):
    """The numbers of kept blocks are checked as they are, not what 32 bits leave of them."""
    c = Select(8, 2, 64, [16 * 30], k, seed=48)
    c.first, c.last = first, last
    with pytest.raises(capi.MbtError) as e:
        c.run()
    assert e.value.code == -1


def test_binding_numbers_and_pools(cuda_lib):
    """Numbers beyond 32 bits, head sizes and formats that are not there, small pools, missing row_seq, other types."""
    c = Attend("fp4", 8, 2, 64, [100], 4, seed=49)
    t = [dev(c.q, torch.float32), 2, raw_pool(c.kp), raw_pool(c.vp), capi.DTYPE_E2M1, 1.0, 1.0, dev(c.pos), dev(c.bt), dev(c.sel),
         c.nb, torch.zeros((1, 512), device=DEV)]
    capi.op_block_attention(*t)
    capi.op_block_attention(*t, stream=torch.cuda.current_stream().cuda_stream)

    def wrong(i, x):
        return t[:i] + [x] + t[i + 1:]

    for args in (wrong(10, c.nb + 2 ** 32), wrong(4, capi.DTYPE_E2M1 + 2 ** 32), wrong(4, 2), wrong(1, 2 - 2 ** 32), wrong(10, 0),
                 wrong(5, 0.0), wrong(6, float("nan"))):
        with pytest.raises(capi.MbtError) as e:
            capi.op_block_attention(*args)
        assert e.value.code == -1
    for args in (wrong(2, t[2][:-1].contiguous()), wrong(3, t[3].cpu()), wrong(0, c.q), wrong(7, dev(np.zeros(2))), wrong(10, c.nb + 1),
                 wrong(8, torch.zeros((0, 7), dtype=torch.int32, device=DEV)), wrong(0, t[0][0])):
        with pytest.raises(ValueError):
            capi.op_block_attention(*args)
    for args in (wrong(5, "1"), wrong(1, 2.0)):
        with pytest.raises(TypeError):
            capi.op_block_attention(*args)
    torch.cuda.synchronize()
