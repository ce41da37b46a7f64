"""The oracle of block selection pinned on its definitions, and the host-side
refusals of its entry points (no GPU)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import build, capi
from oracle.blocks import attention, extend, key_range, rounded_queries, scores, select
from oracle.kv_fp4 import rows_attention


def test_extend_by_hand():
    bt = np.full((4, 3), -1)
    bt[0, 0], bt[1, :2] = 7, (5, 6)
    out, bits = extend([16, 20, 0, 0], [1, 3, 0, 17], bt, 9, [8, 3, 4, 1, 0], 1, 24)
    assert bits == 0
    assert out["bt"].tolist() == [[7, 3, -1], [5, 6, -1], [-1, -1, -1], [4, 1, -1]]
    assert out["held"].tolist() == [17, 23, 0, 17] and out["cu"].tolist() == [0, 1, 4, 4, 21] and out["free_next"] == 4
    assert out["positions"].tolist() == [16, 20, 21, 22] + list(range(17)) + [0] * 3
    assert out["row_seq"].tolist() == [0, 1, 1, 1] + [3] * 17 + [4] * 3
    assert out["slots"].tolist() == [48, 100, 101, 102] + list(range(64, 80)) + [16] + [144] * 3


def test_extend_when_something_runs_out():
    bt = np.full((4, 2), -1)
    bt[3, 0] = 2
    out, bits = extend([0, 0, -1, 5], [16, 17, 4, 2], bt, 9, [6, 7], 0, 40)       # two blocks more than there are
    assert bits == 2 | 8 and out["held"].tolist() == [16, 0, -1, 7] and out["free_next"] == 1
    assert out["bt"].tolist() == [[6, -1], [-1, -1], [-1, -1], [2, -1]] and out["cu"].tolist() == [0, 16, 16, 16, 18]
    out, bits = extend([0, 0, 0, 0], [16, 5, 0, 1], bt, 9, [6, 7, 8], 0, 18)      # the second's rows do not fit, nor those behind
    assert bits == 4 and out["held"].tolist() == [16, 0, 0, 0] and out["free_next"] == 1
    assert extend([0], [1], bt[:1], 9, [6], 2, 4)[1] == 2 and extend([0], [33], bt[:1], 9, [6], 0, 40)[1] == 8
    out, bits = extend([0], [1], bt[:1], 9, [11], 0, 1)                           # an id outside the pool
    assert bits == 2 and out["slots"].tolist() == [-1]


def test_key_range_holds_its_keys_tightly():
    rng = np.random.default_rng(0)
    for i in range(300):
        k = rng.standard_normal((int(rng.integers(1, 17)), 8)) * np.exp(rng.uniform(-40, 40))
        codes, s = key_range(k)
        e = np.log2(s)
        assert e == round(e) and np.abs(codes).max() <= 127 and np.abs(k).max() > 127 * s / 2
        assert np.all(codes[0] * s <= k.min(0)) and np.all(k.min(0) < (codes[0] + 1) * s)
        assert np.all(codes[1] * s >= k.max(0)) and np.all(k.max(0) > (codes[1] - 1) * s)
    assert key_range([[127.0, -1.0]])[1] == 1.0 and key_range([[127.5, 0.0]])[1] == 2.0 and key_range([[63.5, 0.0]])[1] == 0.5
    codes, s = key_range([[1e-40, -1e-40, 0.0]])
    assert s == 2.0 ** -100 and codes.tolist() == [[0, -1, 0], [1, 0, 0]]
    assert key_range([[0.0, -0.0]])[1] == 0.0 and key_range([[np.inf, 0.0]])[1] == np.inf and key_range([[0, np.nan]])[1] == np.inf


def test_scores_bound_the_keys_scores():
    rng = np.random.default_rng(1)
    for _ in range(100):
        q, k = rng.standard_normal((int(rng.integers(1, 9)), 16)).astype(np.float32), rng.standard_normal((5, 16))
        codes, s = key_range(k)
        u = rounded_queries(q)
        assert 512 <= np.abs(u).max() <= 1024
        got = scores(q, codes[None], np.array([s]))[0]
        assert np.all((u @ k.T).sum(0) <= got * (1 + 2.0 ** -24) + 1e-9)
    k = np.array([[3.0, -5.0, 0.0, 127.0]])                       # on the grid: the bound is the score
    codes, s = key_range(k)
    q = np.array([[1.0, 0.5, -0.25, 0.125]])
    assert scores(q, codes[None], np.array([s]))[0] == 512 * 3 - 256 * 5 + 64 * 127
    assert scores(q * 0, codes[None], np.array([s]))[0] == 0 and scores(q * np.nan, codes[None], np.array([s]))[0] == 0
    assert scores(q, codes[None], np.array([np.inf]))[0] == np.inf


def test_select_is_the_best_subset():
    rng = np.random.default_rng(2)
    for _ in range(200):
        held, first, last = int(rng.integers(1, 8)), int(rng.integers(0, 2)), int(rng.integers(1, 3))
        k = first + last + int(rng.integers(0, 4))
        s = rng.integers(-3, 4, held).astype(float)
        kept = {j for j in range(held) if j < first or j >= held - last}
        best = max(s[list(c)].sum() for c in itertools.combinations(range(held), min(k, held)) if kept <= set(c))
        got = select(s, first, last, k)
        assert kept <= set(got) and got == sorted(set(got)) and len(got) == min(k, held) and s[got].sum() == best
        for j in range(held):                                     # of equal scores the earlier
            if j not in got:
                assert all(s[i] > s[j] or (s[i] == s[j] and i < j) for i in got if i not in kept)


def test_attention_over_all_blocks_is_attention():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 6, 2, 16, 8))
    bt = np.array([[3, 0, 5], [1, 2, 4]])
    q, seq, pos = rng.standard_normal((3, 4, 8)), [1, 0, -1], np.array([40, 17, 3])
    sel = [[[0, 1, 2], [2, -1, 0, 1]], [[0, 1, 2], [0, 1, -1]], [[0], [0]]]
    got, most = attention(q, k, v, bt, seq, pos, sel)
    assert np.allclose(got, rows_attention(q, k, v, bt, seq, pos), rtol=0, atol=1e-14)
    assert not got[2].any() and most.shape == got.shape and not most[2].any()
    one, _ = attention(q[:1], k, v, bt, seq[:1], pos[:1], [[[1], [2]]])
    w = np.exp(k[4, 1, :9] @ q[0, 3] / np.sqrt(8))
    assert np.allclose(one.reshape(4, 8)[3], w / w.sum() @ v[4, 1, :9])


# ---------------------------------------------------------------------------
# refusals before any device call (the pointers are never followed)

@pytest.fixture(scope="module")
def lib():
    build.build()
    capi._lib = None
    return capi.load()


P = ctypes.c_void_p(1 << 20)                   # a 16-byte aligned address
ODD = ctypes.c_void_p((1 << 20) + 4)
EXTEND = dict(nseq=4, ctx=P, new=P, bt=P, bt_stride=3, num_blocks=5, free=P, nfree=4, free_at=P, n=8, held=P, cu=P,
              positions=P, row_seq=P, slots=P, free_next=P, err=None, stream=None)
BOUNDS = dict(n=4, positions=P, row_seq=None, nseq=4, bt=P, bt_stride=3, nkv=2, d=64, kpool=P, kv_dtype=0, num_blocks=5,
              bounds=P, scales=P, err=None, stream=None)
SELECT = dict(n=4, q=P, nq=8, nkv=2, d=64, bounds=P, scales=P, positions=P, row_seq=None, nseq=4, bt=P, bt_stride=3,
              num_blocks=5, keep_first=1, keep_last=1, k=2, sel=P, scratch=None, scratch_bytes=0, err=None, stream=None)
ATTEND = dict(n=4, q=P, nq=8, nkv=2, d=64, kpool=P, vpool=P, kv_dtype=0, k_scale=1.0, v_scale=1.0, positions=P,
              row_seq=None, nseq=4, bt=P, bt_stride=3, sel=P, k=2, num_blocks=5, out=P, err=None, stream=None)
BAD = {
    "op_kv_extend": (EXTEND, [
        ("nseq", 0), ("nseq", -3), ("nseq", 2 ** 31 - 1), ("n", 2 ** 30 + 1), ("ctx", None), ("new", None), ("bt", None), ("bt_stride", 0),
        ("bt_stride", (1 << 26) + 1), ("num_blocks", 0), ("free", None), ("nfree", -1), ("free_at", None), ("n", 0),
        ("held", None), ("cu", None), ("positions", None), ("row_seq", None), ("slots", None), ("free_next", None)]),
    "op_key_bounds": (BOUNDS, [
        ("n", 0), ("positions", None), ("nseq", 0), ("nseq", 3), ("bt", None), ("bt_stride", 0), ("bt_stride", (1 << 26) + 1),
        ("nkv", 0), ("nkv", (1 << 16) + 1), ("d", 32), ("d", 96), ("kpool", None), ("kpool", ODD), ("kv_dtype", 2), ("kv_dtype", 4),
        ("kv_dtype", -1), ("num_blocks", 0), ("bounds", None), ("bounds", ODD), ("scales", None)]),
    "op_block_select": (SELECT, [
        ("n", 0), ("q", None), ("q", ODD), ("nq", 0), ("nq", 7), ("nq", 34), ("nkv", 0), ("d", 80), ("bounds", None),
        ("bounds", ODD), ("scales", None), ("positions", None), ("nseq", 0), ("nseq", 3), ("bt", None), ("bt_stride", 0),
        ("num_blocks", 0), ("keep_first", -1), ("keep_last", 0), ("k", 1), ("k", 0), ("keep_first", 2 ** 31 - 1), ("k", (1 << 26) + 1),
        ("sel", None), ("scratch", ODD), ("bt_stride", (1 << 26) + 1)]),
    "op_block_attention": (ATTEND, [
        ("n", 0), ("q", None), ("q", ODD), ("nq", 0), ("nq", 7), ("nq", 34), ("nkv", 0), ("d", 256), ("kpool", None),
        ("kpool", ODD), ("vpool", None), ("vpool", ODD), ("kv_dtype", 2), ("kv_dtype", 4), ("k_scale", 0.0),
        ("k_scale", 2.0 ** -65), ("v_scale", float("nan")), ("v_scale", 2.0 ** 65), ("positions", None), ("nseq", 0),
        ("nseq", 3), ("bt", None), ("bt_stride", 0), ("bt_stride", (1 << 26) + 1), ("sel", None), ("k", 0), ("k", (1 << 26) + 1),
        ("num_blocks", 0), ("out", None), ("out", ODD)]),
}


@pytest.mark.parametrize("fn,name,value", [(f, n, v) for f, (_, bad) in BAD.items() for n, v in bad],
                         ids=lambda x: str(getattr(x, "value", x)))
def test_refused_arguments(lib, fn, name, value):
    args = dict(BAD[fn][0])
    assert name in args
    args[name] = value
    assert getattr(lib, fn)(*args.values()) == -1


def test_binding_refuses_host_tensors_and_wide_numbers(lib):
    i = torch.zeros((4, 1), dtype=torch.int32)
    q, one, slots = torch.zeros((4, 4, 64)), i[:1, 0].contiguous(), torch.zeros(4, dtype=torch.int64)
    p, codes, sc = torch.zeros(6 * 2 * 576, dtype=torch.uint8), torch.zeros((6, 2, 2, 64), dtype=torch.int8), torch.zeros((6, 2))
    sel, pos = torch.zeros((4, 2, 3), dtype=torch.int32), i[:, 0].contiguous()
    with pytest.raises(ValueError):
        capi.op_kv_extend(pos, pos, i, 5, pos, one, pos, torch.zeros(5, dtype=torch.int32), pos, pos, slots, one)
    with pytest.raises(ValueError):
        capi.op_key_bounds(pos, i, p, 2, 64, 3, 5, codes, sc)
    with pytest.raises(ValueError):
        capi.op_block_select(q, 2, codes, sc, pos, i, 5, 1, 1, sel)
    with pytest.raises(ValueError):
        capi.op_block_attention(q, 2, p, p, 3, 1.0, 1.0, pos, i, sel, 5, q.view(4, 256))
