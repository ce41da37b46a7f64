"""The 4-bit cache oracle pinned on its definition, and the host-side refusals
of the 4-bit and prompt-attention entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import build, capi
from oracle.kv_fp4 import (E2M1_VALUES, decode, encode, pack_pool, prompt_positions, round_e2m1, rows_attention,
                           unit_bytes, unpack_pool)
from oracle.numerics import E4M3_VALUES


def test_e2m1_grid_and_ties():
    assert E2M1_VALUES[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert round_e2m1(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 100.0])).tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert round_e2m1(np.array([0.2501, 0.7499, -1.2501, -5.001, -0.1])).tolist() == [1, 1, 11, 15, 8]
    assert np.array_equal(round_e2m1(E2M1_VALUES), np.r_[0:16].astype(np.uint8))


def test_encode_is_nearest_within_its_scale():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 64)) * np.exp(rng.uniform(-3, 3, (7, 1)))
    codes, sc = encode(x, 0.7)
    u = E4M3_VALUES[sc].repeat(16, -1) * 0.7
    best = np.abs(E2M1_VALUES * u[..., None] - x[..., None]).min(-1)
    assert np.allclose(np.abs(decode(codes, sc, 0.7) - x), best, rtol=0, atol=1e-12)
    # the scale puts the group's largest magnitude within an e4m3 half step (2^-4) of 6
    m = np.abs(x).reshape(7, 4, 16).max(-1)
    assert np.all(np.abs(m / (E4M3_VALUES[sc] * 0.7) / 6 - 1) <= 2.0 ** -4 / (1 - 2.0 ** -4))


def test_encode_edges():
    x = np.zeros((5, 16))
    x[1, 3] = np.nan
    x[2, :2] = [np.inf, 5.0]
    x[3, 0] = 2.0 ** -13                       # below half the smallest scale
    x[4] = 1e6                                 # beyond the largest scale: 448 * 6
    codes, sc = encode(x, 1.0)
    assert sc[:, 0].tolist() == [0, 0x7F, 0x7E, 0, 0x7E]
    assert not codes[0].any() and not codes[3].any()
    assert codes[2, 0] == 7 and codes[2, 1] == 0 and np.all(codes[4] == 7)
    assert np.isnan(decode(codes, sc, 1.0)[1]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_pool_layout_round_trips(d):
    rng = np.random.default_rng(d)
    codes = rng.integers(0, 16, (3, 2, 16, d)).astype(np.uint8)
    sc = rng.integers(0, 0x7F, (3, 2, 16, d // 16)).astype(np.uint8)
    pool = pack_pool(codes, sc)
    assert pool.shape == (3, 2, unit_bytes(d)) and unit_bytes(d) == 9 * d
    assert pool[1, 1, 5 * d // 2 + 3] == codes[1, 1, 5, 6] | (codes[1, 1, 5, 7] << 4)
    assert pool[2, 0, 8 * d + 4 * (d // 16) + 1] == sc[2, 0, 4, 1]
    c2, s2 = unpack_pool(pool, d)
    assert np.array_equal(c2, codes) and np.array_equal(s2, sc)


def test_rows_attention_is_softmax_over_the_causal_prefix():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 4, 1, 16, 8))
    bt = np.array([[2, 0, -1]])
    seq, pos = prompt_positions([0, 3], [18], 4)
    assert seq.tolist() == [0, 0, 0, -1] and pos.tolist() == [15, 16, 17, -1]
    q = rng.standard_normal((4, 2, 8))
    got = rows_attention(q, k, v, bt, seq, pos).reshape(4, 2, 8)
    ks, vs = np.concatenate([k[2, 0], k[0, 0]]), np.concatenate([v[2, 0], v[0, 0]])
    w = np.exp(ks[:17] @ q[1, 1] / np.sqrt(8))
    assert np.allclose(got[1, 1], (w[:, None] * vs[:17]).sum(0) / w.sum())
    assert not got[3].any()


# ---------------------------------------------------------------------------
# refusals before any device call (the pointers are never followed)

@pytest.fixture(scope="module")
def lib():
    build.build()
    capi._lib = None
    return capi.load()


P = ctypes.c_void_p(1 << 20)                   # a 16-byte aligned address
ODD = ctypes.c_void_p((1 << 20) + 4)
WRITE = dict(n=4, qkv=P, ld=768, nq=8, nkv=2, d=64, positions=P, row_seq=None, nseq=4, bt=P, bt_stride=3, rope=P,
             max_pos=64, kpool=P, vpool=P, num_blocks=5, k_scale=1.0, v_scale=1.0, q_out=P, err=None, stream=None)
READ = dict(n=4, positions=P, row_seq=None, nseq=4, bt=P, bt_stride=3, nkv=2, d=64, kpool=P, vpool=P, num_blocks=5,
            k_scale=1.0, v_scale=1.0, k_out=P, v_out=P, err=None, stream=None)
DECODE = dict(B=4, q=P, nq=8, nkv=2, d=64, kpool=P, vpool=P, k_scale=1.0, v_scale=1.0, bt=P, bt_stride=3, seq_lens=P,
              num_blocks=5, out=P, err=None, stream=None)
PROMPT = dict(n=4, q=P, nq=8, nkv=2, d=64, nseq=2, cu=P, ctx=P, kpool=P, vpool=P, kv_dtype=3, k_scale=1.0, v_scale=1.0,
              bt=P, bt_stride=3, num_blocks=5, out=P, err=None, stream=None)
BAD = {
    "op_rope_kv_write_fp4": (WRITE, [
        ("n", 0), ("n", -1), ("qkv", None), ("qkv", ODD), ("ld", 767), ("ld", 764), ("nq", 0), ("nkv", 0), ("d", 32),
        ("d", 96), ("positions", None), ("nseq", 0), ("nseq", 3), ("bt", None), ("bt_stride", 0), ("rope", None),
        ("rope", ODD), ("max_pos", 0), ("kpool", None), ("kpool", ODD), ("vpool", None), ("vpool", ODD),
        ("num_blocks", 0), ("k_scale", 0.0), ("k_scale", -1.0), ("k_scale", float("nan")), ("v_scale", float("inf")),
        ("q_out", None), ("q_out", ODD)]),
    "op_kv_read_fp4": (READ, [
        ("n", 0), ("positions", None), ("nseq", 0), ("nseq", 3), ("bt", None), ("bt_stride", 0), ("nkv", 0), ("d", 16),
        ("kpool", None), ("kpool", ODD), ("vpool", None), ("vpool", ODD), ("num_blocks", 0), ("k_scale", 0.0),
        ("v_scale", float("nan")), ("k_out", None), ("k_out", ODD), ("v_out", None), ("v_out", ODD)]),
    "op_paged_attention_fp4": (DECODE, [
        ("B", 0), ("q", None), ("q", ODD), ("nq", 0), ("nq", 7), ("nq", 34), ("nkv", 0), ("d", 256), ("kpool", None),
        ("kpool", ODD), ("vpool", None), ("vpool", ODD), ("k_scale", 0.0), ("v_scale", float("inf")), ("bt", None),
        ("bt_stride", 0), ("seq_lens", None), ("num_blocks", 0), ("out", None), ("out", ODD)]),
    "op_prompt_attention": (PROMPT, [
        ("n", 0), ("q", None), ("q", ODD), ("nq", 0), ("nq", 7), ("nq", 34), ("nkv", 0), ("d", 80), ("nseq", 0),
        ("cu", None), ("ctx", None), ("kpool", None), ("kpool", ODD), ("vpool", None), ("vpool", ODD), ("kv_dtype", 2),
        ("kv_dtype", 4), ("kv_dtype", -1), ("k_scale", float("nan")), ("v_scale", 0.0), ("bt", None), ("bt_stride", 0),
        ("num_blocks", 0), ("out", None), ("out", ODD)]),
}


@pytest.mark.parametrize("fn,name,value", [(f, n, v) for f, (_, bad) in BAD.items() for n, v in bad],
                         ids=lambda x: str(getattr(x, "value", x)))
def test_refused_arguments(lib, fn, name, value):
    args = dict(BAD[fn][0])
    assert name in args
    args[name] = value
    assert getattr(lib, fn)(*args.values()) == -1


def test_unit_bytes_and_rope_table_refusals(lib):
    u = capi.op_kv_unit_bytes
    assert [u(128, k) for k in (0, 1, 2, 3, 4)] == [4096, 2048, 0, 1152, 0]
    assert [u(64, k) for k in (0, 1, 3)] == [2048, 1024, 576] and u(32, 3) == 0
    assert lib.op_rope_table(0, 64, 1e4, P, None) == -1
    assert lib.op_rope_table(4, 63, 1e4, P, None) == -1
    assert lib.op_rope_table(4, 64, 1.0, P, None) == -1
    assert lib.op_rope_table(4, 64, 1e4, None, None) == -1


def test_binding_refuses_host_tensors(lib):
    z = torch.zeros((4, 2, 64))
    i = torch.zeros((4, 1), dtype=torch.int32)
    p = torch.zeros(6 * 2 * 576, dtype=torch.uint8)
    with pytest.raises(ValueError):
        capi.op_paged_attention_fp4(z, 2, p, p, 1.0, 1.0, i, i[:, 0].contiguous(), 5, z.view(4, 128))
    with pytest.raises(ValueError):
        capi.op_prompt_attention(z, 2, i[:, 0].contiguous(), i[:3, 0].contiguous(), p, p, 3, 1.0, 1.0, i, 5, z.view(4, 128))
    with pytest.raises(ValueError):
        capi.op_kv_read_fp4(i[:, 0].contiguous(), i, p, p, 2, 64, 5, 1.0, 1.0, z, z)
    with pytest.raises(ValueError):
        capi.op_rope_kv_write_fp4(torch.zeros((4, 384)), 2, 2, 64, i[:, 0].contiguous(), i, z, p, p, 5, 1.0, 1.0, z)


@pytest.mark.parametrize("fn", list(BAD))
@pytest.mark.parametrize("name,value", [("k_scale", 2.0 ** -65), ("v_scale", 2.0 ** 65), ("bt_stride", (1 << 26) + 1)])
def test_limits_of_scales_and_tables(lib, fn, name, value):
    assert getattr(lib, fn)(*dict(BAD[fn][0], **{name: value}).values()) == -1
