"""The 4-bit paged KV cache and prompt attention, as their plain definitions in
float64.

Test infrastructure only (see the package docstring).

Format: value = e2m1(code) * e4m3(scale) * g with one 4-bit code per value (sign,
two exponent bits with bias 1, one mantissa bit), one e4m3 scale per 16
neighbouring channels of a token's head and the tensor's scale g. A pool is
[num_blocks + 1][n_kv_heads][unit]: per (block, KV head) the codes of 16 tokens
[16][d / 2] (channel 2j in the low half of byte j), then their scales
[16][d / 16].
"""
from __future__ import annotations

import numpy as np

from .numerics import E4M3_VALUES, bf16_decode, e4m3_decode, round_e4m3

__all__ = ["E2M1_VALUES", "GROUP", "BLOCK", "round_e2m1", "encode", "decode", "unit_bytes", "pack_pool", "unpack_pool",
           "pool_values", "rows_attention", "prompt_positions"]

GROUP, BLOCK = 16, 16


def _e2m1_table() -> np.ndarray:
    v = np.empty(16)
    for code in range(16):
        e, m = (code >> 1) & 3, code & 1
        mag = m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)
        v[code] = -mag if code & 8 else mag
    return v


E2M1_VALUES = _e2m1_table()
_POS = E2M1_VALUES[:8]


def round_e2m1(x: np.ndarray) -> np.ndarray:
    """float64 -> e2m1 codes, nearest (a tie goes to the even code), saturating at +-6."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), 6.0)
    d = np.abs(mag[..., None] - _POS)
    near = d == d.min(-1, keepdims=True)
    # among one or two equally near codes the even one
    code = np.where(near.sum(-1) > 1, (near * (np.arange(8) % 2 == 0)).argmax(-1), near.argmax(-1))
    return (code | (np.signbit(x) * 8)).astype(np.uint8)


def encode(x: np.ndarray, g: float):
    """x [..., d] float64 -> (codes [..., d], scale codes [..., d / 16])."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, GROUP)
    nan = np.isnan(b).any(-1)
    m = np.abs(np.where(np.isnan(b), 0.0, b)).max(-1)
    sc = round_e4m3(np.minimum(m / (6.0 * g), 448.0))
    sc = np.where(nan, 0x7F, sc).astype(np.uint8)
    u = np.where(nan, 0.0, e4m3_decode(np.where(nan, 0, sc)))[..., None] * g
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(u > 0, np.clip(b / u, -8.0, 8.0), 0.0)
    return round_e2m1(r).reshape(x.shape), sc


def decode(codes: np.ndarray, scales: np.ndarray, g: float) -> np.ndarray:
    v = E2M1_VALUES[codes].reshape(*codes.shape[:-1], -1, GROUP) * E4M3_VALUES[scales][..., None]
    return v.reshape(codes.shape) * g


def unit_bytes(d: int) -> int:
    return BLOCK * (d // 2 + d // GROUP)


def pack_pool(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [blocks, nkv, 16, d], scales [blocks, nkv, 16, d / 16] -> [blocks, nkv, unit] bytes."""
    n, h = codes.shape[:2]
    return np.concatenate(((codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(n, h, -1), scales.reshape(n, h, -1)), -1)


def unpack_pool(pool: np.ndarray, d: int):
    n, h = pool.shape[:2]
    raw = pool[..., :BLOCK * d // 2].reshape(n, h, BLOCK, d // 2)
    codes = np.stack((raw & 15, raw >> 4), -1).reshape(n, h, BLOCK, d)
    return codes, pool[..., BLOCK * d // 2:].reshape(n, h, BLOCK, d // GROUP)


def pool_values(pool: np.ndarray, kind: str, d: int, g: float) -> np.ndarray:
    """Raw pool -> float64 values [blocks, nkv, 16, d]; kind "bf16" (uint16 bits), "fp8" (e4m3 codes) or "fp4"."""
    if kind == "fp4":
        return decode(*unpack_pool(pool, d), g)
    return (bf16_decode(pool) if kind == "bf16" else e4m3_decode(pool)) * g


def prompt_positions(cu, ctx, n: int):
    """(sequence, position) of each of n packed rows; sequence -1 for rows of none."""
    seq, pos = np.full(n, -1), np.full(n, -1)
    for s in range(len(ctx)):
        k = int(cu[s + 1]) - int(cu[s])
        seq[cu[s]:cu[s + 1]] = s
        pos[cu[s]:cu[s + 1]] = int(ctx[s]) - k + np.arange(k)
    return seq, pos


def rows_attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, bt: np.ndarray, seq, last) -> np.ndarray:
    """q [n][nq][d]; k, v [blocks][nkv][16][d] values; row i attends over tokens 0..last[i] of sequence seq[i] (none
    when last[i] < 0: zeros). Only the attended tokens are touched. Returns [n][nq * d]."""
    n, nq, d = q.shape
    nkv = k.shape[1]
    out = np.zeros((n, nq, d))
    for s in set(int(x) for x in seq):
        rows = np.flatnonzero((np.asarray(seq) == s) & (np.asarray(last) >= 0))
        if s < 0 or not len(rows):
            continue
        most = int(np.max(np.asarray(last)[rows])) + 1
        ids = bt[s, :-(-most // BLOCK)]
        ks = k[ids].transpose(1, 0, 2, 3).reshape(nkv, -1, d)
        vs = v[ids].transpose(1, 0, 2, 3).reshape(nkv, -1, d)
        for i in rows:
            t = int(last[i]) + 1
            for h in range(nq):
                g = h // (nq // nkv)
                w = ks[g, :t] @ q[i, h].astype(np.float64) / np.sqrt(d)
                w = np.exp(w - w.max())
                out[i, h] = (w / w.sum()) @ vs[g, :t]
    return out.reshape(n, nq * d)
