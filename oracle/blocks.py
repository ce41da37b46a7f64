"""Attention over selected blocks of the paged cache and what prepares it, as
their plain definitions in float64 and Python integers.

Test infrastructure only (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["BLOCK", "BLOCKS", "POS", "SEQLEN", "extend", "key_range", "rounded_queries", "scores", "select", "attention"]

BLOCK = 16
BLOCKS, POS, SEQLEN = 2, 4, 8                  # error bits: blocks, rows or positions, lengths


def extend(ctx, new, bt, num_blocks, free, at, n):
    """Sequences one after another. Returns (dict of outputs, error bits); bt is copied."""
    bt, bits, width = np.array(bt), 0, bt.shape[1]
    at_ok = 0 <= at <= len(free)
    bits |= 0 if at_ok else BLOCKS
    asked, want, taken, held, cu, rows = 0, at, at, [], [0], []
    for s, (c, k) in enumerate(zip(map(int, ctx), map(int, new))):
        ok = c >= 0 and k >= 0 and c + k <= width * BLOCK
        if not ok:
            bits |= SEQLEN
            k = 0
        first = -(-c // BLOCK)
        need = -(-(c + k) // BLOCK) - first if k else 0
        asked, want = asked + k, want + need
        if k and asked > n:
            bits |= POS
            k = need = 0
        elif need and (not at_ok or want > len(free)):
            bits |= BLOCKS
            k = need = 0
        for j in range(need):
            bt[s, first + j] = free[want - need + j]
            if not 0 <= bt[s, first + j] <= num_blocks:
                bits |= BLOCKS
        taken += need
        held.append(c + k)
        cu.append(cu[-1] + k)
        for p in range(c, c + k):
            b = int(bt[s, p // BLOCK])
            good = 0 <= b <= num_blocks
            bits |= 0 if good else BLOCKS
            rows.append((p, s, b * BLOCK + p % BLOCK if good else -1))
    rows += [(0, len(held), num_blocks * BLOCK)] * (n - len(rows))
    p, s, slot = (np.array(x, dtype=np.int64) for x in zip(*rows))
    return dict(bt=bt, held=np.array(held), cu=np.array(cu), positions=p, row_seq=s, slots=slot, free_next=taken), bits


def key_range(k):
    """Keys [tokens][d] -> (codes [2][d], scale)."""
    k = np.asarray(k, dtype=np.float64)
    codes = np.zeros((2, k.shape[1]), dtype=np.int64)
    if not np.isfinite(k).all():
        return codes, math.inf
    most = np.abs(k).max()
    if most == 0:
        return codes, 0.0
    e = -100
    while most > 127 * 2.0 ** e:
        e += 1
    return np.stack((np.floor(k.min(0) / 2.0 ** e), np.ceil(k.max(0) / 2.0 ** e))).astype(np.int64), 2.0 ** e


def rounded_queries(q):
    """[G][d] -> integers."""
    q = np.asarray(q, dtype=np.float64)
    most = np.abs(q).max()
    if most == 0 or not np.isfinite(q).all():
        return np.zeros(q.shape, dtype=np.int64)
    return np.rint(q * 2.0 ** (10 - math.frexp(most)[1])).astype(np.int64)


def scores(q, codes, scale):
    """Queries [G][d] of a KV head, codes [blocks][2][d], scale [blocks] -> fp32 scores as float64."""
    u = rounded_queries(q)
    p, m = np.maximum(u, 0).sum(0), np.minimum(u, 0).sum(0)
    codes = np.asarray(codes, dtype=np.int64)
    with np.errstate(over="ignore", invalid="ignore"):
        s = (codes[:, 1] @ p + codes[:, 0] @ m).astype(np.float32) * np.asarray(scale, dtype=np.float32)
    return np.where(np.isfinite(scale), s, np.inf).astype(np.float64)


def select(score, first, last, k):
    """Ascending places of the k chosen blocks (fewer if there are fewer)."""
    held = len(score)
    order = sorted(range(held), key=lambda j: (not (j < first or j >= held - last), -score[j], j))
    return sorted(order[:k])


def attention(q, k, v, bt, seq, pos, sel):
    """q [n][nq][d]; k, v [blocks][nkv][16][d]; row i attends over tokens <= pos[i] of blocks sel[i][kv head] (negative
    entries skipped) of sequence seq[i] (none where seq[i] < 0). Returns [n][nq * d] and the largest |V| it may reach."""
    n, nq, d = q.shape
    nkv = k.shape[1]
    out, most = np.zeros((n, nq, d)), np.zeros((n, nq, 1))
    for i in range(n):
        if seq[i] < 0:
            continue
        for h in range(nkv):
            ks, vs = [np.zeros((0, d))], [np.zeros((0, d))]
            for j in sel[i][h]:
                if 0 <= j <= pos[i] // BLOCK:
                    t = min(BLOCK, int(pos[i]) - int(j) * BLOCK + 1)
                    ks.append(k[bt[seq[i], j], h, :t])
                    vs.append(v[bt[seq[i], j], h, :t])
            ks, vs = np.concatenate(ks), np.concatenate(vs)
            if not len(ks):
                continue
            g = slice(h * (nq // nkv), (h + 1) * (nq // nkv))
            w = q[i, g].astype(np.float64) @ ks.T / math.sqrt(d)
            w = np.exp(w - w.max(-1, keepdims=True))
            out[i, g] = w / w.sum(-1, keepdims=True) @ vs
            most[i, g] = np.abs(vs).max()
    return out.reshape(n, nq * d), np.broadcast_to(most, (n, nq, d)).reshape(n, nq * d)
