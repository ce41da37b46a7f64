"""Attention over selected blocks of the paged KV cache and what prepares it, as timed cases with their plain forms.

Four operators, called one after another in a serving step:

* extend: sequences get blocks from a free list for their new tokens; the packed rows' sequences, positions and
  slots are laid out (op_kv_extend);
* bounds: each block's keys are summed up, per KV head, by a range per channel: two 8-bit codes and a power of two
  (op_key_bounds; BF16, e4m3 and 4-bit caches);
* select: every query takes, per KV head, the blocks of its context whose ranges allow the largest scores
  (op_block_select);
* attend: softmax attention over the selected blocks alone (op_block_attention; the same three caches).

A cache block holds 16 tokens. Values of the 4-bit cache are e2m1 * e4m3 * g: per (block, KV head) the codes of 16
tokens [16][d / 2] (channel 2j in the low half of byte j), then their scales [16][d / 16].

Ranges: with M the largest magnitude among a block's keys of a KV head (in the cache's units, before the tensor's
scale), e is the smallest exponent >= -100 with M <= 127 * 2^e, and channel i has low_i = floor(min k_i / 2^e) and
high_i = ceil(max k_i / 2^e); scale = 2^e (0 where M = 0, +inf and all codes 0 where a key is not finite).

Scores: the queries of a KV head's group are rounded to integers u = rint(q * 2^(10 - x)), 2^x being the smallest power
of two above their largest magnitude (all 0 where one is not finite); with P_i the sum of the group's positive u of
channel i and N_i that of the negative ones, score = fp32(sum_i P_i high_i + N_i low_i) * scale, or +inf where the
scale is. The first keep_first and last keep_last blocks of a context are always taken, then the largest scores up to
k blocks in all; of equal scores the earlier block."""
import math

import numpy as np
import torch

own = False

BLOCK = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
K_SCALE, V_SCALE = 0.875, 1.25
CHUNK = 1 << 27                     # values a plain form works on at a time


def listed():
    return [
        # one decode step of the 8B-class batch: 64 sequences grow by a token each (latency)
        dict(name="extend 64 by one", op="extend", seqs=64, ctx_lo=256, ctx_hi=2048, new_lo=1, new_hi=1),
        # a large mixed step: prompts of all lengths behind prefixes of all lengths, some sequences without rows
        dict(name="extend 512 ragged", op="extend", seqs=512, ctx_lo=0, ctx_hi=8192, new_lo=0, new_hi=255),
        # the blocks that a decode step of 64 sequences has written to (latency)
        dict(name="bounds 8b 64 rows bf16", op="bounds", kv="bf16", seqs=64, ctx_lo=256, ctx_hi=2048, new_lo=1,
             new_hi=1, nkv=8, d=128),
        # four packed prompts of about 1000 tokens, the 70B-class cache
        dict(name="bounds 70b prompts e4m3", op="bounds", kv="e4m3", seqs=4, ctx_lo=0, ctx_hi=900, new_lo=1000,
             new_hi=1043, nkv=8, d=128),
        # all of a long prompt at once, 1B-class heads of 64 channels, 4-bit cache
        dict(name="bounds 1b 50k fp4", op="bounds", kv="fp4", seqs=1, ctx_lo=0, ctx_hi=0, new_lo=50021, new_hi=50021,
             nkv=8, d=64),
        # a single sequence being decoded over a long context (latency)
        dict(name="select 8b one of 32k", op="select", seqs=1, rows=1, ctx_lo=32765, ctx_hi=32765, nq=32, nkv=8, d=128,
             k=64, first=1, last=2),
        # a decode batch over long ragged contexts
        dict(name="select 70b 64 of 32k", op="select", seqs=64, rows=1, ctx_lo=16001, ctx_hi=32765, nq=64, nkv=8, d=128,
             k=128, first=1, last=4),
        # two sequences of a million tokens
        dict(name="select 8b 2 of 1M", op="select", seqs=2, rows=1, ctx_lo=999000, ctx_hi=1000003, nq=32, nkv=8, d=128,
             k=256, first=1, last=8),
        # a single sequence being decoded (latency)
        dict(name="attend 8b one bf16", op="attend", kv="bf16", seqs=1, rows=1, ctx_lo=32765, ctx_hi=32765, nq=32, nkv=8,
             d=128, k=64),
        # the 8B-class decode batch over contexts of up to 8k
        dict(name="attend 8b 64 bf16", op="attend", kv="bf16", seqs=64, rows=1, ctx_lo=4001, ctx_hi=8189, nq=32, nkv=8,
             d=128, k=64),
        # the 70B-class decode batch, twice as many blocks
        dict(name="attend 70b 64 e4m3", op="attend", kv="e4m3", seqs=64, rows=1, ctx_lo=4001, ctx_hi=8189, nq=64, nkv=8,
             d=128, k=128),
        # pieces of prompts, every row with blocks of its own, 1B-class heads, 4-bit cache
        dict(name="attend 1b pieces fp4", op="attend", kv="fp4", seqs=3, rows=170, ctx_lo=9001, ctx_hi=16381, nq=32,
             nkv=8, d=64, k=48),
    ]


HEADS = ((32, 8, 64), (32, 8, 128), (40, 8, 128), (64, 8, 128), (4, 2, 64), (8, 8, 128), (16, 1, 128))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("extend", "bounds", "select", "attend"))
    nq, nkv, d = rng.choice(HEADS)
    if op == "extend":
        seqs = _log(rng, 1, 512)
        new = _log(rng, 1, 65536 // seqs)
        return dict(op=op, seqs=seqs, ctx_lo=0, ctx_hi=_log(rng, 1, 16384), new_lo=rng.choice((0, 1, new)), new_hi=new)
    kv = rng.choice(("bf16", "e4m3", "fp4"))
    if op == "bounds":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, 16384 // seqs)
        return dict(op=op, kv=kv, seqs=seqs, ctx_lo=0, ctx_hi=_log(rng, 1, 4096), new_lo=rng.randint(1, new), new_hi=new,
                    nkv=nkv, d=d)
    seqs = _log(rng, 1, 64)
    rows = 1 if rng.random() < 0.6 else _log(rng, 2, max(2, 256 // seqs))
    if op == "select":
        hi = _log(rng, rows, max(rows, min(1000000, 1500000 // (seqs * rows))))
        k = _log(rng, 1, 256)
        first = rng.randint(0, min(4, k - 1))
        return dict(op=op, seqs=seqs, rows=rows, ctx_lo=rng.randint(rows, hi), ctx_hi=hi, nq=nq, nkv=nkv, d=d, k=k,
                    first=first, last=rng.randint(1, min(8, k - first)))
    hi = _log(rng, rows, max(rows, min(65536, 500000 // seqs)))
    return dict(op=op, kv=kv, seqs=seqs, rows=rows, ctx_lo=rng.randint(rows, hi), ctx_hi=hi, nq=nq, nkv=nkv, d=d,
                k=_log(rng, 1, max(1, min(256, 8000 // (seqs * rows)))))


# ---------------------------------------------------------------------------
# sizes

def _spread(c, what, salt):
    """One number per sequence in [lo, hi], in a fixed scattered order."""
    lo, span = c[what + "_lo"], c[what + "_hi"] - c[what + "_lo"] + 1
    return [lo + ((i + salt) * 2654435761 + span // 2) % span for i in range(c["seqs"])]


def _blocks(tokens):
    return -(-tokens // BLOCK)


def _key_bytes(kv, d):
    return {"bf16": 2 * d, "e4m3": d, "fp4": d // 2 + d // 16}[kv]


def _rows(c):
    """(sequence, position) of the rows: each sequence's last ones. Sequences of an extend or bounds case grow from
    ctx by new tokens; those of the others hold ctx tokens, of which `rows` are queries."""
    ctx = _spread(c, "ctx", 0)
    if c["op"] in ("extend", "bounds"):
        return [(s, p) for s, (a, k) in enumerate(zip(ctx, _spread(c, "new", 7))) for p in range(a, a + k)]
    return [(s, p) for s, a in enumerate(ctx) for p in range(a - c["rows"], a)]


def work(case):
    c = case
    if c["op"] == "extend":
        ctx, new = _spread(c, "ctx", 0), _spread(c, "new", 7)
        took = sum(_blocks(a + k) - _blocks(a) for a, k in zip(ctx, new))
        n = sum(new)
        return {"bytes": 8 * c["seqs"] + 8 * c["seqs"] + 4 + 8 * took + 16 * n, "flops": 8 * c["seqs"] + 8 * n}
    nkv, d = c["nkv"], c["d"]
    if c["op"] == "bounds":
        bytes_, flops = 0, 0
        for a, k in zip(_spread(c, "ctx", 0), _spread(c, "new", 7)):
            tokens = a + k - a // BLOCK * BLOCK if k else 0
            bytes_ += 8 * k + tokens * nkv * _key_bytes(c["kv"], d) + _blocks(tokens) * (4 + nkv * (2 * d + 4))
            flops += 2 * tokens * nkv * d
        return {"bytes": bytes_, "flops": flops}
    rows = _rows(c)
    n, nq, k = len(rows), c["nq"], c["k"]
    if c["op"] == "select":
        seen = [p // BLOCK + 1 for _, p in rows]
        held = sum(_blocks(a) for a in _spread(c, "ctx", 0))
        return {"bytes": held * (4 + nkv * (2 * d + 4)) + n * (8 + nq * d * 4) + n * nkv * k * 4,
                "flops": sum(seen) * nkv * 4 * d}
    seen = [min(k, p // BLOCK + 1) for _, p in rows]
    tokens = sum(min(_blocks(a), sum(b for b, (q, _) in zip(seen, rows) if q == s)) * BLOCK
                 for s, a in enumerate(_spread(c, "ctx", 0)))
    return {"bytes": 2 * tokens * nkv * _key_bytes(c["kv"], d) + n * nkv * k * 4 + 2 * n * nq * d * 4 + 8 * n,
            "flops": 4 * sum(seen) * BLOCK * nq * d}


# ---------------------------------------------------------------------------
# inputs

def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(tokens, gen, spare=0, width=None):
    """Block tables [sequences][width] of distinct scattered ids (unused entries -1), the ids left over, and the
    number of blocks."""
    need = [_blocks(t) for t in tokens]
    blocks = max(1, sum(need) + spare)
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(need), width or max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = ids[at:at + k]
        at += k
    return bt, ids[at:].contiguous(), blocks


def _pool(kv, blocks, nkv, d, g, gen):
    """Normally distributed values in the cache format."""
    x = torch.randn((blocks, nkv, BLOCK, d), generator=gen, device="cuda").div_(g)
    if kv == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    if kv == "bf16":
        return x.to(torch.bfloat16)
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    b = b / scale.float().unsqueeze(-1)
    code = sum((b.abs() > t).to(torch.uint8) for t in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))
    code = (code | ((b < 0).to(torch.uint8) << 3)).flatten(-2)
    return torch.cat(((code[..., 0::2] | (code[..., 1::2] << 4)).flatten(2), scale.view(torch.uint8).flatten(2)), -1)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx = _spread(c, "ctx", 0)
    s = dict(c=c)
    if c["op"] == "extend":
        new = _spread(c, "new", 7)
        took = sum(_blocks(a + k) - _blocks(a) for a, k in zip(ctx, new))
        width = max(1, max(_blocks(a + k) for a, k in zip(ctx, new)))
        s["bt"], free, s["blocks"] = _tables(ctx, gen, took + 40, width)
        n = -(-max(1, sum(new)) // 8) * 8                         # captured sizes are multiples of 8: rows left over are padding
        s["free"], s["at"] = torch.cat((free[:5], free)), _int32([5])   # five entries taken earlier
        s["ctx"], s["new"] = _int32(ctx), _int32(new)
        s["held"], s["cu"], s["next"] = torch.empty_like(s["ctx"]), _int32([0] * (len(ctx) + 1)), _int32([0])
        s["positions"], s["row_seq"] = _int32([0] * n), _int32([0] * n)
        s["slots"] = torch.zeros(n, dtype=torch.int64, device="cuda")
        return s
    rows = _rows(c)
    nkv, d = c["nkv"], c["d"]
    s["positions"], s["row_seq"] = _int32([p for _, p in rows]), _int32([q for q, _ in rows])
    if c["op"] == "bounds":
        s["bt"], _, s["blocks"] = _tables([a + k for a, k in zip(ctx, _spread(c, "new", 7))], gen)
        s["k"] = _pool(c["kv"], s["blocks"] + 1, nkv, d, K_SCALE, gen)
        s["codes"] = torch.zeros((s["blocks"] + 1, nkv, 2, d), dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros((s["blocks"] + 1, nkv), device="cuda")
        return s
    s["bt"], _, s["blocks"] = _tables(ctx, gen)
    n, nq, k = len(rows), c["nq"], c["k"]
    s["q"] = torch.randn((n, nq, d), generator=gen, device="cuda")
    s["sel"] = torch.empty((n, nkv, k), dtype=torch.int32, device="cuda")
    if c["op"] == "select":
        # ranges as 16 normally distributed keys around a block's own middle have them
        shape = (s["blocks"] + 1, nkv, d)
        mid = torch.randn(shape, generator=gen, device="cuda") * 12.0
        half = 45.0 + 8.0 * torch.randn(shape, generator=gen, device="cuda")
        s["codes"] = torch.stack(((mid - half).floor(), (mid + half).ceil()), 2).clamp_(-127, 127).to(torch.int8)
        s["scales"] = torch.exp2(torch.randint(-6, -4, shape[:2], generator=gen, device="cuda").float())
        return s
    s["k"] = _pool(c["kv"], s["blocks"] + 1, nkv, d, K_SCALE, gen)
    s["v"] = _pool(c["kv"], s["blocks"] + 1, nkv, d, V_SCALE, gen)
    # blocks at random per (row, KV head), in order, the row's own among them
    last = (s["positions"] // BLOCK)[:, None, None]
    at = torch.rand((n, nkv, s["bt"].shape[1]), generator=gen, device="cuda")
    j = torch.arange(s["bt"].shape[1], device="cuda")
    at = torch.where(j > last, 2.0, torch.where(j == last, -1.0, at))
    pick = at.argsort(-1)[..., :k]
    pick = torch.where(pick > last, 1 << 30, pick).sort(-1)[0]
    s["sel"].fill_(-1)[..., :pick.shape[-1]] = torch.where(pick < 1 << 30, pick, -1).to(torch.int32)
    s["out"] = torch.empty((n, nq * d), device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms

def _plain_extend(s):
    ctx, new, bt, free = s["ctx"].long(), s["new"].long(), s["bt"], s["free"]
    nseq, width = bt.shape
    n, at = s["positions"].shape[0], s["at"].long()
    valid = (ctx >= 0) & (new >= 0) & (ctx + new <= width * BLOCK)
    new = torch.where(valid, new, 0)
    have = (ctx + BLOCK - 1) // BLOCK
    need = torch.where(valid, (ctx + new + BLOCK - 1) // BLOCK - have, 0)
    first = at + need.cumsum(0) - need
    fits = (new == 0) | ((new.cumsum(0) <= n) & ((need == 0) | (first + need <= free.shape[0])))
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    j = torch.arange(width, device=bt.device)
    grown = (j >= have[:, None]) & (j < (have + need)[:, None])
    bt.copy_(torch.where(grown, free[(first[:, None] + j - have[:, None]).clamp(0, free.shape[0] - 1)], bt))
    s["held"].copy_(ctx + new)
    s["cu"][1:] = new.cumsum(0)
    s["next"].copy_(at + need.sum())
    row = torch.arange(n, device=bt.device)
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    live, q = seq < nseq, seq.clamp(max=nseq - 1)
    pos = torch.where(live, ctx[q] + row - s["cu"].long()[q], 0)
    block = bt[q, (pos // BLOCK).clamp(max=width - 1)].long()
    slot = torch.where((block >= 0) & (block <= s["blocks"]), block * BLOCK + pos % BLOCK, -1)
    s["row_seq"].copy_(seq)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(live, slot, s["blocks"] * BLOCK))
    return _extended(s)


def _extended(s):
    return {k: s[k] for k in ("bt", "held", "cu", "next", "positions", "row_seq", "slots")}


def _values(raw, kv, d, dtype):
    """Values, before the tensor's scale, of units gathered from a pool: [..., 16, d]."""
    if kv == "bf16":
        return raw.to(dtype)
    if kv == "e4m3":
        return raw.view(torch.float8_e4m3fn).to(dtype)
    n = BLOCK * d // 2
    codes = raw[..., :n].unflatten(-1, (BLOCK, d // 2))
    codes = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    scale = raw[..., n:].unflatten(-1, (BLOCK, d // 16)).contiguous().view(torch.float8_e4m3fn).to(dtype)
    lut = torch.tensor(E2M1, dtype=dtype, device=raw.device)
    return (lut[codes.int()].unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2)


def _power(e):
    """2^e in 64 bits, from its bits: torch.ldexp goes through a power that a GPU rounds."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _plain_bounds(s):
    """Every row works on its block as its last row in the block has it (rows of a block write the same)."""
    c = s["c"]
    seq, pos = s["row_seq"].long(), s["positions"].long()
    row = torch.arange(len(pos), device=pos.device)
    ends = torch.searchsorted(seq, seq, right=True) - 1                  # the sequence's last row
    last = pos + torch.minimum(BLOCK - 1 - pos % BLOCK, ends - row)
    block = s["bt"][seq, last // BLOCK].long()
    step = max(1, CHUNK // (c["nkv"] * BLOCK * c["d"]))
    for a in range(0, len(pos), step):
        at, upto = block[a:a + step], last[a:a + step] % BLOCK
        k = _values(s["k"][at], c["kv"], c["d"], torch.float32)
        live = (torch.arange(BLOCK, device=pos.device) <= upto[:, None])[:, None, :, None]
        zero = torch.zeros((), device=pos.device)
        most = torch.where(live, k.abs(), zero).amax((-1, -2))
        bad = ~torch.where(live, k, zero).isfinite().all(-1).all(-1)
        frac, e = torch.frexp(torch.where(bad, zero, most))
        e = (e - torch.where(frac <= 127.0 / 128.0, 7, 6)).clamp(min=-100)
        unit = _power(e)[..., None]
        low = (torch.where(live, k, math.inf).amin(-2).double() / unit).floor()
        high = (torch.where(live, k, -math.inf).amax(-2).double() / unit).ceil()
        code = torch.where((bad | (most == 0))[..., None, None], 0.0, torch.stack((low, high), 2))
        s["codes"][at] = code.to(torch.int8)
        s["scales"][at] = torch.where(bad, math.inf, torch.where(most == 0, 0.0, unit[..., 0])).float()
    return s["codes"], s["scales"]


def _plain_select(s):
    c = s["c"]
    nq, nkv, d, k = c["nq"], c["nkv"], c["d"], c["k"]
    G, width = nq // nkv, s["bt"].shape[1]
    j = torch.arange(width, device="cuda")
    step = max(1, CHUNK // (nkv * width * 2 * d))
    for a in range(0, s["q"].shape[0], step):
        seq, pos = s["row_seq"][a:a + step].long(), s["positions"][a:a + step].long()
        q = s["q"][a:a + step].view(-1, nkv, G, d).double()
        most = q.abs().amax((-1, -2), keepdim=True)
        fine = most.isfinite() & (most > 0)
        x = torch.frexp(torch.where(fine, most, 1.0))[1]
        u = torch.where(fine, torch.round(q * _power(10 - x)), 0.0)
        w = torch.cat((u.clamp(max=0).sum(2), u.clamp(min=0).sum(2)), -1)          # [rows, nkv, 2 d]: with low, with high
        ids = s["bt"][seq].long()
        ids = torch.where((ids < 0) | (ids > s["blocks"]), s["blocks"], ids)
        code = s["codes"][ids].flatten(-2).transpose(1, 2).double()                # [rows, nkv, width, 2 d]
        scale = s["scales"][ids].transpose(1, 2)
        score = (code @ w.unsqueeze(-1)).squeeze(-1).float() * scale
        score = torch.where(scale == math.inf, math.inf, score).double().clamp(-1e200, 1e200)
        held = (pos // BLOCK + 1)[:, None, None]
        kept = (j < c["first"]) | (j >= held - c["last"])
        score = torch.where(j < held, torch.where(kept, 1e250, score), -1e250)
        pick = score.sort(stable=True, dim=-1, descending=True)[1][..., :k]
        pick = torch.where(pick < held, pick, 1 << 30).sort(-1)[0]
        s["sel"][a:a + step] = -1
        s["sel"][a:a + step, :, :pick.shape[-1]] = torch.where(pick < 1 << 30, pick, -1).to(torch.int32)
    return s["sel"]


def _plain_attend(s):
    c = s["c"]
    nq, nkv, d, k, kv = c["nq"], c["nkv"], c["d"], c["k"], c["kv"]
    G = nq // nkv
    head = torch.arange(nkv, device="cuda")[:, None]
    tok = torch.arange(BLOCK, device="cuda")
    step = max(1, CHUNK // (nkv * k * BLOCK * d))
    for a in range(0, s["q"].shape[0], step):
        seq, pos = s["row_seq"][a:a + step].long(), s["positions"][a:a + step].long()
        sel = s["sel"][a:a + step].long()                                          # [rows, nkv, k]
        ids = s["bt"][seq[:, None, None], sel.clamp(min=0)].long()
        kk = _values(s["k"][ids, head], kv, d, torch.float32).flatten(2, 3) * K_SCALE
        vv = _values(s["v"][ids, head], kv, d, torch.float32).flatten(2, 3) * V_SCALE
        seen = ((sel >= 0)[..., None] & (sel[..., None] * BLOCK + tok <= pos[:, None, None, None])).flatten(2)
        vv = torch.where(seen[..., None], vv, torch.zeros((), device="cuda"))
        q = s["q"][a:a + step].view(-1, nkv, G, d)
        score = torch.where(seen.unsqueeze(2), (q @ kk.transpose(-1, -2)) / math.sqrt(d), -math.inf)
        most = score.amax(-1, keepdim=True)
        p = torch.exp(score - torch.where(most == -math.inf, torch.zeros_like(most), most))
        total = p.sum(-1, keepdim=True)
        o = (p @ vv) / torch.where(total == 0, torch.ones_like(total), total)
        s["out"][a:a + step] = o.reshape(-1, nq * d)
    return s["out"]


def _own(s):
    from memory_bound_transformer_gb300 import capi
    c = s["c"]
    if c["op"] == "extend":
        capi.op_kv_extend(s["ctx"], s["new"], s["bt"], s["blocks"], s["free"], s["at"], s["held"], s["cu"], s["positions"],
                          s["row_seq"], s["slots"], s["next"])
        return _extended(s)
    kinds = {"bf16": capi.DTYPE_BF16, "e4m3": capi.DTYPE_E4M3, "fp4": capi.DTYPE_E2M1}
    nkv, d = c["nkv"], c["d"]
    if c["op"] == "bounds":
        capi.op_key_bounds(s["positions"], s["bt"], s["k"], nkv, d, kinds[c["kv"]], s["blocks"], s["codes"], s["scales"],
                           row_seq=s["row_seq"])
        return s["codes"], s["scales"]
    if c["op"] == "select":
        capi.op_block_select(s["q"], nkv, s["codes"], s["scales"], s["positions"], s["bt"], s["blocks"], c["first"],
                             c["last"], s["sel"], row_seq=s["row_seq"])
        return s["sel"]
    capi.op_block_attention(s["q"], nkv, s["k"], s["v"], kinds[c["kv"]], K_SCALE, V_SCALE, s["positions"], s["bt"],
                            s["sel"], s["blocks"], s["out"], row_seq=s["row_seq"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"extend": _plain_extend, "bounds": _plain_bounds, "select": _plain_select,
            "attend": _plain_attend}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_extend(s):
    """One sequence after another, one row after another."""
    bt, free = s["bt"].cpu().numpy().copy(), s["free"].cpu().numpy()
    ctx, new = s["ctx"].tolist(), s["new"].tolist()
    n, at, asked, rows = s["positions"].shape[0], int(s["at"]), 0, []
    want, held, cu = at, [], [0]
    for i, (a, k) in enumerate(zip(ctx, new)):
        need = _blocks(a + k) - _blocks(a)
        asked, want = asked + k, want + need
        ok = k == 0 or (asked <= n and (need == 0 or want <= len(free)))
        if ok and need:
            bt[i, _blocks(a):_blocks(a) + need] = free[want - need:want]
            at = want
        k = k if ok else 0
        held.append(a + k)
        cu.append(cu[-1] + k)
        rows += [(i, p, int(bt[i, p // BLOCK]) * BLOCK + p % BLOCK) for p in range(a, a + k)]
    rows += [(len(ctx), 0, s["blocks"] * BLOCK)] * (n - len(rows))
    rows = np.array(rows, dtype=np.int64).reshape(n, 3)
    dev = lambda x: torch.as_tensor(np.ascontiguousarray(x), device="cuda")  # noqa: E731
    return dict(bt=dev(bt), held=_int32(held), cu=_int32(cu), next=_int32([at]), positions=dev(rows[:, 1].astype(np.int32)),
                row_seq=dev(rows[:, 0].astype(np.int32)), slots=dev(rows[:, 2]))


def _exact_bounds(s):
    """One block after another."""
    c = s["c"]
    codes, scales = torch.zeros_like(s["codes"]), torch.zeros_like(s["scales"])
    grown = {}
    for q, p in _rows(c):
        grown[q, p // BLOCK] = p % BLOCK + 1
    for (q, b), tokens in grown.items():
        at = int(s["bt"][q, b])
        k = _values(s["k"][at], c["kv"], c["d"], torch.float64)[:, :tokens].cpu().numpy()
        for h in range(c["nkv"]):
            most = np.abs(k[h]).max()
            if most == 0:
                continue
            e = -100
            if most > 127 * 2.0 ** e:
                e = int(math.floor(math.log2(most / 127))) - 1
                while most > 127 * 2.0 ** e:
                    e += 1
            pair = np.stack((np.floor(k[h].min(0) / 2.0 ** e), np.ceil(k[h].max(0) / 2.0 ** e)))
            codes[at, h] = torch.as_tensor(pair, device="cuda").to(torch.int8)
            scales[at, h] = 2.0 ** e
    return codes, scales


def _exact_select(s):
    """One row and KV head after another, ranks counted by a lexicographic sort."""
    c = s["c"]
    G, d, k = c["nq"] // c["nkv"], c["d"], c["k"]
    sel = torch.full_like(s["sel"], -1)
    for i, (r, p) in enumerate(_rows(c)):
        held = p // BLOCK + 1
        ids = s["bt"][r, :held].long()
        code, scale = s["codes"][ids].double(), s["scales"][ids].cpu().numpy()
        for h in range(c["nkv"]):
            q = s["q"][i, h * G:(h + 1) * G].double()
            top = float(q.abs().max())
            u = torch.zeros_like(q) if top == 0 or not math.isfinite(top) else (q * 2.0 ** (10 - math.frexp(top)[1])).round()
            dot = (code[:, h, 1] * torch.relu(u).sum(0) - code[:, h, 0] * torch.relu(-u).sum(0)).sum(-1)
            score = (dot.cpu().numpy().astype(np.float32) * scale[:, h]).astype(np.float64)
            j = np.arange(held)
            kept = (j < c["first"]) | (j >= held - c["last"])
            order = np.lexsort((j, -score, ~kept))[:k]
            sel[i, h, :len(order)] = torch.as_tensor(np.sort(order).astype(np.int32), device="cuda")
    return sel


def _exact_attend(s):
    """One row and KV head after another."""
    c = s["c"]
    G, d, kv = c["nq"] // c["nkv"], c["d"], c["kv"]
    out = torch.zeros((len(s["q"]), c["nq"], d), dtype=torch.float64, device="cuda")
    sel = s["sel"].cpu().numpy()
    for i, (r, p) in enumerate(_rows(c)):
        for h in range(c["nkv"]):
            pick = sel[i, h][sel[i, h] >= 0]
            ids = s["bt"][r, torch.as_tensor(pick, device="cuda").long()].long()
            seen = (pick[:, None] * BLOCK + np.arange(BLOCK)).reshape(-1) <= p
            seen = torch.as_tensor(np.flatnonzero(seen), device="cuda")
            k = _values(s["k"][ids, h], kv, d, torch.float64).reshape(-1, d)[seen] * K_SCALE
            v = _values(s["v"][ids, h], kv, d, torch.float64).reshape(-1, d)[seen] * V_SCALE
            w = torch.softmax(s["q"][i, h * G:(h + 1) * G].double() @ k.T * d ** -0.5, -1)
            out[i, h * G:(h + 1) * G] = w @ v
    return out.view(len(s["q"]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "bounds": _exact_bounds, "select": _exact_select, "attend": _exact_attend}[case["op"]](s)
