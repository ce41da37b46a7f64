"""The 4-bit paged KV cache's operators and prompt attention, as timed cases with their plain forms.

Three paths, each called as a serving program calls it:

* append: the rows of a QKV projection are rotated, their keys and values go into the 4-bit paged cache, and
  the rows are read back from it as fp32 values (op_rope_kv_write_fp4, op_kv_read_fp4);
* decode: one query token per sequence attends over its cached context (op_paged_attention_fp4);
* prompt: packed prompts attend causally over the paged cache, which holds their own rows and what came before
  (op_prompt_attention; BF16, e4m3 and 4-bit caches).

The 4-bit cache holds one e2m1 code per value and one e4m3 scale per 16 channels of a token's head; with the
tensor's fp32 scale g a code stands for e2m1 * e4m3 * g. A (block, KV head) of a pool is 16 tokens: their codes
[16][d / 2] (channel 2j in the low half of byte j), then their scales [16][d / 16].
"""
import math

import torch

own = False

BLOCK = 16
# e2m1: sign, two exponent bits, one mantissa bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
K_SCALE, V_SCALE = 0.875, 1.25
THETA = 10000.0


def listed():
    return [
        # one decode step of 64 sequences writes its rows (8B-class heads): latency
        dict(name="append 64 rows 8b", op="append", n=64, nq=32, nkv=8, d=128, seqs=64, max_pos=4096),
        # four packed prompts of 1021 tokens (70B-class heads): bandwidth
        dict(name="append 4084 rows 70b", op="append", n=4084, nq=64, nkv=8, d=128, seqs=4, max_pos=4096),
        # a single sequence being decoded, 8B-class heads: latency
        dict(name="decode 8b batch 1", op="decode", B=1, lo=2048, hi=2048, nq=32, nkv=8, d=128),
        # the 8B-class batch workload: contexts spread over 256..2048
        dict(name="decode 8b batch 64", op="decode", B=64, lo=256, hi=2048, nq=32, nkv=8, d=128),
        # the 70B-class batch workload: 64 contexts of 2048
        dict(name="decode 70b batch 64", op="decode", B=64, lo=2048, hi=2048, nq=64, nkv=8, d=128),
        # the 32B-class workload, five query heads per KV head, short ragged contexts
        dict(name="decode 32b batch 32", op="decode", B=32, lo=64, hi=256, nq=40, nkv=8, d=128),
        # few sequences with long contexts: the context has to be split
        dict(name="decode 70b long", op="decode", B=4, lo=30001, hi=32765, nq=64, nkv=8, d=128),
        # one short prompt, 1B-class heads of 64 channels: latency
        dict(name="prompt 1b 33", op="prompt", kv="fp4", lens="33", prefix="0", nq=32, nkv=8, d=64),
        # packed prompts of different lengths, an empty one among them, BF16 cache
        dict(name="prompt 8b packed bf16", op="prompt", kv="bf16", lens="1024,1,300,17,0,777,513,128",
             prefix="0,700,0,0,5,33,0,0", nq=32, nkv=8, d=128),
        # a prompt of ordinary length over the 4-bit cache
        dict(name="prompt 8b 2048 fp4", op="prompt", kv="fp4", lens="2048", prefix="0", nq=32, nkv=8, d=128),
        # the next piece of a long prompt: 1000 new tokens over 8200 cached ones
        dict(name="prompt 70b piece fp4", op="prompt", kv="fp4", lens="1000", prefix="8200", nq=64, nkv=8, d=128),
        # the largest: a 4096-token prompt, 70B-class heads, e4m3 cache as that workload has it
        dict(name="prompt 70b 4096 e4m3", op="prompt", kv="e4m3", lens="4096", prefix="0", nq=64, nkv=8, d=128),
    ]


HEADS = ((32, 8, 64), (32, 8, 128), (40, 8, 128), (64, 8, 128), (4, 2, 64), (8, 8, 128), (16, 1, 128))


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prompt"))
    nq, nkv, d = rng.choice(HEADS)
    if op == "append":
        n = _log(rng, 1, 4096)
        return dict(op=op, n=n, nq=nq, nkv=nkv, d=d, seqs=min(n, _log(rng, 1, 64)), max_pos=4096)
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(32768, 131072 // B))
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, nq=nq, nkv=nkv, d=d)
    nseq = rng.randint(1, 6)
    most = 2500 // nseq
    lens = [rng.choice((0, 1)) if rng.random() < 0.15 else _log(rng, 1, most) for _ in range(nseq)]
    lens[0] = max(lens[0], 1)
    prefix = [0 if rng.random() < 0.6 else _log(rng, 1, 1500) for _ in range(nseq)]
    return dict(op=op, kv=rng.choice(("bf16", "e4m3", "fp4")), lens=",".join(map(str, lens)),
                prefix=",".join(map(str, prefix)), nq=nq, nkv=nkv, d=d)


# ---------------------------------------------------------------------------
# sizes

def _ints(text):
    return [int(x) for x in text.split(",")]


def _contexts(c):
    """Context lengths spread over [lo, hi] in a fixed scattered order."""
    span = c["hi"] - c["lo"] + 1
    return [c["lo"] + (i * 2654435761 + span // 2) % span for i in range(c["B"])]


def _rows(c):
    """(sequence, position) of each row of an append: the rows spread evenly over the sequences, each run of
    rows behind some tokens cached before."""
    per, more = divmod(c["n"], c["seqs"])
    got = []
    for s in range(c["seqs"]):
        k = per + (s < more)
        at = (s * 97) % max(1, c["max_pos"] - k + 1)
        got += [(s, at + j) for j in range(k)]
    return got


def _token_bytes(kv, d):
    return {"bf16": 2 * d, "e4m3": d, "fp4": d // 2 + d // 16}[kv]


def work(case):
    c = case
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    if c["op"] == "append":
        n = c["n"]
        angles = len({p for _, p in _rows(c)}) * d * 4
        cache = 2 * n * nkv * _token_bytes("fp4", d)
        return {"bytes": n * (nq + 2 * nkv) * d * 4 + angles + n * nq * d * 4 + 2 * cache + 2 * n * nkv * d * 4,
                "flops": n * (nq + nkv) * d * 3 + 4 * n * nkv * d}
    if c["op"] == "decode":
        total = sum(_contexts(c))
        return {"bytes": 2 * total * nkv * _token_bytes("fp4", d) + 2 * c["B"] * nq * d * 4,
                "flops": 4 * total * nq * d}
    lens, prefix = _ints(c["lens"]), _ints(c["prefix"])
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, prefix))
    cached = sum(n + p for n, p in zip(lens, prefix) if n)
    return {"bytes": 2 * cached * nkv * _token_bytes(c["kv"], d) + 2 * sum(lens) * nq * d * 4,
            "flops": 4 * pairs * nq * d}


# ---------------------------------------------------------------------------
# inputs

def _quantise(x, g):
    """x [..., d] fp64 -> e2m1 codes (0..15) and e4m3 scale bits of its blocks of 16 channels.

    scale = e4m3(max |x| / (6 g)), code = e2m1(x / (scale g)), both to nearest (ties to even) and saturating."""
    b = x.unflatten(-1, (-1, 16))
    want = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0)
    # the e4m3 grid: 8 steps per binade, steps of 2^-9 below 2^-6
    e = torch.floor(torch.log2(want.clamp(min=2.0 ** -6)))
    e = e + (want >= torch.exp2(e + 1)).to(e.dtype) - (want < torch.exp2(e)).to(e.dtype) * (want >= 2.0 ** -6)
    step = torch.exp2(e - 3)
    scale = torch.round(want / step) * step
    bits = scale.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    unit = (scale * g).unsqueeze(-1)
    a = b.abs()
    code = ((a > 0.25 * unit).to(torch.uint8) + (a >= 0.75 * unit) + (a > 1.25 * unit) + (a >= 1.75 * unit)
            + (a > 2.5 * unit) + (a >= 3.5 * unit) + (a > 5.0 * unit))
    code = torch.where(unit > 0, code, torch.zeros_like(code)) | ((b < 0).to(torch.uint8) << 3)
    return code.flatten(-2), bits


def _pool_of(codes, bits):
    """codes [blocks, nkv, 16, d], scale bits [blocks, nkv, 16, d / 16] -> pool bytes [blocks, nkv, unit]."""
    return torch.cat(((codes[..., 0::2] | (codes[..., 1::2] << 4)).flatten(2), bits.flatten(2)), dim=-1).contiguous()


def _pool(kv, blocks, nkv, d, g, gen):
    x = torch.randn((blocks, nkv, BLOCK, d), generator=gen, device="cuda")
    if kv == "fp4":
        return _pool_of(*_quantise(x.double(), g))
    if kv == "e4m3":
        return (x / g).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return (x / g).to(torch.bfloat16)


def _tables(tokens, gen):
    """Block tables [sequences][width] of distinct scattered block ids for so many tokens each, and the blocks."""
    need = [max(1, -(-t // BLOCK)) for t in tokens]
    blocks = sum(need) + 1
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, k in enumerate(need):
        bt[s, :k] = ids[at:at + k]
        at += k
    return bt, blocks


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    s = dict(c=c)
    if c["op"] == "append":
        rows = _rows(c)
        s["bt"], blocks = _tables([max([p for q, p in rows if q == i], default=0) + 1 for i in range(c["seqs"])], gen)
        s["qkv"] = torch.randn((c["n"], (nq + 2 * nkv) * d), generator=gen, device="cuda")
        s["positions"], s["row_seq"] = _int32([p for _, p in rows]), _int32([q for q, _ in rows])
        # cos and sin of the rotations, kept by a program for all its calls
        angle = (torch.arange(c["max_pos"], dtype=torch.float64, device="cuda")[:, None]
                 * THETA ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d))
        s["rope"] = torch.stack((torch.cos(angle), torch.sin(angle)), dim=-1).float().contiguous()
        unit = BLOCK * _token_bytes("fp4", d)
        s["k"] = torch.zeros((blocks + 1, nkv, unit), dtype=torch.uint8, device="cuda")
        s["v"] = torch.zeros_like(s["k"])
        s["q_out"] = torch.empty((c["n"], nq, d), device="cuda")
        s["k_out"] = torch.empty((c["n"], nkv, d), device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        lens = [1] * c["B"] if c["op"] == "decode" else _ints(c["lens"])
        held = _contexts(c) if c["op"] == "decode" else [n + p for n, p in zip(lens, _ints(c["prefix"]))]
        kv = c.get("kv", "fp4")
        s["bt"], blocks = _tables(held, gen)
        s["k"], s["v"] = _pool(kv, blocks + 1, nkv, d, K_SCALE, gen), _pool(kv, blocks + 1, nkv, d, V_SCALE, gen)
        s["q"] = torch.randn((sum(lens), nq, d), generator=gen, device="cuda")
        s["held"] = _int32(held)
        s["cu"] = _int32([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["out"] = torch.empty((sum(lens), nq * d), device="cuda")
        if c["op"] == "prompt":
            s["most_q"] = max(lens)
    s["blocks"] = blocks
    return s


# ---------------------------------------------------------------------------
# plain forms

def _values(pool, kv, nkv, d, g, dtype):
    """The values that a pool stands for: [blocks, nkv, 16, d]."""
    if kv == "bf16":
        return pool.to(dtype) * g
    if kv == "e4m3":
        return pool.view(torch.float8_e4m3fn).to(dtype) * g
    n = BLOCK * d // 2
    raw = pool[..., :n].reshape(-1, nkv, BLOCK, d // 2)
    codes = torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2)
    scale = pool[..., n:].reshape(-1, nkv, BLOCK, d // 16).view(torch.float8_e4m3fn).to(dtype)
    lut = torch.tensor(E2M1, dtype=dtype, device=pool.device)
    return (lut[codes.int()].unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2) * g


def _plain_append(s):
    c = s["c"]
    nq, nkv, d, n = c["nq"], c["nkv"], c["d"], c["n"]
    x = s["qkv"].view(n, nq + 2 * nkv, d).double()          # 64 bits: values next to a border of the 4-bit grid
    turn = s["rope"][s["positions"].long()].double()[:, None]
    cos, sin = turn[..., 0], turn[..., 1]
    a, b = x[:, :nq + nkv, :d // 2], x[:, :nq + nkv, d // 2:]
    turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    block = s["bt"][s["row_seq"].long(), (s["positions"] // BLOCK).long()].long()
    slot = (s["positions"] % BLOCK).long()
    half = BLOCK * d // 2
    for pool, y, g, out in ((s["k"], turned[:, nq:], K_SCALE, s["k_out"]), (s["v"], x[:, nq + nkv:], V_SCALE, s["v_out"])):
        codes, bits = _quantise(y, g)
        pool[:, :, :half].view(-1, nkv, BLOCK, d // 2)[block, :, slot] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        pool[:, :, half:].view(-1, nkv, BLOCK, d // 16)[block, :, slot] = bits
        back = torch.cat((pool[:, :, :half].view(-1, nkv, BLOCK, d // 2)[block, :, slot],
                          pool[:, :, half:].view(-1, nkv, BLOCK, d // 16)[block, :, slot]), dim=-1)
        raw, scale = back[..., :d // 2], back[..., d // 2:].contiguous().view(torch.float8_e4m3fn).float()
        lut = torch.tensor(E2M1, device=pool.device)
        vals = lut[torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2).int()]
        out.copy_((vals.unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2) * g)
    s["q_out"].copy_(turned[:, :nq])
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_attention(s, lens_max):
    """Every sequence padded to the longest prompt and the longest context, masked where there is nothing."""
    c = s["c"]
    nq, nkv, d, kv = c["nq"], c["nkv"], c["d"], c.get("kv", "fp4")
    cu, held = s["cu"].long(), s["held"].long()
    lens = cu[1:] - cu[:-1]
    at = torch.arange(lens_max, device="cuda")
    row = (cu[:-1, None] + at).clamp(max=s["q"].shape[0] - 1)            # [sequences, queries]
    live = at < lens[:, None]
    place = held[:, None] - lens[:, None] + at                           # the queries' positions
    bt = s["bt"].clamp(min=0).long()
    width = bt.shape[1] * BLOCK
    k = _values(s["k"], kv, nkv, d, K_SCALE, torch.float32)[bt].transpose(1, 2).reshape(-1, nkv, width, d)
    v = _values(s["v"], kv, nkv, d, V_SCALE, torch.float32)[bt].transpose(1, 2).reshape(-1, nkv, width, d)
    tok = torch.arange(width, device="cuda")
    v = torch.where((tok < held[:, None])[:, None, :, None], v, torch.zeros((), device="cuda"))
    q = s["q"][row].view(-1, lens_max, nkv, nq // nkv, d).permute(0, 2, 3, 1, 4).reshape(-1, nkv, nq // nkv * lens_max, d)
    score = (q @ k.transpose(-1, -2)).view(-1, nkv, nq // nkv, lens_max, width) / math.sqrt(d)
    seen = (tok <= place[..., None]) & (tok < held[:, None, None]) & live[..., None]
    score = torch.where(seen[:, None, None], score, torch.full((), -math.inf, device="cuda"))
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(most == -math.inf, torch.zeros_like(most), most))
    total = p.sum(-1, keepdim=True)
    o = p.view(-1, nkv, nq // nkv * lens_max, width) @ v
    o = o.view(-1, nkv, nq // nkv, lens_max, d) / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(-1, lens_max, nq * d)[live])
    return s["out"]


def _own(s):
    from memory_bound_transformer_gb300 import capi
    c = s["c"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    if c["op"] == "append":
        capi.op_rope_kv_write_fp4(s["qkv"], nq, nkv, d, s["positions"], s["bt"], s["rope"], s["k"], s["v"], s["blocks"],
                                  K_SCALE, V_SCALE, s["q_out"], row_seq=s["row_seq"])
        capi.op_kv_read_fp4(s["positions"], s["bt"], s["k"], s["v"], nkv, d, s["blocks"], K_SCALE, V_SCALE, s["k_out"],
                            s["v_out"], row_seq=s["row_seq"])
        return s["q_out"], s["k_out"], s["v_out"]
    if c["op"] == "decode":
        capi.op_paged_attention_fp4(s["q"], nkv, s["k"], s["v"], K_SCALE, V_SCALE, s["bt"], s["held"], s["blocks"], s["out"])
        return s["out"]
    kinds = {"bf16": capi.DTYPE_BF16, "e4m3": capi.DTYPE_E4M3, "fp4": capi.DTYPE_E2M1}
    capi.op_prompt_attention(s["q"], nkv, s["cu"], s["held"], s["k"], s["v"], kinds[c["kv"]], K_SCALE, V_SCALE, s["bt"],
                             s["blocks"], s["out"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state, 1 if op == "decode" else state["most_q"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and one KV head at a time

def _nearest(x, grid):
    """The entry of an increasing grid nearest to x >= 0; between two equally near the one at an even place."""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    wide = torch.float64
    dev = "cuda"
    if c["op"] == "append":
        e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=wide, device=dev)
        e4m3 = torch.tensor([m / 8 * 2.0 ** -6 for m in range(8)]
                            + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1], dtype=wide, device=dev)
        x = s["qkv"].to(wide).view(c["n"], nq + 2 * nkv, d)
        z = torch.view_as_complex(s["rope"].to(wide))[s["positions"].long()][:, None]
        y = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous())[:, :nq + nkv] * z
        y = torch.cat((y.real, y.imag), dim=-1)
        got = [y[:, :nq]]
        for t, g in ((y[:, nq:], K_SCALE), (x[:, nq + nkv:], V_SCALE)):
            b = t.reshape(-1, 16)
            scale = _nearest(b.abs().amax(1) / (6 * g), e4m3)[:, None] * g
            got.append((torch.where(scale > 0, _nearest(b.abs() / scale, e2m1) * scale, 0.0) * torch.sign(b)).view(c["n"], nkv, d))
        return tuple(got)
    kv = c.get("kv", "fp4")
    out = torch.zeros((s["q"].shape[0], nq, d), dtype=wide, device=dev)
    G = nq // nkv
    edges, held = s["cu"].tolist(), s["held"].tolist()
    for i, size in enumerate(held):
        lo, hi = edges[i], edges[i + 1]
        if hi == lo or size == 0:
            continue
        ids = s["bt"][i, :-(-size // BLOCK)].long()
        kk = _values(s["k"][ids], kv, nkv, d, K_SCALE, wide)
        vv = _values(s["v"][ids], kv, nkv, d, V_SCALE, wide)
        place = torch.arange(hi - lo, device=dev) + size - (hi - lo)
        for h in range(nkv):
            k, v = kk[:, h].reshape(-1, d)[:size], vv[:, h].reshape(-1, d)[:size]
            for at in range(lo, hi, 1024):
                to = min(hi, at + 1024)
                q = s["q"][at:to, h * G:(h + 1) * G].to(wide)
                w = torch.einsum("ngd,td->ngt", q, k) * d ** -0.5
                w.masked_fill_((torch.arange(size, device=dev) > place[at - lo:to - lo, None])[:, None], -math.inf)
                out[at:to, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(w, -1), v)
    return out.view(-1, nq * d)
