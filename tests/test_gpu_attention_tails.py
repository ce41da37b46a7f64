"""A dominant token in front of thousands of equal ones (an attention sink): the
others' probabilities are far below the largest, and their shares add up.

Token 0's key gives every query a score `nats` above the others', whose keys are
zero; its value is zero and theirs are one (4-bit: the nearest that its scale's
grid has). So the output is that value times the others' share,
n e^-nats / (1 + n e^-nats), in every channel.

Tolerance: 2e-5 * max |V|, that of all attention here. Probabilities enter the
MMAs as FP16 high and low parts of 2^14 p / p_max: off by half of FP16's
smallest step at most, 2^-25 * 2^-14 of the largest, which 2^15 tokens add up to
2^-24. Unscaled it would be 2^-25 each, 1e-3 over 32768 tokens."""
import numpy as np
import pytest
import torch

from memory_bound_transformer_gb300 import capi
from oracle.kv_fp4 import encode, pack_pool, pool_values, rows_attention
from oracle.numerics import round_bf16, round_e4m3
from tests.test_gpu_kv_fp4 import dev, tables
from tests.test_gpu_prompt_attention import KINDS, to_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
TAILS = [(4096, 16.2), (4096, 18.0), (9200, 17.5), (32768, 16.2), (32768, 18.0), (32768, 24.0)]


def pools(kind, lens, nkv, d, seed=1):
    """(K, V, table, blocks, the others' value) of sequences whose token 0 is the sink: key 6 in channel 0, value 0."""
    bt, nb = tables(lens, seed)
    kv = np.zeros((2, 2, nkv, 16, d))                     # [K, V][an ordinary block, a sequence's first one]
    kv[1] = 1.0
    kv[0, 1, :, 0, 0] = 6.0
    kv[1, 1, :, 0] = 0.0
    which = np.zeros(nb + 1, int)
    which[bt[:, 0]] = 1
    enc = {"fp4": lambda x: pack_pool(*encode(x, 1.0)), "bf16": round_bf16, "fp8": round_e4m3}[kind]
    k, v = enc(kv[0]), enc(kv[1])
    held = pool_values(v, kind, d, 1.0)[0]
    assert np.ptp(held) == 0
    return to_gpu(k[which]), to_gpu(v[which]), bt, nb, held.max()


def queries(n, nq, d, nats):
    """Channel 0 gives `nats` with the sink's key after the scale 1 / sqrt(d); the others meet only zeros."""
    q = np.random.default_rng(3).standard_normal((n, nq, d)).astype(np.float32)
    q[..., 0] = nats * np.sqrt(d) / 6.0
    return q, float(q[0, 0, 0]) * 6.0 / np.sqrt(d)


def share(n, nats):
    t = n * np.exp(-nats)
    return t / (1 + t)


@pytest.mark.parametrize("n,nats", TAILS)
@pytest.mark.parametrize("rows,nq,nkv,d", [(1, 4, 1, 64), (40, 16, 8, 128), (3, 16, 1, 128)])
def test_single_token_fp4(cuda_lib, rows, nq, nkv, d, n, nats):
    lens = [n + 1] * rows if rows < 40 else [n + 1] + [20] * (rows - 1)
    k, v, bt, nb, one = pools("fp4", lens, nkv, d)
    q, nats = queries(rows, nq, d, nats)
    out = torch.zeros((rows, nq * d), device=DEV)
    capi.op_paged_attention_fp4(dev(q, torch.float32), nkv, k, v, 1.0, 1.0, dev(bt), dev(lens), nb, out)
    for got, size in zip(out.double().cpu().numpy(), lens):
        assert np.abs(got - one * share(size - 1, nats)).max() <= 2e-5 * one


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n,nats", TAILS)
@pytest.mark.parametrize("nq,nkv,d", [(4, 1, 64), (8, 2, 128), (1, 1, 128)])
def test_prompt(cuda_lib, kind, nq, nkv, d, n, nats):
    k, v, bt, nb, one = pools(kind, [n + 1], nkv, d)
    q, nats = queries(3, nq, d, nats)
    out = torch.zeros((3, nq * d), device=DEV)
    capi.op_prompt_attention(dev(q, torch.float32), nkv, dev([0, 3]), dev([n + 1]), k, v, KINDS[kind], 1.0, 1.0, dev(bt), nb, out)
    for i, got in enumerate(out.double().cpu().numpy()):
        assert np.abs(got - one * share(n - 2 + i, nats)).max() <= 2e-5 * one


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,nats", TAILS)
@pytest.mark.parametrize("rows,nq,nkv,d", [(1, 4, 1, 64), (48, 16, 8, 128), (3, 16, 1, 128)])
def test_single_token_bf16_and_e4m3(cuda_lib, kind, rows, nq, nkv, d, n, nats):
    lens = [n + 1] * rows if rows < 40 else [n + 1] + [20] * (rows - 1)
    k, v, bt, nb, one = pools(kind, lens, nkv, d)
    bt[bt < 0] = nb
    q, nats = queries(rows, nq, d, nats)
    out = torch.zeros((rows, nq * d), device=DEV)
    capi.op_paged_attention(dev(q, torch.float32), nkv, k, v, KINDS[kind], 1.0, 1.0, dev(bt), dev(lens), nb, out)
    for got, size in zip(out.double().cpu().numpy(), lens):
        assert np.abs(got - one * share(size - 1, nats)).max() <= 2e-5 * one


@pytest.mark.parametrize("k_scale", [-0.75, 0.0, 2.0 ** -130, 1.5])
def test_single_token_e4m3_takes_any_k_scale(cuda_lib, k_scale):
    """A scale of either sign, 0 and one below fp32's normal range."""
    nq, nkv, d, lens = 8, 2, 64, [37, 1, 300, 64]
    bt, nb = tables(lens, 5)
    bt[bt < 0] = nb
    rng = np.random.default_rng(6)
    k, v = (round_e4m3(rng.standard_normal((nb + 1, nkv, 16, d))) for _ in range(2))
    q = (rng.standard_normal((len(lens), nq, d)) * 0.6).astype(np.float32)
    out = torch.zeros((len(lens), nq * d), device=DEV)
    capi.op_paged_attention(dev(q, torch.float32), nkv, to_gpu(k), to_gpu(v), capi.DTYPE_E4M3, k_scale, 1.25, dev(bt), dev(lens),
                            nb, out)
    vals = pool_values(v, "fp8", d, 1.25)
    ref = rows_attention(q, pool_values(k, "fp8", d, k_scale), vals, bt, np.arange(len(lens)), np.array(lens) - 1)
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 2e-5 * np.abs(vals).max()
