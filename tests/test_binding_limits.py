"""Sizes beyond 32 bits never reach the library: ctypes would pass what is left of them."""
import pytest
import torch

from memory_bound_transformer_gb300 import capi


@pytest.mark.parametrize("shape", [(1, 2 ** 32 + 3), (2 ** 31, 1)])
def test_dimensions(shape):
    with pytest.raises(ValueError, match="2\\^31"):
        capi._shape("op", "bt", torch.empty(shape, dtype=torch.int32, device="meta"), 2)
    assert capi._shape("op", "bt", torch.empty((1, 2 ** 31 - 1), dtype=torch.int32, device="meta"), 2)[1] == 2 ** 31 - 1


@pytest.mark.parametrize("nkv,d,num_blocks,kind", [
    (2, 64, 5 - 2 ** 32, capi.DTYPE_E2M1), (2, 64, 5, capi.DTYPE_E4M3 + 2 ** 32), (2 - 2 ** 32, 64, 5, capi.DTYPE_E2M1),
    (2, 64 + 2 ** 32, 5, capi.DTYPE_E2M1), (2, 64, 0, capi.DTYPE_E2M1), (0, 64, 5, capi.DTYPE_E2M1), (2, 96, 5, capi.DTYPE_E2M1)])
def test_pool_sizes(nkv, d, num_blocks, kind):
    pool = torch.zeros(6 * 2 * 1152, dtype=torch.uint8)
    with pytest.raises(capi.MbtError) as e:
        capi._pools("op", pool, pool, 0, nkv, d, num_blocks, kind)
    assert e.value.code == -1


@pytest.mark.gpu
def test_row_stride(cuda_lib):
    """Rows 2^32 + 384 values apart are not rows of 384 values."""
    nq, nkv, d = 2, 2, 64
    stride = 2 ** 32 + (nq + 2 * nkv) * d
    qkv = torch.empty(stride + 384, device="cuda").as_strided((2, 384), (stride, 1))
    i = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    pool = torch.zeros(6 * 2 * 576, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        capi.op_rope_kv_write_fp4(qkv, nq, nkv, d, i[:, 0].contiguous(), i, torch.zeros((4, d // 2, 2), device="cuda"), pool, pool,
                                  5, 1.0, 1.0, torch.zeros((2, nq, d), device="cuda"))
