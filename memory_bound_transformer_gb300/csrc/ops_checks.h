// Argument checks that the entry points of the paged cache's operators share.
#pragma once

#include <stdint.h>

#include <cuda_runtime.h>

#include "../../include/mbt.h"
#include "internal.h"

namespace mbt {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
// A tensor's scale. Beyond these its products with block scales, queries and
// their reciprocals could leave fp32's range.
inline bool scale_ok(float s) { return s >= 0x1p-64f && s <= 0x1p64f; }
// A row of a block table: its token count, rounded up to tiles, stays an int.
inline bool table_ok(const int32_t* bt, int bt_stride) { return bt && bt_stride >= 1 && bt_stride <= (1 << 26); }
// Heads and head size that the cache's kernels take.
inline bool heads_ok(int nq, int nkv, int d) {
  return nq >= 1 && nkv >= 1 && nq % nkv == 0 && nq / nkv <= 16 && (d == 64 || d == 128);
}
inline bool cache_ok(int kv_dtype) {
  return kv_dtype == (int)MBT_DTYPE_BF16 || kv_dtype == (int)MBT_DTYPE_E4M3 || kv_dtype == (int)MBT_DTYPE_E2M1;
}
inline int kv_type(int kv_dtype) {
  return kv_dtype == (int)MBT_DTYPE_BF16 ? KV_BF16 : kv_dtype == (int)MBT_DTYPE_E4M3 ? KV_E4M3 : KV_FP4;
}
inline int status(cudaError_t e) {
  if (e == cudaSuccess) return MBT_OK;
  return e == cudaErrorInvalidValue ? MBT_ERR_BAD_ARG : MBT_ERR_CUDA;
}
// SM count of the current device; the kernels' shared-memory limits are raised
// once per device (ops_fp4.cu).
int device_setup(int* sms);

}  // namespace mbt
