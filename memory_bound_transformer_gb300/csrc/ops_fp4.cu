// Kernel-level entry points of the 4-bit paged KV cache and of prompt
// attention (include/mbt_ops.h).
#include <algorithm>
#include <cmath>
#include <mutex>
#include <new>
#include <vector>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"
#include "ops_checks.h"
#include "../../include/mbt_ops.h"

namespace mbt {
// SM count of the current device; the kernels' shared-memory limits are raised
// once per device.
int device_setup(int* sms) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static int known[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MBT_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!known[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MBT_ERR_NO_DEVICE;
    if (attn_fp4_init() != cudaSuccess || prompt_attention_init() != cudaSuccess || block_select_init() != cudaSuccess ||
        block_attention_init() != cudaSuccess)
      return MBT_ERR_CUDA;
    known[dev] = n;
  }
  *sms = known[dev];
  return MBT_OK;
}
}  // namespace mbt

using namespace mbt;

extern "C" {

size_t op_kv_unit_bytes(int d, int kv_dtype) {
  if (d != 64 && d != 128) return 0;
  if (kv_dtype == MBT_DTYPE_BF16) return (size_t)kBlockTokens * d * 2;
  if (kv_dtype == MBT_DTYPE_E4M3) return (size_t)kBlockTokens * d;
  return kv_dtype == MBT_DTYPE_E2M1 ? (size_t)fp4_unit_bytes(d) : 0;
}

int op_rope_table(int max_pos, int d, float theta, float* table, void* stream) {
  if (max_pos < 1 || (d != 64 && d != 128) || !(theta > 1.f) || !std::isfinite(theta) || !table) return MBT_ERR_BAD_ARG;
  const int half = d / 2;
  float* host = new (std::nothrow) float[(size_t)max_pos * d];
  if (!host) return MBT_ERR_OOM;
  for (int i = 0; i < half; ++i) {
    const double w = std::pow((double)theta, -2.0 * i / (double)d);
    for (int p = 0; p < max_pos; ++p) {
      host[(size_t)p * d + 2 * i] = (float)std::cos((double)p * w);
      host[(size_t)p * d + 2 * i + 1] = (float)std::sin((double)p * w);
    }
  }
  cudaStream_t s = (cudaStream_t)stream;
  int rc = cudaMemcpyAsync(table, host, (size_t)max_pos * d * sizeof(float), cudaMemcpyHostToDevice, s) == cudaSuccess
               ? MBT_OK : MBT_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) rc = MBT_ERR_CUDA;
  delete[] host;
  return rc;
}

int op_rope_kv_write_fp4(int n, const float* qkv, int ld_qkv, int nq, int nkv, int d, const int32_t* positions,
                         const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride, const float* rope,
                         int max_pos, void* kpool, void* vpool, int num_blocks, float k_scale, float v_scale,
                         float* q_out, uint32_t* err, void* stream) {
  if (n < 1 || !qkv || nq < 1 || nkv < 1 || (d != 64 && d != 128) || !positions || nseq < 1 || (!row_seq && nseq < n) ||
      !table_ok(bt, bt_stride) || !rope || max_pos < 1 || !kpool || !vpool || num_blocks < 1 || !q_out ||
      !scale_ok(k_scale) || !scale_ok(v_scale))
    return MBT_ERR_BAD_ARG;
  if (ld_qkv % 4 || (long long)ld_qkv < ((long long)nq + 2LL * nkv) * d || !aligned16(qkv) || !aligned16(rope) ||
      !aligned16(kpool) || !aligned16(vpool) || !aligned16(q_out))
    return MBT_ERR_BAD_ARG;
  RopeKvFp4Args a = {};
  a.n = n; a.qkv = qkv; a.ld_qkv = ld_qkv; a.nq = nq; a.nkv = nkv; a.d = d;
  a.positions = positions; a.row_seq = row_seq; a.nseq = nseq; a.bt = bt; a.bt_stride = bt_stride;
  a.rope = rope; a.max_pos = max_pos; a.kpool = kpool; a.vpool = vpool; a.num_blocks = num_blocks;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.inv6_k = (float)(1.0 / (6.0 * (double)k_scale)); a.inv6_v = (float)(1.0 / (6.0 * (double)v_scale));
  a.q_out = q_out; a.err = err;
  return status(launch_rope_kv_write_fp4(a, (cudaStream_t)stream));
}

int op_kv_read_fp4(int n, const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                   int nkv, int d, const void* kpool, const void* vpool, int num_blocks, float k_scale, float v_scale,
                   float* k_out, float* v_out, uint32_t* err, void* stream) {
  if (n < 1 || !positions || nseq < 1 || (!row_seq && nseq < n) || !table_ok(bt, bt_stride) || nkv < 1 ||
      (d != 64 && d != 128) || !kpool || !vpool || num_blocks < 1 || !scale_ok(k_scale) || !scale_ok(v_scale) ||
      !k_out || !v_out)
    return MBT_ERR_BAD_ARG;
  if (!aligned16(kpool) || !aligned16(vpool) || !aligned16(k_out) || !aligned16(v_out)) return MBT_ERR_BAD_ARG;
  KvReadFp4Args a = {};
  a.n = n; a.positions = positions; a.row_seq = row_seq; a.nseq = nseq; a.bt = bt; a.bt_stride = bt_stride;
  a.nkv = nkv; a.d = d; a.kpool = kpool; a.vpool = vpool; a.num_blocks = num_blocks; a.k_scale = k_scale;
  a.v_scale = v_scale; a.k_out = k_out; a.v_out = v_out; a.err = err;
  return status(launch_kv_read_fp4(a, (cudaStream_t)stream));
}

int op_paged_attention_fp4(int B, const float* q, int nq, int nkv, int d, const void* kpool, const void* vpool,
                           float k_scale, float v_scale, const int32_t* bt, int bt_stride, const int32_t* seq_lens,
                           int num_blocks, float* out, uint32_t* err, void* stream) {
  if (B < 1 || !q || !heads_ok(nq, nkv, d) || !kpool || !vpool || !scale_ok(k_scale) || !scale_ok(v_scale) ||
      !table_ok(bt, bt_stride) || !seq_lens || num_blocks < 1 || !out)
    return MBT_ERR_BAD_ARG;
  if (!aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out)) return MBT_ERR_BAD_ARG;
  int sms = 0;
  const int rc = device_setup(&sms);
  if (rc != MBT_OK) return rc;
  AttnFp4Args a = {};
  a.B = B; a.q = q; a.nq = nq; a.nkv = nkv; a.d = d; a.kpool = kpool; a.vpool = vpool;
  a.k_scale = k_scale; a.v_scale = v_scale; a.bt = bt; a.bt_stride = bt_stride; a.seq_lens = seq_lens;
  a.num_blocks = num_blocks; a.out = out; a.err = err;
  if (attn_fp4_plan(&a, sms) != cudaSuccess) return MBT_ERR_BAD_ARG;
  return status(launch_attention_fp4(a, (cudaStream_t)stream));
}

int op_prompt_attention(int n, const float* q, int nq, int nkv, int d, int nseq, const int32_t* cu_seqlens,
                        const int32_t* ctx_lens, const void* kpool, const void* vpool, int kv_dtype, float k_scale,
                        float v_scale, const int32_t* bt, int bt_stride, int num_blocks, float* out, uint32_t* err,
                        void* stream) {
  if (n < 1 || !q || !heads_ok(nq, nkv, d) || nseq < 1 || !cu_seqlens || !ctx_lens || !kpool || !vpool ||
      !scale_ok(k_scale) || !scale_ok(v_scale) || !table_ok(bt, bt_stride) || num_blocks < 1 || !out)
    return MBT_ERR_BAD_ARG;
  if (!cache_ok(kv_dtype)) return MBT_ERR_BAD_ARG;
  if (!aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out)) return MBT_ERR_BAD_ARG;
  int sms = 0;
  const int rc = device_setup(&sms);
  if (rc != MBT_OK) return rc;
  PromptArgs a = {};
  a.n = n; a.q = q; a.nq = nq; a.nkv = nkv; a.d = d; a.kpool = kpool; a.vpool = vpool;
  a.kv = kv_type(kv_dtype);
  a.k_scale = k_scale; a.v_scale = v_scale; a.nseq = nseq; a.cu = cu_seqlens; a.lens = ctx_lens; a.bt = bt;
  a.bt_stride = bt_stride; a.num_blocks = num_blocks; a.out = out; a.err = err;
  return status(launch_prompt_attention(a, (cudaStream_t)stream));
}

}  // extern "C"
