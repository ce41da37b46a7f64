// Kernel-level entry points of attention over selected blocks of the paged KV
// cache (include/mbt_ops.h).
#include "internal.h"
#include "ops_checks.h"
#include "../../include/mbt_ops.h"

using namespace mbt;

namespace {
constexpr int kMostRows = 1 << 30, kMostPicks = 1 << 26, kMostHeads = 1 << 16;   // the kernels' indexes stay ints
bool rows_ok(int n, const int32_t* positions, const int32_t* row_seq, int nseq, int nkv) {
  return n >= 1 && n <= kMostRows && positions && nseq >= 1 && (row_seq || nseq >= n) && nkv >= 1 && nkv <= kMostHeads;
}
}  // namespace

extern "C" {

int op_kv_extend(int nseq, const int32_t* ctx_lens, const int32_t* new_lens, int32_t* bt, int bt_stride, int num_blocks,
                 const int32_t* free_blocks, int nfree, const int32_t* free_at, int n, int32_t* held, int32_t* cu_seqlens,
                 int32_t* positions, int32_t* row_seq, int64_t* slots, int32_t* free_next, uint32_t* err, void* stream) {
  if (nseq < 1 || nseq > kMostRows || !ctx_lens || !new_lens || !table_ok(bt, bt_stride) || num_blocks < 1 || nfree < 0 ||
      (nfree > 0 && !free_blocks) || !free_at || n < 1 || n > kMostRows || !held || !cu_seqlens || !positions || !row_seq || !slots ||
      !free_next)
    return MBT_ERR_BAD_ARG;
  KvExtendArgs a = {};
  a.nseq = nseq; a.ctx_lens = ctx_lens; a.new_lens = new_lens; a.bt = bt; a.bt_stride = bt_stride;
  a.num_blocks = num_blocks; a.free_blocks = free_blocks; a.nfree = nfree; a.free_at = free_at; a.n = n; a.held = held;
  a.cu = cu_seqlens; a.positions = positions; a.row_seq = row_seq; a.slots = slots; a.free_next = free_next; a.err = err;
  return status(launch_kv_extend(a, (cudaStream_t)stream));
}

int op_key_bounds(int n, const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                  int nkv, int d, const void* kpool, int kv_dtype, int num_blocks, int8_t* bounds, float* scales,
                  uint32_t* err, void* stream) {
  if (!rows_ok(n, positions, row_seq, nseq, nkv) || !table_ok(bt, bt_stride) || (d != 64 && d != 128) || !kpool ||
      !cache_ok(kv_dtype) || num_blocks < 1 || !bounds || !scales || !aligned16(kpool) || !aligned16(bounds))
    return MBT_ERR_BAD_ARG;
  int sms = 0;
  const int rc = device_setup(&sms);
  if (rc != MBT_OK) return rc;
  KeyBoundsArgs a = {};
  a.n = n; a.positions = positions; a.row_seq = row_seq; a.nseq = nseq; a.bt = bt; a.bt_stride = bt_stride; a.nkv = nkv;
  a.d = d; a.kpool = kpool; a.kv = kv_type(kv_dtype); a.num_blocks = num_blocks; a.bounds = bounds; a.scales = scales;
  a.err = err;
  return status(launch_key_bounds(a, sms, (cudaStream_t)stream));
}

size_t op_block_select_scratch(int n, int nkv, int bt_stride, int k) {
  int sms = 0;
  BlockSelectArgs a = {};
  a.n = n; a.nkv = nkv; a.bt_stride = bt_stride; a.k = k;
  if (n < 1 || n > kMostRows || nkv < 1 || nkv > kMostHeads || bt_stride < 1 || bt_stride > kMostPicks || k < 1 || k > kMostPicks ||
      device_setup(&sms) != MBT_OK || block_select_plan(&a, sms) != cudaSuccess)
    return 0;
  return block_select_scratch(a);
}

int op_block_select(int n, const float* q, int nq, int nkv, int d, const int8_t* bounds, const float* scales,
                    const int32_t* positions, const int32_t* row_seq, int nseq, const int32_t* bt, int bt_stride,
                    int num_blocks, int keep_first, int keep_last, int k, int32_t* sel, void* scratch, size_t scratch_bytes,
                    uint32_t* err, void* stream) {
  if (!rows_ok(n, positions, row_seq, nseq, nkv) || !q || !heads_ok(nq, nkv, d) || !bounds || !scales ||
      !table_ok(bt, bt_stride) || num_blocks < 1 || keep_first < 0 || keep_last < 1 ||
      (long long)keep_first + keep_last > k || k > kMostPicks || !sel || !aligned16(q) || !aligned16(bounds) || !aligned16(scratch))
    return MBT_ERR_BAD_ARG;
  int sms = 0;
  const int rc = device_setup(&sms);
  if (rc != MBT_OK) return rc;
  BlockSelectArgs a = {};
  a.n = n; a.q = q; a.nq = nq; a.nkv = nkv; a.d = d; a.bounds = bounds; a.scales = scales; a.positions = positions;
  a.row_seq = row_seq; a.nseq = nseq; a.bt = bt; a.bt_stride = bt_stride; a.num_blocks = num_blocks;
  a.keep_first = keep_first; a.keep_last = keep_last; a.k = k; a.sel = sel; a.err = err;
  if (block_select_plan(&a, sms) != cudaSuccess) return MBT_ERR_BAD_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t bytes = block_select_scratch(a);
  if (!bytes || scratch)
    return scratch_bytes < bytes ? MBT_ERR_SCRATCH : status(launch_block_select(a, scratch, sms, s));
  if (cudaMallocAsync(&scratch, bytes, s) != cudaSuccess) return MBT_ERR_OOM;
  const int done = status(launch_block_select(a, scratch, sms, s));
  const cudaError_t freed = cudaFreeAsync(scratch, s);
  return done != MBT_OK ? done : status(freed);
}

int op_block_attention(int n, const float* q, int nq, int nkv, int d, const void* kpool, const void* vpool, int kv_dtype,
                       float k_scale, float v_scale, const int32_t* positions, const int32_t* row_seq, int nseq,
                       const int32_t* bt, int bt_stride, const int32_t* sel, int k, int num_blocks, float* out,
                       uint32_t* err, void* stream) {
  if (!rows_ok(n, positions, row_seq, nseq, nkv) || !q || !heads_ok(nq, nkv, d) || !kpool || !vpool || !cache_ok(kv_dtype) ||
      !scale_ok(k_scale) || !scale_ok(v_scale) || !table_ok(bt, bt_stride) || !sel || k < 1 || k > kMostPicks || num_blocks < 1 || !out ||
      !aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out))
    return MBT_ERR_BAD_ARG;
  int sms = 0;
  const int rc = device_setup(&sms);
  if (rc != MBT_OK) return rc;
  BlockAttnArgs a = {};
  a.n = n; a.q = q; a.nq = nq; a.nkv = nkv; a.d = d; a.kv = kv_type(kv_dtype); a.kpool = kpool; a.vpool = vpool;
  a.k_scale = k_scale; a.v_scale = v_scale; a.positions = positions; a.row_seq = row_seq; a.nseq = nseq; a.bt = bt;
  a.bt_stride = bt_stride; a.sel = sel; a.k = k; a.num_blocks = num_blocks; a.out = out; a.err = err;
  return status(launch_block_attention(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
