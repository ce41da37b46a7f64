// Attention of query rows over a paged KV cache (BF16, e4m3 or 4-bit), one
// warp per (row, query head): the plain form of
//   o = sum_t softmax_t(q . K_t / sqrt(d)) V_t   over the row's t < limit
// with the running maximum and sum of a one-pass softmax, fp32 throughout.
// Row i of a packed prompt at position p attends over t <= p; a decode row
// over t < its sequence's length.
#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kRowsThreads = 128;

// V consecutive channels (from channel V * lane) of token slot `slot` of a unit.
template <int D, int KV>
__device__ __forceinline__ void load_vals(const unsigned char* unit, int slot, int lane, float (&v)[D / 32]) {
  constexpr int V = D / 32;
  if (KV == KV_FP4) {
    const float s = e4m3_to_f32(unit[kBlockTokens * (D / 2) + slot * (D / kFp4Group) + lane * V / kFp4Group]);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      uint32_t h[4];
      e2m1x8_to_h2(unit[slot * (D / 2) + (lane * V + i) / 2], h);
      const float2 f = h2_to_float2(h[0]);
      v[i] = f.x * s;
      v[i + 1] = f.y * s;
    }
  } else if (KV == KV_E4M3) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e4m3_to_f32(unit[slot * D + lane * V + i]);
  } else {
    const uint16_t* u = reinterpret_cast<const uint16_t*>(unit) + slot * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float((uint32_t)u[i] << 16);
  }
}

template <int D, int KV>
__global__ void __launch_bounds__(kRowsThreads) attention_rows_kernel(const RowsAttnArgs a) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)a.n * a.nq) return;
  const int row = (int)(item / a.nq), head = (int)(item % a.nq), h = head / (a.nq / a.nkv);
  int seq = -1, limit = 0;
  bool bad = false;
  if (a.cu) {
    for (int s = 0; s < a.nseq; ++s) {
      const int lo = a.cu[s], hi = a.cu[s + 1];
      if (row >= lo && row < hi) { seq = s; limit = a.lens[s] - (hi - lo) + (row - lo) + 1; break; }
    }
    if (seq < 0) return;                                // rows of no sequence stay as they are
    bad = a.lens[seq] < 0 || a.lens[seq] > (long long)a.bt_stride * kBlockTokens;
  } else {
    seq = row;
    limit = a.lens[row];
    bad = limit < 1 || limit > (long long)a.bt_stride * kBlockTokens;
  }
  if (bad) {
    if (lane == 0) set_err(a.err, MBT_DEV_SEQLEN_RANGE);
    limit = 0;
  }
  const size_t ub = KV == KV_FP4 ? fp4_unit_bytes(D) : (size_t)kBlockTokens * D * (KV == KV_E4M3 ? 1 : 2);
  float q[V], o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    q[i] = a.q[((size_t)row * a.nq + head) * D + lane * V + i] * (1.4426950408889634f / sqrtf((float)D) * a.k_scale);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < limit; ++t) {
    int blk = a.bt[(size_t)seq * a.bt_stride + t / kBlockTokens];
    if (blk < 0 || blk > a.num_blocks) {
      if (lane == 0) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      blk = a.num_blocks;
    }
    const size_t off = ((size_t)blk * a.nkv + h) * ub;
    float k[V], v[V];
    load_vals<D, KV>(reinterpret_cast<const unsigned char*>(a.kpool) + off, t % kBlockTokens, lane, k);
    load_vals<D, KV>(reinterpret_cast<const unsigned char*>(a.vpool) + off, t % kBlockTokens, lane, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += q[i] * k[i];
    s = warp_sum(s);
    const float mn = fmaxf(m, s), mu = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(m - mu), p = exp2f(s - mu);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * al + p * v[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    a.out[((size_t)row * a.nq + head) * D + lane * V + i] = limit > 0 ? o[i] / l * a.v_scale : 0.f;
}

template <int D>
void rows_launch(const RowsAttnArgs& a, unsigned grid, cudaStream_t s) {
  if (a.kv == KV_FP4) attention_rows_kernel<D, KV_FP4><<<grid, kRowsThreads, 0, s>>>(a);
  else if (a.kv == KV_E4M3) attention_rows_kernel<D, KV_E4M3><<<grid, kRowsThreads, 0, s>>>(a);
  else attention_rows_kernel<D, KV_BF16><<<grid, kRowsThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_attention_rows(const RowsAttnArgs& a, cudaStream_t s) {
  const long long items = (long long)a.n * a.nq;
  const long long grid = (items + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.d == 64) rows_launch<64>(a, (unsigned)grid, s);
  else rows_launch<128>(a, (unsigned)grid, s);
  return cudaGetLastError();
}

}  // namespace mbt
