// Softmax attention over selected blocks of the paged KV cache:
//   o_h = sum_t softmax_t(q_h . K_t / sqrt(d)) V_t   over the tokens t <= p of the
// blocks chosen for the row and the KV head of h, one pass with the running
// maximum and sum of the softmax.
#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kBaThreads = 128;

// Values of D / 32 neighbouring channels of a token, before the tensor's scale.
template <int D, int KV>
__device__ __forceinline__ void values(const unsigned char* unit, int token, int lane, float (&x)[D / 32]) {
  constexpr int N = D / 32;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = lane * N + i;
    if constexpr (KV == KV_BF16) {
      x[i] = __bfloat162float(reinterpret_cast<const bf16*>(unit)[token * D + c]);
    } else if constexpr (KV == KV_E4M3) {
      x[i] = e4m3_to_f32(unit[token * D + c]);
    } else {
      const uint32_t code = unit[token * (D / 2) + c / 2] >> (4 * (c & 1)) & 15u;
      uint32_t p[2];
      e2m1x4_to_h2(code, p);
      x[i] = h2_to_float2(p[0]).x * e4m3_to_f32(unit[kBlockTokens * (D / 2) + token * (D / kFp4Group) + c / kFp4Group]);
    }
  }
}

// A CTA per (row, KV head), a warp per query head in turn, a lane per D / 32 channels.
template <int D, int KV>
__global__ void __launch_bounds__(kBaThreads) block_attention_kernel(const BlockAttnArgs a) {
  constexpr int N = D / 32;
  constexpr size_t UNIT = KV == KV_BF16 ? kBlockTokens * D * 2 : KV == KV_E4M3 ? kBlockTokens * D : fp4_unit_bytes(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = (int)(blockIdx.x % (unsigned)a.nkv), row = (int)(blockIdx.x / (unsigned)a.nkv), G = a.nq / a.nkv;
  const int pos = a.positions[row], seq = a.row_seq ? a.row_seq[row] : row;
  const bool ok = pos >= 0 && pos / kBlockTokens < a.bt_stride && seq >= 0 && seq < a.nseq;
  if (!ok && h == 0 && threadIdx.x == 0) set_err(a.err, MBT_DEV_POS_RANGE);
  const int* sel = a.sel + (size_t)blockIdx.x * a.k;
  for (int g = warp; g < G; g += kBaThreads / 32) {
    const size_t at = ((size_t)row * a.nq + (size_t)h * G + g) * D + lane * N;
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) { q[i] = a.q[at + i]; o[i] = 0.f; }
    for (int j = 0; ok && j < a.k; ++j) {
      const int e = sel[j];
      if (e < 0) continue;
      if (e > pos / kBlockTokens) { set_err(a.err, MBT_DEV_BLOCK_RANGE); continue; }
      int id = a.bt[(size_t)seq * a.bt_stride + e];
      if (id < 0 || id > a.num_blocks) { set_err(a.err, MBT_DEV_BLOCK_RANGE); id = a.num_blocks; }
      const size_t off = ((size_t)id * a.nkv + h) * UNIT;
      const int live = min(kBlockTokens, pos - e * kBlockTokens + 1);
      float s[kBlockTokens], mn = m, x[N];
#pragma unroll
      for (int t = 0; t < kBlockTokens; ++t) {
        s[t] = 0.f;
        values<D, KV>(reinterpret_cast<const unsigned char*>(a.kpool) + off, min(t, live - 1), lane, x);
#pragma unroll
        for (int i = 0; i < N; ++i) s[t] = fmaf(q[i], x[i], s[t]);
        s[t] = warp_sum(s[t]) * (a.k_scale / sqrtf((float)D));
        s[t] += s[t] - s[t];                                         // an infinite score is no score: NaN
        if (t >= live) s[t] = -INFINITY;
        mn = fmaxf(mn, s[t]);
      }
      // a block's sums on their own first: long sums of equal shares would round one way
      const float f = expf(m - mn);
      float lb = 0.f, ob[N] = {};
#pragma unroll
      for (int t = 0; t < kBlockTokens; ++t) {
        if (t >= live) continue;
        const float p = expf(s[t] - mn);
        lb += p;
        values<D, KV>(reinterpret_cast<const unsigned char*>(a.vpool) + off, t, lane, x);
#pragma unroll
        for (int i = 0; i < N; ++i) ob[i] += p * x[i];
      }
      m = mn;
      l = l * f + lb;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = o[i] * f + ob[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) a.out[at + i] = l == 0.f ? 0.f : o[i] * (a.v_scale / l);
  }
}

}  // namespace

cudaError_t launch_block_attention(const BlockAttnArgs& a, cudaStream_t s) {
  const long long grid = (long long)a.n * a.nkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)grid, kBaThreads, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.d == 64)
    return a.kv == KV_BF16 ? go(block_attention_kernel<64, KV_BF16>) : a.kv == KV_E4M3 ? go(block_attention_kernel<64, KV_E4M3>)
                                                                                       : go(block_attention_kernel<64, KV_FP4>);
  return a.kv == KV_BF16 ? go(block_attention_kernel<128, KV_BF16>) : a.kv == KV_E4M3 ? go(block_attention_kernel<128, KV_E4M3>)
                                                                                      : go(block_attention_kernel<128, KV_FP4>);
}

}  // namespace mbt
