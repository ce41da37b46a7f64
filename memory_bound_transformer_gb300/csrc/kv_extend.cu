// Block tables and row layout for a step's new tokens, from the sequences'
// lengths alone: sequence s with ctx_s cached and new_s new tokens needs
//   need_s = ceil((ctx_s + new_s) / 16) - ceil(ctx_s / 16)
// blocks, which are those of the free list behind the ones that sequences before
// it need, and its rows stand behind theirs: two prefix sums, and a third over
// the sequences that fit ("Kernels, Fusion & CUDA Graphs", "The serving engine's
// kernel stack": block tables of the paged cache).
#include "common.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;

__device__ __forceinline__ int blocks_for(long long tokens) { return (int)((tokens + kBlockTokens - 1) / kBlockTokens); }

// Inclusive sum over the CTA's threads; `total` is the last one's. scratch: 33 entries.
__device__ __forceinline__ long long block_scan(long long v, long long* scratch, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  total = scratch[31];
  return v + (warp ? scratch[warp - 1] : 0);
}

// Last entry of the non-decreasing edge[0 .. n] that is <= x, for edge[0] <= x < edge[n].
__device__ __forceinline__ int segment_of(const int* edge, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (edge[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One CTA: tables, lengths and row edges, 1024 sequences at a time. What a
// sequence reads of arrays that may be written in place it reads before.
__global__ void __launch_bounds__(kPlanThreads) kv_extend_kernel(const KvExtendArgs a) {
  __shared__ long long scratch[33];
  __shared__ int took_edge[kPlanThreads + 1], sm_seq[kPlanThreads];
  const int tid = threadIdx.x;
  const int at0 = *a.free_at;
  const bool at_ok = at0 >= 0 && at0 <= a.nfree;
  if (!at_ok && tid == 0) set_err(a.err, MBT_DEV_BLOCK_RANGE);
  long long needed = 0, asked = 0, rows = 0, taken = 0;
  if (tid == 0) a.cu[0] = 0;
  for (int s0 = 0; s0 < a.nseq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const bool in = s < a.nseq;
    const int ctx = in ? a.ctx_lens[s] : 0;
    int add = in ? a.new_lens[s] : 0;
    if (ctx < 0 || add < 0 || (long long)ctx + add > (long long)a.bt_stride * kBlockTokens) {
      set_err(a.err, MBT_DEV_SEQLEN_RANGE);
      add = 0;
    }
    const int have = blocks_for(ctx);
    int need = add ? blocks_for((long long)ctx + add) - have : 0;
    long long t0, t1, t2;
    const long long need_end = needed + block_scan(need, scratch, t0);
    const long long ask_end = asked + block_scan(add, scratch, t1);
    needed += t0;
    asked += t1;
    if (add && ask_end > a.n) {
      set_err(a.err, MBT_DEV_POS_RANGE);
      add = need = 0;
    } else if (need && (!at_ok || at0 + need_end > a.nfree)) {
      set_err(a.err, MBT_DEV_BLOCK_RANGE);
      add = need = 0;
    }
    // those that fit need the first blocks of the list: what others ask lies behind
    const long long row_end = rows + block_scan(add, scratch, t1), took_end = block_scan(need, scratch, t2);
    if (in) {
      a.held[s] = ctx + add;
      a.cu[s + 1] = (int)row_end;
    }
    rows += t1;
    took_edge[tid + 1] = (int)took_end;
    sm_seq[tid] = have;
    if (tid == 0) took_edge[0] = 0;
    __syncthreads();
    for (int i = tid; i < (int)t2; i += kPlanThreads) {
      const int q = segment_of(took_edge, kPlanThreads, i), id = a.free_blocks[at0 + taken + i];
      if (id < 0 || id > a.num_blocks) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      a.bt[(size_t)(s0 + q) * a.bt_stride + sm_seq[q] + i - took_edge[q]] = id;
    }
    taken += t2;
    __syncthreads();
  }
  if (tid == 0) *a.free_next = at0 + (int)taken;
}

// The packed rows, one per thread.
__global__ void __launch_bounds__(kRowThreads) kv_rows_kernel(const KvExtendArgs a) {
  const int i = blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= a.n) return;
  int seq = a.nseq, pos = 0;
  long long slot = (long long)a.num_blocks * kBlockTokens;
  if (i < a.cu[a.nseq]) {
    seq = segment_of(a.cu, a.nseq, i);
    pos = a.held[seq] - a.cu[seq + 1] + i;
    const int blk = a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens];
    const bool ok = blk >= 0 && blk <= a.num_blocks;
    if (!ok) set_err(a.err, MBT_DEV_BLOCK_RANGE);
    slot = ok ? (long long)blk * kBlockTokens + pos % kBlockTokens : -1;
  }
  a.positions[i] = pos;
  a.row_seq[i] = seq;
  a.slots[i] = slot;
}

}  // namespace

cudaError_t launch_kv_extend(const KvExtendArgs& a, cudaStream_t s) {
  kv_extend_kernel<<<1, kPlanThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  kv_rows_kernel<<<(unsigned)((a.n + (long long)kRowThreads - 1) / kRowThreads), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mbt
