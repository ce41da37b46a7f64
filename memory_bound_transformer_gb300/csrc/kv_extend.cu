// Block tables and row layout for a step's new tokens, from the sequences'
// lengths alone: sequence s with ctx_s cached and new_s new tokens needs
//   need_s = ceil((ctx_s + new_s) / 16) - ceil(ctx_s / 16)
// blocks, which are those of the free list behind the ones that sequences before
// it need, and its rows stand behind theirs: two prefix sums, and the same over
// those that fit where not all do ("Kernels, Fusion & CUDA Graphs", "The serving
// engine's kernel stack": block tables of the paged cache).
//
// Each CTA computes the sums, which costs less than a second launch or handing them
// over, and lays out its share of the rows; the row that begins a block enters it
// into the table. Where lengths are updated in place the CTAs are one cluster of up
// to eight, and none writes before all have read. Bound by latency (lengths, sums, a
// free or table entry per row). In a graph, us: 64 sequences by a token each 2.2;
// 512 by 65 k rows 3.9 (in place 9.4; one CTA for the sums and tables and a grid
// for the rows 9.1, and 2.5 more of the caller's time).
#include "common.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kPlanThreads = 1024;           // most threads of a CTA, a sequence each at a time
// Most CTAs. In a graph, us, with 1, 8, 32, 128 and 256 CTAs: 512 sequences by 32 tokens
// 14.5, 4.1, 3.8, 3.9, 4.6, by 128 49, 8.8, 4.2, 3.9, 5.7; 16 by 16384 197, 28, 10, 5.1, 8.0.
constexpr int kPlanGrid = 128;
constexpr int kPlanCluster = 8;              // in place, portable clusters: 512 by 128 with 1, 2, 4, 8 CTAs 50, 27, 15, 9.4
constexpr int kPlanRows = 2;                 // rows of a thread at a time (four: 1024 rows 4.9 us against 4.4)

__device__ __forceinline__ int blocks_for(long long tokens) { return (int)((tokens + kBlockTokens - 1) / kBlockTokens); }

struct Pair { long long x, y; };
// Inclusive sums over the CTA's threads; `total` are the last one's. scratch: 32 entries.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* scratch, Pair& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto scan = [&](Pair p) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, p.x, o), y = __shfl_up_sync(0xffffffffu, p.y, o);
      if (lane >= o) { p.x += x; p.y += y; }
    }
    return p;
  };
  v = scan(v);
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  const Pair w = scan(lane < warps ? scratch[lane] : Pair{0, 0});     // every warp for itself
  total.x = __shfl_sync(0xffffffffu, w.x, 31);
  total.y = __shfl_sync(0xffffffffu, w.y, 31);
  const long long x = __shfl_sync(0xffffffffu, w.x, max(warp - 1, 0)), y = __shfl_sync(0xffffffffu, w.y, max(warp - 1, 0));
  if (warp) { v.x += x; v.y += y; }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) kv_extend_kernel(const KvExtendArgs a) {
  __shared__ Pair scratch[32];
  __shared__ int took_edge[kPlanThreads + 1], row_edge[kPlanThreads + 1], sm_have[kPlanThreads], sm_ctx[kPlanThreads];
  const int tid = threadIdx.x, threads = blockDim.x, rank = blockIdx.x;
  // Comes to wait itself, but lets no successor start early: attention may read
  // tables and lengths before it waits.
  pdl_wait();
  const int at0 = *a.free_at;
  const bool at_ok = at0 >= 0 && at0 <= a.nfree;
  if (!at_ok && tid == 0) set_err(a.err, MBT_DEV_BLOCK_RANGE);
  long long needed = 0, asked = 0, rows = 0, taken = 0;
  if (tid == 0) took_edge[0] = row_edge[0] = 0;
  for (int s0 = 0; s0 < a.nseq; s0 += threads) {
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
    Pair total;
    const Pair end = block_scan(Pair{need, add}, scratch, total);     // blocks and rows up to this sequence
    // those that fit get the first blocks of the list: what others ask lies behind
    Pair got = end, got_total = total;
    if (asked + total.y > a.n || !at_ok || at0 + needed + total.x > a.nfree) {
      if (add && asked + end.y > a.n) {
        set_err(a.err, MBT_DEV_POS_RANGE);
        add = need = 0;
      } else if (need && (!at_ok || at0 + needed + end.x > a.nfree)) {
        set_err(a.err, MBT_DEV_BLOCK_RANGE);
        add = need = 0;
      }
      got = block_scan(Pair{need, add}, scratch, got_total);
    }
    took_edge[tid + 1] = (int)got.x;
    row_edge[tid + 1] = (int)got.y;
    sm_have[tid] = have;
    sm_ctx[tid] = ctx;
    if (a.in_place) cluster_sync_all();                               // every CTA has read these sequences
    else __syncthreads();
    if (in && rank == 0) {
      a.held[s] = ctx + add;
      a.cu[s + 1] = (int)(rows + got.y);
    }
    const int count = (int)got_total.y, stride = threads * gridDim.x;
    for (int i0 = rank * threads + tid; i0 < count; i0 += kPlanRows * stride) {
      int q[kPlanRows], id[kPlanRows];                                // the row's sequence: the last edge <= the row
#pragma unroll
      for (int u = 0; u < kPlanRows; ++u) q[u] = 0;
      for (int step = threads >> 1; step > 0; step >>= 1)
#pragma unroll
        for (int u = 0; u < kPlanRows; ++u)
          if (row_edge[q[u] + step] <= i0 + u * stride) q[u] += step;
#pragma unroll
      for (int u = 0; u < kPlanRows; ++u) {
        const int i = i0 + u * stride, pos = sm_ctx[q[u]] + i - row_edge[q[u]], b = pos / kBlockTokens;
        if (i >= count) continue;
        id[u] = b >= sm_have[q[u]] ? a.free_blocks[at0 + taken + took_edge[q[u]] + b - sm_have[q[u]]]
                                   : a.bt[(size_t)(s0 + q[u]) * a.bt_stride + b];
      }
#pragma unroll
      for (int u = 0; u < kPlanRows; ++u) {
        const int i = i0 + u * stride, pos = sm_ctx[q[u]] + i - row_edge[q[u]], b = pos / kBlockTokens;
        if (i >= count) continue;
        const bool ok = id[u] >= 0 && id[u] <= a.num_blocks;
        if (!ok) set_err(a.err, MBT_DEV_BLOCK_RANGE);
        if (b >= sm_have[q[u]] && pos % kBlockTokens == 0) a.bt[(size_t)(s0 + q[u]) * a.bt_stride + b] = id[u];
        const int row = (int)rows + i;
        a.positions[row] = pos;
        a.row_seq[row] = s0 + q[u];
        a.slots[row] = ok ? (long long)id[u] * kBlockTokens + pos % kBlockTokens : -1;
      }
    }
    needed += total.x;
    asked += total.y;
    rows += got_total.y;
    taken += got_total.x;
    __syncthreads();                                                  // the edges may be written again
  }
  for (int i = (int)rows + rank * threads + tid; i < a.n; i += threads * gridDim.x) {
    a.positions[i] = 0;
    a.row_seq[i] = a.nseq;
    a.slots[i] = (long long)a.num_blocks * kBlockTokens;
  }
  if (tid == 0 && rank == 0) {
    a.cu[0] = 0;
    *a.free_next = at0 + (int)taken;
  }
}

}  // namespace

cudaError_t launch_kv_extend(const KvExtendArgs& in, cudaStream_t s) {
  KvExtendArgs a = in;
  void* p[] = {&a};
  // few sequences and rows: a barrier of few warps. In a graph, us, with 128, 512 and 1024
  // threads: 64 sequences by a token each 2.2, 2.5, 3.2; 512 6.2, 2.9, 3.5; 1000 11.5, 4.7, 4.1.
  // (1000 rows of one sequence would be quicker with 512: 4.4, 2.7, 3.6.)
  const int most = a.nseq > a.n ? a.nseq : a.n, threads = most <= 128 ? 128 : most <= 512 ? 512 : kPlanThreads;
  a.in_place = a.held == a.ctx_lens || a.free_next == a.free_at;
  int ctas = 1;
  while (ctas * kPlanThreads < a.n && ctas < (a.in_place ? kPlanCluster : kPlanGrid)) ctas *= 2;
  return launch_ex((const void*)kv_extend_kernel, dim3(ctas), dim3(threads), 0, s, p, true, -1, a.in_place ? ctas : 0);
}

}  // namespace mbt
