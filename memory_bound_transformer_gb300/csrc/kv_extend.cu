// Block tables and row layout for a step's new tokens, from the sequences'
// lengths alone: sequence s with ctx_s cached and new_s new tokens needs
//   need_s = ceil((ctx_s + new_s) / 16) - ceil(ctx_s / 16)
// blocks, which are those of the free list behind the ones that sequences before
// it need, and its rows stand behind theirs: two prefix sums, and the same over
// those that fit where not all do ("Kernels, Fusion & CUDA Graphs", "The serving
// engine's kernel stack": block tables of the paged cache). Bound by latency: 64
// sequences by a token each take 3.1 us in a graph, 512 by 65 k rows, in two
// launches, 9.2.
#include "common.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kPlanThreads = 1024;           // most threads of the tables' CTA, a sequence each
// Rows up to which that CTA lays them out itself: 1024 rows of 64 sequences 4.7 us
// (5.4 in two launches), 2048 6.0 (5.5), 4096 7.9 (5.5).
constexpr int kPlanRows = 1024;
constexpr int kRowThreads = 256;
constexpr int kRowSeqs = 4096;               // row edges that the rows' CTAs keep in shared memory

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

// Row i of sequence seq (nseq: padding) at position pos.
__device__ __forceinline__ void lay_row(const KvExtendArgs& a, int i, int seq, int pos) {
  long long slot = (long long)a.num_blocks * kBlockTokens;
  if (seq < a.nseq) {
    const int blk = a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens];
    const bool ok = blk >= 0 && blk <= a.num_blocks;
    if (!ok) set_err(a.err, MBT_DEV_BLOCK_RANGE);
    slot = ok ? (long long)blk * kBlockTokens + pos % kBlockTokens : -1;
  }
  a.positions[i] = pos;
  a.row_seq[i] = seq;
  a.slots[i] = slot;
}

// One CTA: tables, lengths and row edges, a sequence per thread at a time, and the
// rows where they are few. What a sequence reads of arrays that may be written in
// place it reads before. Bound by latency: the lengths, the free list's entries
// and the rows' table entries are three round trips, a launch the rest.
__global__ void __launch_bounds__(kPlanThreads) kv_extend_kernel(const KvExtendArgs a) {
  __shared__ Pair scratch[32];
  __shared__ int took_edge[kPlanThreads + 1], row_edge[kPlanThreads + 1], sm_have[kPlanThreads], sm_ctx[kPlanThreads];
  const int tid = threadIdx.x, threads = blockDim.x;
  pdl_launch_dependents();
  const int at0 = *a.free_at;
  const bool at_ok = at0 >= 0 && at0 <= a.nfree;
  if (!at_ok && tid == 0) set_err(a.err, MBT_DEV_BLOCK_RANGE);
  long long needed = 0, asked = 0, rows = 0, taken = 0;
  if (tid == 0) a.cu[0] = took_edge[0] = row_edge[0] = 0;
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
    if (in) {
      a.held[s] = ctx + add;
      a.cu[s + 1] = (int)(rows + got.y);
    }
    took_edge[tid + 1] = (int)got.x;
    row_edge[tid + 1] = (int)(rows + got.y);
    sm_have[tid] = have;
    sm_ctx[tid] = ctx;
    __syncthreads();
    for (int i = tid; i < (int)got_total.x; i += threads) {
      const int q = segment_of(took_edge, threads, i), id = a.free_blocks[at0 + taken + i];
      if (id < 0 || id > a.num_blocks) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      a.bt[(size_t)(s0 + q) * a.bt_stride + sm_have[q] + i - took_edge[q]] = id;
    }
    __syncthreads();
    if (a.here) {
      for (int i = (int)rows + tid; i < (int)(rows + got_total.y); i += threads) {
        const int q = segment_of(row_edge, threads, i);
        lay_row(a, i, s0 + q, sm_ctx[q] + i - row_edge[q]);
      }
      __syncthreads();
    }
    needed += total.x;
    asked += total.y;
    rows += got_total.y;
    taken += got_total.x;
    if (tid == 0) row_edge[0] = (int)rows;
  }
  if (a.here)
    for (int i = (int)rows + tid; i < a.n; i += threads) lay_row(a, i, a.nseq, 0);
  if (tid == 0) *a.free_next = at0 + (int)taken;
}

// The packed rows of a large step, one per thread.
__global__ void __launch_bounds__(kRowThreads) kv_rows_kernel(const KvExtendArgs a) {
  __shared__ int edge[kRowSeqs + 1];
  pdl_wait();
  const bool small = a.nseq <= kRowSeqs;
  if (small) {
    for (int s = threadIdx.x; s <= a.nseq; s += kRowThreads) edge[s] = a.cu[s];
    __syncthreads();
  }
  const int* cu = small ? edge : a.cu;
  const int i = blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= a.n) return;
  if (i >= cu[a.nseq]) return lay_row(a, i, a.nseq, 0);
  const int seq = segment_of(cu, a.nseq, i);
  lay_row(a, i, seq, a.held[seq] - cu[seq + 1] + i);
}

}  // namespace

cudaError_t launch_kv_extend(const KvExtendArgs& in, cudaStream_t s) {
  KvExtendArgs a = in;
  void* p[] = {&a};
  // few sequences or rows: a barrier of few warps. Rows beyond a few per thread go to a grid of their own.
  const int most = a.nseq > a.n ? a.nseq : a.n, threads = most <= 128 ? 128 : most <= 512 ? 512 : kPlanThreads;
  a.here = a.n <= kPlanRows;
  const cudaError_t e = launch_ex((const void*)kv_extend_kernel, dim3(1), dim3(threads), 0, s, p, false, -1);
  if (e != cudaSuccess || a.here) return e;
  return launch_pdl((const void*)kv_rows_kernel, dim3((unsigned)((a.n + (long long)kRowThreads - 1) / kRowThreads)),
                    dim3(kRowThreads), 0, s, p);
}

}  // namespace mbt
