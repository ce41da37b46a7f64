// Single-token attention over the 4-bit paged KV cache (format in fp4.cuh):
//   o_h = sum_t softmax_t(q_h . K_t / sqrt(d)) V_t   over t < seq_len[b],
// one pass with the running maximum and sum of the softmax; the query heads of
// a KV head share its stream ("GPU Inference Internals", "The KV-Cache Ledger":
// grouped-query attention).
//
// What bounds it: at 9/16 byte a value the cache streams at HBM rate only if a
// 64-token tile (9.2 KB at d = 128) costs an SM fewer than ~395 cycles. So
// the work per cached value is what is kept small:
// * Queries and probabilities enter mma.sync.m16n8k16 as FP16 high and low
//   parts (2^-22 relative) stacked on M: rows 0..7 the high parts of the group's
//   heads, rows 8..15 the low parts. One MMA serves both, S = row g + row g + 8
//   sits in one thread, and the S accumulators are the A fragments of P V as
//   they stand: nothing is transposed or shuffled. Probabilities are relative to
//   2^-14 of the largest so far, not to the largest: FP16's smallest steps, which
//   take from many small ones what their sum still counts, then lie at 2^-39 of
//   the largest (2^-22 holds down to 2^-17 of it). The factor cancels in o / l.
// * K and V fragments come straight from the raw codes. The contraction may
//   run over the channels in any order, so thread (g, t) of a warp takes D / 4
//   neighbouring channels of a token (one 16-byte load at d = 128) and the
//   queries are laid out the same way; likewise D / 8 neighbouring output
//   channels of V. Per pair of values: one hardware conversion (e2m1x2 to
//   f16x2) and one FP16 multiply by the group's e4m3 scale; both exact (2 + 4
//   significant bits). V's pairs are two tokens of one channel: the nibbles of
//   two tokens' words are interleaved first, half an operation a pair.
// * Every warp runs its own ring of 64-token steps (four cache blocks) filled by
//   16-byte asynchronous copies: no block-wide barrier in the loop.
// * The tensor core's fp32 accumulation truncates, so chains are kept short
//   (D / 16 steps for S, four for P V) and the sums over steps are IEEE fp32.
// Conversions and multiplies issue every second cycle and an MMA every eighth
// per SM quarter (measured), so a 64-token step's 128 MMAs, 256 conversions and
// 256 multiplies take 1024, 512 and 512 cycles of three pipes, against 1580 at
// the HBM rate; with the ~700 instructions around them a quarter takes 2390
// cycles a step (2130 without the loads), with two warps as with three or four:
// 4.5 TB/s over long contexts. Taking one part out saves what it issues: half the
// MMAs 470, the softmax 250, K's or V's multiplies 130, the nibble interleave
// 120, the scales 105. (With four heads per KV head half of the MMAs' rows are
// zeros, with more than eight the stream is read and converted once per eight.)
// Around the loop a launch has ~5 us: the lengths, ids and queries (one round
// trip), the first step's blocks, one step, the merges. 64 rows of 64 + 2 x 8
// heads of 128 over 2048 tokens: 51 us (3.0 TB/s: 512 CTAs are 1.7 waves of two
// an SM); one row of 32 + 2 x 8 heads over 2048: 5.6 us (both in a graph).
#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kF4Warps = 4;
constexpr int kF4Threads = 32 * kF4Warps;
constexpr int kF4PerSm = 2;                 // CTAs per SM (217 registers a thread; three at 168 spill and are no faster)
constexpr int kF4Stages = 2;                // steps of a warp's ring
constexpr int kF4Step = 64;                 // tokens per step: four cache blocks
constexpr int kF4Blocks = kF4Step / kBlockTokens;
constexpr int kF4Heads = 8;                 // query heads per CTA (MMA rows, high and low parts)
constexpr int kF4Cluster = 8;               // most CTAs of a cluster
constexpr float kF4Up = 14.f;               // probabilities go up to 2^14

template <int D>
struct Fp4Shape {
  static constexpr int UNIT = fp4_unit_bytes(D);
  static constexpr int STAGE = 2 * kF4Blocks * UNIT;  // K and V of a step's blocks
  static constexpr int KS = D / 16;                   // MMA steps over the channels
  static constexpr int NT = D / 8;                    // n-tiles of the output = channels of a thread
  static constexpr int RING = kF4Warps * kF4Stages * STAGE;
  static constexpr int OUT = kF4Warps * kF4Heads * D * 4;   // the warps' outputs
  static constexpr int SMEM = RING;                   // the outputs take the drained ring's place
  static_assert(OUT <= RING, "");
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 bytes (low first) as an FP16 pair.
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// x = hi + lo to 2^-22, both as FP16 pairs.
__device__ __forceinline__ void split_h2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(x0, x1);
  const float2 h = h2_to_float2(hi);
  lo = pack_h2(x0 - h.x, x1 - h.y);
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// One (block, KV head) unit to shared memory, 16 bytes per lane and copy (the
// lane's offset is in both addresses).
template <int UNIT>
__device__ __forceinline__ void copy_unit(uint32_t dst, const unsigned char* src, int lane) {
#pragma unroll
  for (int c = 0; c < UNIT; c += 512)
    if (c + 512 <= UNIT || c + lane * 16 < UNIT)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + c), "l"(src + c) : "memory");
}
// The same from a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Steps of a row, 0 for a length outside its table.
__device__ __forceinline__ int steps_of(const AttnFp4Args& a, int seq) {
  return seq < 1 || seq > (long long)a.bt_stride * kBlockTokens ? 0 : (seq + kF4Step - 1) / kF4Step;
}

// Lanes 0..3: the table's ids of step j's four blocks in row b.
__device__ __forceinline__ int step_ids(const AttnFp4Args& a, int b, int j, int blocks, int lane) {
  return lane < kF4Blocks && lane < blocks ? __ldg(a.bt + (size_t)b * a.bt_stride + kF4Blocks * j + lane) : 0;
}
// Requests one step into a ring stage: the K and V units of its blocks (the
// lane's offset is in all addresses). id: step_ids, checked here and not where
// it is loaded, one request earlier (the load's latency stays hidden).
template <int D>
__device__ __forceinline__ void request_step(const AttnFp4Args& a, uint32_t dst, int h, int id, int blocks, int lane) {
  constexpr int UNIT = Fp4Shape<D>::UNIT;
  if (lane < min(blocks, kF4Blocks) && (uint32_t)id > (uint32_t)a.num_blocks) {   // out of range: the null block
    set_err(a.err, MBT_DEV_BLOCK_RANGE);
    id = a.num_blocks;
  }
#pragma unroll
  for (int blk = 0; blk < kF4Blocks; ++blk) {
    const size_t off = ((size_t)__shfl_sync(0xffffffffu, id, blk) * a.nkv + h) * UNIT + lane * 16;
    if (blk < blocks) {
      copy_unit<UNIT>(dst + 2 * blk * UNIT, reinterpret_cast<const unsigned char*>(a.kpool) + off, lane);
      copy_unit<UNIT>(dst + (2 * blk + 1) * UNIT, reinterpret_cast<const unsigned char*>(a.vpool) + off, lane);
    }
  }
}
__device__ __forceinline__ int blocks_from(int seq, int j) {          // cache blocks from step j's first on
  return (seq + kBlockTokens - 1) / kBlockTokens - kF4Blocks * j;
}

// One warp's part of a (row, KV head): queries of up to eight heads as MMA
// fragments, running maximum less kF4Up (log2 domain), sum (this lane's share)
// and output.
template <int D>
struct Fp4Warp {
  using S = Fp4Shape<D>;
  uint32_t qh[2 * S::KS], ql[2 * S::KS];
  float fac, m, l;
  float o[S::NT][2];

  // Head g's channels t4 * D / 4 .. of the queries.
  __device__ __forceinline__ void load(const AttnFp4Args& a, size_t head0, int gn, int lane, float (&x)[D / 4]) {
    const int g = lane >> 2, t4 = lane & 3;
    const float4* src = reinterpret_cast<const float4*>(a.q + (head0 + g) * D + t4 * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float4 v = g < gn ? __ldg(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
  }
  // A power-of-two scale per head puts the largest in [2^13, 2^14) (FP16 range,
  // subnormals far below), then high and low parts; `fac` takes scores back to
  // the log2 domain.
  __device__ __forceinline__ void start(const AttnFp4Args& a, const float (&x)[D / 4]) {
    uint32_t big = 0;                                                // largest magnitude's bits; a NaN's are larger than inf's
#pragma unroll
    for (int i = 0; i < D / 4; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int e = min(120, 140 - (int)(big >> 23));                  // 2^e: scores of still smaller queries are 0 either way
    const float up = __int_as_float((e + 127) << 23);
    fac = 1.4426950408889634f / sqrtf((float)D) * a.k_scale * __int_as_float((127 - e) << 23);
    fac = fmaxf(fac, 1.2e-38f);                                      // masked scores (-inf) stay -inf
    if (big >= 0x7f800000u) fac = __int_as_float(0x7fc00000);        // a non-finite query: its row is NaN
#pragma unroll
    for (int i = 0; i < 2 * S::KS; ++i) split_h2(x[2 * i] * up, x[2 * i + 1] * up, qh[i], ql[i]);
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < S::NT; ++i) o[i][0] = o[i][1] = 0.f;
  }

  // One step in the ring stage; `live` of its 64 tokens (or more) are in the context.
  __device__ __forceinline__ void step(const unsigned char* stage, int live, int lane) {
    const int g = lane >> 2, t4 = lane & 3;
    constexpr int TT = kF4Step / 8;                                  // n-tiles of tokens
    // S = Q K^T. Column c of n-tile nt is token 8 nt + (c >> 1) + 4 (c & 1): a
    // V load below then meets rows of both parities (banks).
    float s[TT][4];
    const unsigned char* krow = stage + ((g >> 1) + 4 * (g & 1)) * (D / 2) + t4 * (D / 8);
    const unsigned char* kscl = stage + kBlockTokens * (D / 2) + ((g >> 1) + 4 * (g & 1)) * (D / 16) + t4 * (D / 64);
#pragma unroll
    for (int wp = 0; wp < D / 64; ++wp) {                            // 16 channels, one scale: two words, four MMA steps
      uint32_t w[TT][2], sc[TT];
#pragma unroll
      for (int nt = 0; nt < TT; ++nt) {
        const int off = 2 * (nt >> 1) * S::UNIT + 8 * (nt & 1) * (D / 2);
        const uint2 v = *reinterpret_cast<const uint2*>(krow + off + 8 * wp);
        w[nt][0] = v.x; w[nt][1] = v.y;
        sc[nt] = e4m3x2_h2((uint32_t)kscl[2 * (nt >> 1) * S::UNIT + 8 * (nt & 1) * (D / 16) + wp] * 0x0101u);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int q = 8 * wp + 4 * j;
        const uint32_t a0[4] = {qh[q], ql[q], qh[q + 1], ql[q + 1]}, a1[4] = {qh[q + 2], ql[q + 2], qh[q + 3], ql[q + 3]};
#pragma unroll
        for (int nt = 0; nt < TT; ++nt) {
          uint32_t k[4];
          e2m1x8_to_h2(w[nt][j], k);
#pragma unroll
          for (int e = 0; e < 4; ++e) k[e] = hmul2(k[e], sc[nt]);
          if (wp == 0 && j == 0) mma_f16_zero(s[nt], a0, k[0], k[1]);
          else mma_f16(s[nt], a0, k[0], k[1]);
          mma_f16(s[nt], a1, k[2], k[3]);
        }
      }
    }
    // softmax of head g over this thread's tokens (8 nt + t4, + 4)
    float p[TT][2], mx = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < TT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) p[nt][e] = s[nt][e] + s[nt][e + 2];
    if (live < kF4Step) {
#pragma unroll
      for (int nt = 0; nt < TT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (8 * nt + t4 + 4 * e >= live) p[nt][e] = -INFINITY;
    }
#pragma unroll
    for (int nt = 0; nt < TT; ++nt) mx = fmaxf(mx, fmaxf(p[nt][0], p[nt][1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(m, fmaf(mx, fac, -kF4Up)), mu = mn == -INFINITY ? 0.f : mn;
    const float al = ex2(m - mu);
    m = mn;
    l *= al;
    uint32_t pa[TT / 2][4];                                          // A fragments of P: high and low parts of 16 tokens
#pragma unroll
    for (int nt = 0; nt < TT; ++nt) {
      p[nt][0] = ex2(fmaf(p[nt][0], fac, -mu));
      p[nt][1] = ex2(fmaf(p[nt][1], fac, -mu));
      l += p[nt][0] + p[nt][1];
      split_h2(p[nt][0], p[nt][1], pa[nt / 2][2 * (nt & 1)], pa[nt / 2][2 * (nt & 1) + 1]);
    }
    // O = O * al + P V: this thread's channels are g * D / 8 .., its tokens
    // those of its probabilities; rows past the context get scale 0
    uint32_t vs[TT];
#pragma unroll
    for (int nt = 0; nt < TT; ++nt) {
      const unsigned char* sb = stage + (2 * (nt >> 1) + 1) * S::UNIT + kBlockTokens * (D / 2) +
                                (8 * (nt & 1) + t4) * (D / 16) + (g * (D / 8)) / 16;
      vs[nt] = (uint32_t)sb[0] | ((uint32_t)sb[4 * (D / 16)] << 8);
    }
    if (live < kF4Step) {
#pragma unroll
      for (int nt = 0; nt < TT; ++nt) {
        if (8 * nt + t4 >= live) vs[nt] = 0;                         // token + 4 lies past it too
        else if (8 * nt + t4 + 4 >= live) vs[nt] &= 0xffu;
      }
    }
#pragma unroll
    for (int nt = 0; nt < TT; ++nt) vs[nt] = e4m3x2_h2(vs[nt]);
    const unsigned char* vrow = stage + S::UNIT + t4 * (D / 2) + g * (D / 16);
#pragma unroll
    for (int wd = 0; wd < D / 64; ++wd) {                            // 8 channels of the thread at a time
      uint32_t va[TT], vb[TT];                                       // the codes of tokens 8 nt + t4 and + 4
#pragma unroll
      for (int nt = 0; nt < TT; ++nt) {
        const int off = 2 * (nt >> 1) * S::UNIT + 8 * (nt & 1) * (D / 2) + 4 * wd;
        va[nt] = *reinterpret_cast<const uint32_t*>(vrow + off);
        vb[nt] = *reinterpret_cast<const uint32_t*>(vrow + off + 4 * (D / 2));
      }
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {                            // channels 0, 2, 4, 6, then 1, 3, 5, 7 of both tokens
        uint32_t f[TT][4];
#pragma unroll
        for (int nt = 0; nt < TT; ++nt) {
          e2m1x8_to_h2(odd ? ((va[nt] >> 4) & 0x0f0f0f0fu) | (vb[nt] & 0xf0f0f0f0u)
                           : (va[nt] & 0x0f0f0f0fu) | ((vb[nt] << 4) & 0xf0f0f0f0u), f[nt]);
#pragma unroll
          for (int c = 0; c < 4; ++c) f[nt][c] = hmul2(f[nt][c], vs[nt]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float acc[4];
          mma_f16_zero(acc, pa[0], f[0][c], f[1][c]);
#pragma unroll
          for (int k = 1; k < TT / 2; ++k) mma_f16(acc, pa[k], f[2 * k][c], f[2 * k + 1][c]);
          const int ch = 8 * wd + 2 * c + odd;
          o[ch][0] = fmaf(o[ch][0], al, acc[0] + acc[2]);
          o[ch][1] = fmaf(o[ch][1], al, acc[1] + acc[3]);
        }
      }
    }
  }

  // The warp's state to shared memory: so [head][D], sm_m and sm_l [head].
  __device__ __forceinline__ void leave(float* so, float* sm_m, float* sm_l, int lane) {
    const int g = lane >> 2, t4 = lane & 3;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t4 == 0) { sm_m[g] = m; sm_l[g] = l; }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // column 2 t4 + c of every n-tile: channels (2 t4 + c) * D / 8 ..
      float4* dst = reinterpret_cast<float4*>(so + g * D + (2 * t4 + c) * (D / 8));
#pragma unroll
      for (int i = 0; i < S::NT; i += 4) dst[i / 4] = make_float4(o[i][c], o[i + 1][c], o[i + 2][c], o[i + 3][c]);
    }
  }
};

// Element e of the CTA's merged output (not normalised), with the maximum and
// sum of its head.
template <int D>
__device__ __forceinline__ float merge_warps(const float* so, const float (*sm_m)[kF4Heads], const float (*sm_l)[kF4Heads],
                                             int e, float& M, float& L) {
  const int hr = e / D;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kF4Warps; ++w) M = fmaxf(M, sm_m[w][hr]);
  const float mu = M == -INFINITY ? 0.f : M;
  float acc = 0.f;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kF4Warps; ++w) {
    const float f = ex2(sm_m[w][hr] - mu);
    L = fmaf(sm_l[w][hr], f, L);
    acc = fmaf(so[w * kF4Heads * D + e], f, acc);
  }
  return acc;
}

// The row with `rank` longer ones before it (equal lengths in order), for at
// most kF4Threads rows; all threads call it.
__device__ __forceinline__ int row_of_rank(const AttnFp4Args& a, int rank) {
  __shared__ __align__(16) int sm_len[kF4Threads], sm_row;
  const int tid = threadIdx.x, mine = tid < a.B ? __ldg(a.seq_lens + tid) : INT_MIN;
  sm_len[tid] = mine;
  __syncthreads();
  int before = 0;
  for (int j = 0; j < a.B; j += 4) {
    const int4 v = *reinterpret_cast<const int4*>(sm_len + j);
    before += (v.x > mine || (v.x == mine && j < tid)) + (v.y > mine || (v.y == mine && j + 1 < tid)) +
              (v.z > mine || (v.z == mine && j + 2 < tid)) + (v.w > mine || (v.w == mine && j + 3 < tid));
  }
  if (tid < a.B && before == rank) sm_row = tid;
  __syncthreads();
  return sm_row;
}

// One cluster of 1..8 CTAs per pair (row, KV head, group of eight heads), whose
// warps take the row's steps in turn; the CTAs' parts merge through distributed
// shared memory. One launch, no scratch. (One wave of clusters of four that share
// all pairs' steps evenly balances better, but finding the shares from the
// lengths costs 4 us: 37 / 54 / 94 us against 33 / 51 / 45, longest rows first, for
// 64 rows of 256 to 2048 tokens, 64 of 2048 and 4 of 32k.)
template <int D>
__global__ void __launch_bounds__(kF4Threads, kF4PerSm) attention_fp4_kernel(const AttnFp4Args a) {
  using S = Fp4Shape<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[kF4Warps][kF4Heads], sm_l[kF4Warps][kF4Heads];
  __shared__ float cta_m[kF4Heads], cta_l[kF4Heads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sp = (int)(blockIdx.x % (unsigned)a.cluster);
  const int pair = (int)(blockIdx.x / (unsigned)a.cluster);          // (row, KV head, group of 8 heads)
  const int hb = pair % a.hblocks, h = (pair / a.hblocks) % a.nkv;
  int b = pair / a.hblocks / a.nkv;
  const int gn = min(kF4Heads, a.nq / a.nkv - hb * kF4Heads);
  auto first_head = [&]() { return (size_t)b * a.nq + (size_t)h * (a.nq / a.nkv) + hb * kF4Heads; };

  // Three loads that do not depend on one another: the row's length, the
  // queries, and the block ids of this warp's first steps (its steps are dealt
  // over the cluster's warps in turn, so they are known without the length).
  const int first = sp * kF4Warps + warp, stride = a.cluster * kF4Warps;
  int seq, id, id2;
  Fp4Warp<D> w;
  float x[D / 4];
  auto load_row = [&]() {
    seq = __ldg(a.seq_lens + b);
    id = step_ids(a, b, first, a.bt_stride - kF4Blocks * first, lane);
    id2 = step_ids(a, b, first + stride, a.bt_stride - kF4Blocks * (first + stride), lane);
    w.load(a, first_head(), gn, lane, x);
  };
  load_row();
  if (a.sorted) {                                                    // under way for the row in order; often it is that one
    const int row = row_of_rank(a, b);
    if (row != b) { b = row; load_row(); }
  }
  const size_t head0 = first_head();
  const int steps = steps_of(a, seq);
  if (!steps && tid == 0 && sp == 0 && h == 0 && hb == 0) set_err(a.err, MBT_DEV_SEQLEN_RANGE);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kF4Stages * S::STAGE;
  int next = first;
  auto request = [&](int stage) {                                    // the warp's next step, ids two requests ahead
    if (next < steps) {
      request_step<D>(a, ring + stage * S::STAGE + lane * 16, h, id, blocks_from(seq, next), lane);
      next += stride;
      id = id2;
      if (next + stride < steps) id2 = step_ids(a, b, next + stride, blocks_from(seq, next + stride), lane);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kF4Stages - 1; ++i) request(i);
  w.start(a, x);
  int st = 0, fill = kF4Stages - 1;
#pragma unroll 1
  for (int j = first; j < steps; j += stride) {
    request(fill);
    asm volatile("cp.async.wait_group %0;" ::"n"(kF4Stages - 1) : "memory");
    __syncwarp();
    w.step(smem + (warp * kF4Stages + st) * S::STAGE, seq - j * kF4Step, lane);
    __syncwarp();                                                    // the stage may be refilled
    fill = st;
    st = st + 1 == kF4Stages ? 0 : st + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                                                   // every ring is drained
  float* so = reinterpret_cast<float*>(smem);                        // [warp][head][D]
  w.leave(so + warp * kF4Heads * D, sm_m[warp], sm_l[warp], lane);
  __syncthreads();
  for (int e = tid; e < gn * D; e += kF4Threads) {
    float M, L;
    const float acc = merge_warps<D>(so, sm_m, sm_l, e, M, L);
    if (a.cluster == 1) {
      a.out[head0 * D + e] = steps ? acc * (a.v_scale / L) : 0.f;
    } else {
      so[e] = acc;                                                   // of warp 0's part: read by this thread only
      if (e % D == 0) { cta_m[e / D] = M; cta_l[e / D] = L; }
    }
  }
  if (a.cluster == 1) return;
  cluster_sync_all();
  for (int e = sp * kF4Threads + tid; e < gn * D; e += a.cluster * kF4Threads) {
    float pm[kF4Cluster], pl[kF4Cluster], po[kF4Cluster], M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
    for (int r = 0; r < kF4Cluster; ++r) {
      const bool in = r < a.cluster;
      pm[r] = in ? ld_dsmem_f32(&cta_m[e / D], r) : -INFINITY;
      pl[r] = in ? ld_dsmem_f32(&cta_l[e / D], r) : 0.f;
      po[r] = in ? ld_dsmem_f32(&so[e], r) : 0.f;
      M = fmaxf(M, pm[r]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int r = 0; r < kF4Cluster; ++r) {
      const float f = ex2(pm[r] - mu);
      L = fmaf(pl[r], f, L);
      acc = fmaf(po[r], f, acc);
    }
    a.out[head0 * D + e] = steps ? acc * (a.v_scale / L) : 0.f;
  }
  cluster_sync_all();                                                // stay resident until the others have read
}

template <int D>
cudaError_t fp4_launch(const AttnFp4Args& a, cudaStream_t s) {
  AttnFp4Args args = a;
  void* p[] = {&args};
  const long long grid = (long long)a.B * a.nkv * a.hblocks * a.cluster;
  return launch_ex((const void*)attention_fp4_kernel<D>, dim3((unsigned)grid), dim3(kF4Threads), Fp4Shape<D>::SMEM, s, p,
                   false, 100, a.cluster > 1 ? a.cluster : 0);
}

template <int D>
cudaError_t fp4_init() {
  return cudaFuncSetAttribute((const void*)attention_fp4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Fp4Shape<D>::SMEM);
}

}  // namespace

cudaError_t attn_fp4_plan(AttnFp4Args* a, int num_sms) {
  a->hblocks = (a->nq / a->nkv + kF4Heads - 1) / kF4Heads;
  const long long pairs = (long long)a->B * a->nkv * a->hblocks;
  if (pairs * kF4Cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  // one wave of clusters, no CTA with less than a step per warp of a full table
  const long long steps = ((long long)a->bt_stride * kBlockTokens + kF4Step - 1) / kF4Step;
  const long long want = std::min(steps / kF4Warps, (long long)kF4PerSm * num_sms / pairs);
  a->cluster = (int)std::max<long long>(1, std::min<long long>(kF4Cluster, want));
  // More than a wave of long rows: the longest first, so that the last wave's are
  // short. Finding them costs ~500 cycles a CTA, and a round trip where the row is
  // another than in order: 64 x 8 pairs of 256..2048 tokens 39.1 -> 32.7 us, of
  // 2048 each 49.4 -> 50.6; 128 x 8 of 64..8192 193 -> 164, of 100..1000 43.0 ->
  // 46.6; 40 x 8 (1.05 waves) of 128..4096 39.1 -> 40.9. So from 32 steps and five
  // quarters of a wave on.
  a->sorted = a->B <= kF4Threads && steps >= 32 && 4 * pairs * a->cluster > 5LL * kF4PerSm * num_sms;
  return cudaSuccess;
}

cudaError_t launch_attention_fp4(const AttnFp4Args& a, cudaStream_t s) {
  return a.d == 64 ? fp4_launch<64>(a, s) : fp4_launch<128>(a, s);
}

cudaError_t attn_fp4_init() {
  const cudaError_t e = fp4_init<64>();
  return e != cudaSuccess ? e : fp4_init<128>();
}

}  // namespace mbt
