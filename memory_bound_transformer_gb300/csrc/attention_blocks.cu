// Softmax attention over selected blocks of the paged KV cache:
//   o_h = sum_t softmax_t(q_h . K_t / sqrt(d)) V_t   over the tokens t <= p of the
// blocks chosen for the row and the KV head of h, one pass with the running
// maximum and sum of the softmax ("GPU Inference Internals", "The KV-Cache
// Ledger": the bytes of the cache are what a decode step reads).
//
// What bounds it: every chosen block is read once, 2 x 16 tokens of d values in
// runs of 1 to 4 KB (a gather of those alone reaches 6.1 to 6.2 TB/s), so the work
// per value has to stay below what the SM issues meanwhile.
// * Queries and probabilities enter mma.sync.m16n8k16 as parts stacked on M: rows
//   0..7 the high parts of the group's heads, rows 8..15 the next. Over a BF16
//   cache they are three BF16 parts (24 bits; the third in a second MMA, or for up
//   to four heads in the same one), over the narrow caches, whose values FP16 holds
//   exactly, two FP16 parts (2^-22), probabilities relative to 2^-14 of the largest
//   so that FP16's smallest steps lie at 2^-39 of it. Over those, up to four heads are
//   turned over, keys on M and parts on N: half the MMAs, softmax and output registers
//   (the 4-bit case of 510 rows below 64 us against 77; 256 rows of 32 + 2 x 8 heads of
//   128 over 64 e4m3 blocks 94 against 105, 4-bit 73 against 88; 20 or 24 warps per SM at
//   d = 64 64 and 68, 16 at d = 128 99 and 72).
// * The contraction may run over channels in any order: thread (g, t) of a warp
//   takes 16-byte pieces of a key, and the queries are laid out the same way. V's
//   pairs are two tokens of one channel, interleaved from two tokens' words. The
//   score accumulators are the A fragments of P V as they stand (turned over: the B
//   fragments after a transposition).
// * The tensor core's fp32 accumulation truncates, so chains are short (d / 16
//   steps for scores, a step's blocks for P V) and sums over steps are IEEE fp32.
// * A warp takes whole blocks from the row's list and has rings of two steps of its
//   own for K and for V, filled by 16-byte asynchronous copies and refilled as soon
//   as read: no barrier in the loop. (Straight into registers, which hold one step,
//   the e4m3 case below took 69 us against 66 at that stage.)
// * Few (row, KV head) pairs are shared by clusters, many get CTAs of two warps or
//   one, so that one wave of up to 12 warps per SM (16 at d = 64) holds them.
// Measured in a graph, us: 64 rows of 32 + 2 x 8 heads of 128 over 64 BF16 blocks
// 47 to 48.5 (5.6 to 5.8 TB/s; the copies alone 46.8 with three warps a CTA, 52.8 then),
// 128 rows 88 (6.2 TB/s); 64 rows of 64 + 2 x 8 heads of 128 over 128 e4m3 blocks 51.3
// (copies 48), over 128 4-bit blocks 54 (copies 32: conversions and scales; 32 + 2 x 8
// heads 42); 510 rows of 32 + 2 x 8 heads of 64 over 48 4-bit blocks each 59.7 (issue 67 %
// while active, in 3.4 waves of CTAs); one row of 32 + 2 x 8 heads of 128 over 64 BF16
// blocks 8.1, of which some 7 are the launch, four round trips (position, entry, table,
// block) and the merge.
#include <algorithm>
#include <type_traits>

#include <cuda_fp16.h>

#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

constexpr int kBaWarps = 4;                 // most warps of a CTA
__host__ __device__ constexpr int ba_per_sm(int d) { return d == 64 ? 16 : 12; }   // warps per SM (128, 168 registers a thread)
constexpr int kBaHeads = 8;                 // query heads per CTA (MMA rows)
constexpr int kBaCluster = 8;               // most CTAs of a cluster
constexpr int kBaStages = 2;                // steps of a warp's rings of K and V

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_b2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Parts of two values as 16-bit pairs: FP16 high and low, or BF16 high, middle and low.
template <bool BF>
__device__ __forceinline__ void split(float x0, float x1, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  if constexpr (BF) {
    p0 = pack_b2(x0, x1);
    x0 -= bf16_lo(p0); x1 -= bf16_hi(p0);
    p1 = pack_b2(x0, x1);
    p2 = pack_b2(x0 - bf16_lo(p1), x1 - bf16_hi(p1));
  } else {
    p0 = pack_h2(x0, x1);
    const float2 h = h2_to_float2(p0);
    p1 = pack_h2(x0 - h.x, x1 - h.y);
    p2 = 0;
  }
}
// The two FP16 parts of a value as a pair.
__device__ __forceinline__ uint32_t parts(float x) {
  return pack_h2(x, x - __half2float(__float2half_rn(x)));
}
// Of an 8 x 8 matrix of 16-bit values, whose row `lane / 4` a lane has two neighbours of, the transpose.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// d = a b + d, or + 0 where the sum begins.
template <bool BF, bool ZERO = false>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF && ZERO)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (ZERO)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The four e4m3 codes of a word as two FP16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_h2(uint32_t w) {           // of the low two
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(r) : "r"(w));
  return r;
}

// A lane's N words of shared memory.
template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const unsigned char* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// How a block's K and V lie over a warp. Thread (g, t) = (lane / 4, lane % 4)
// holds a quarter of the channels of the keys of columns g, token (g >> 1) + 4
// (g & 1) and that + 8, and an eighth of those of the values t, t + 4, t + 8 and
// t + 12.
template <int D, int KV>
struct Lay {
  static constexpr bool BF = KV == KV_BF16;
  static constexpr int ROW = KV == KV_BF16 ? 2 * D : KV == KV_E4M3 ? D : D / 2;   // bytes of a token
  static constexpr int UNIT = KV == KV_FP4 ? fp4_unit_bytes(D) : kBlockTokens * ROW;
  static constexpr int KB = ROW / 4 < 16 ? ROW / 4 : 16, KP = ROW / 4 / KB;       // bytes of a key's piece, pieces
  static constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16, VP = ROW / 8 / VB;       // of a value's
  static constexpr int KC = D / 4 / KP, VC = D / 8 / VP;                          // channels of a piece
  static constexpr int TB = KV == KV_BF16 ? 1 : KV == KV_E4M3 || D == 128 ? 2 : 4;   // blocks of a step
  static constexpr int KS = D / 16, NT = D / 8;                                   // MMA steps of a score, n-tiles of the output
  static constexpr int STAGE = TB * UNIT, RING = 2 * kBaStages * STAGE;           // K or V of a step; a warp's ring
  static constexpr int WARP = RING + (BF ? D * 4 : 0);                            // with the sums of values that are not finite
  static_assert(RING >= kBaHeads * D * 4, "the warp's output takes the drained ring's place");
  // channel of a lane's i-th query value; of the c-th value of column g of the output's n-tiles
  static __device__ __forceinline__ int q_channel(int t, int i) { return i / KC * 4 * KC + KC * t + i % KC; }
  static __device__ __forceinline__ int v_channel(int g, int c) { return c / VC * 8 * VC + VC * g + c % VC; }
  // What a token's 16-byte pieces are exchanged by within 128 bytes of shared
  // memory, so that eight lanes meet eight different ones, of two keys or of four
  // values.
  static __device__ __forceinline__ int swap(int tok) {
    return (tok & 4) ^ (ROW >= 128 ? (tok & 3) << 1 : ROW == 64 ? tok & 2 : 0);
  }
  // Place of byte `b` of a token in a unit in shared memory.
  static __device__ __forceinline__ int place(int tok, int b) { return (((tok * ROW + b) >> 4) ^ swap(tok)) << 4 | (b & 15); }
};

// The chosen blocks of a warp: entries first, first + stride, .. of the row's
// list, 32 at a time, a lane per entry.
struct Picks {
  const int* sel; const int* table;
  int k, stride, at, last, num_blocks;      // at: this lane's next entry; last: the context's last block
  uint32_t* err;
  uint32_t mask;                            // entries of this turn still to do
  int e, id, e2;                            // this turn's entry and block id, the next turn's entry

  __device__ __forceinline__ int entry() {
    const int x = at < k ? __ldg(sel + at) : -1;
    at = at < k ? at + 32 * stride : k;     // below k + 32 * stride: the caller sees to its range
    return x;
  }
  __device__ __forceinline__ void turn() {
    e = e2;
    if (e > last) {
      set_err(err, MBT_DEV_BLOCK_RANGE);
      e = -1;
    }
    mask = __ballot_sync(0xffffffffu, e >= 0);
    id = e >= 0 ? __ldg(table + e) : 0;
    if ((uint32_t)id > (uint32_t)num_blocks) {
      set_err(err, MBT_DEV_BLOCK_RANGE);
      id = num_blocks;
    }
    e2 = entry();
  }
  __device__ __forceinline__ bool any() {                             // warp-uniform
    while (!mask) {
      if (!__any_sync(0xffffffffu, at < k || e2 >= 0)) return false;
      turn();
    }
    return true;
  }
  // The next block: its id, and its first token relative to the row's position
  // (0 or less: live), or an id with no live token.
  __device__ __forceinline__ void take(int& blk, int& live, int pos) {
    if (mask) {
      const int src = __ffs(mask) - 1;
      mask &= mask - 1;
      blk = __shfl_sync(0xffffffffu, id, src);
      live = min(kBlockTokens, pos - __shfl_sync(0xffffffffu, e, src) * kBlockTokens + 1);
    } else {
      blk = num_blocks;
      live = 0;
    }
  }
};

// FEW: at most four heads. Over a BF16 cache their three parts then fit the MMA's
// 16 rows: rows 0..3 the high, 8..11 the middle and 4..7 the low ones, whose
// products lanes 16 apart exchange. Over the narrow caches the products are turned
// over: keys, and V's channels, lie along M's 16 and the two parts of four heads
// along N's eight, columns 2 h and 2 h + 1. A lane then has the scores of head t for
// the tokens of rows g and g + 8, none for heads that are not there, and both parts
// of a product; an 8 x 8 transposition makes P's B fragments of two parts packed
// into a word.
template <int D, int KV, bool FEW>
struct BlockWarp {
  using L = Lay<D, KV>;
  static constexpr bool BF = L::BF;
  static constexpr bool LOW = BF && !FEW;                             // low parts in MMAs of their own
  static constexpr bool TURN = FEW && !BF;
  static constexpr int S = TURN ? L::TB : 2 * L::TB, E = TURN ? 1 : 2;   // pairs of scores, outputs per channel
  using Frag = std::conditional_t<TURN, uint2, uint4>;                // the queries' fragment of an MMA step
  float m, l, o[L::NT][E];

  // The parts of lane's head as those of its two MMA rows.
  static __device__ __forceinline__ void rows(uint32_t& hi, uint32_t& mid, uint32_t lo, int lane) {
    if (lane & 16) { hi = lo; mid = 0; }
  }
  __device__ __forceinline__ void start() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = 0.f;
  }
  // Requests the K or V units of a step's blocks into a stage (a shared address).
  static __device__ __forceinline__ void request(uint32_t stage, const unsigned char* pool, const int (&blk)[L::TB], int nkv, int h, int lane) {
    constexpr int N = L::UNIT / 16, ROWS = kBlockTokens * L::ROW / 16;
#pragma unroll
    for (int b = 0; b < L::TB; ++b) {
      const unsigned char* unit = pool + ((size_t)blk[b] * nkv + h) * L::UNIT + lane * 16;
#pragma unroll
      for (int i = 0; i < N; i += 32) {
        const int c = i + lane, to = c < ROWS ? c ^ L::swap(c * 16 / L::ROW) : c;
        if (i + 32 <= N || c < N)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(stage + b * L::UNIT + to * 16), "l"(unit + i * 16) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Token of a block that s[i][e] of a lane is for.
  static __device__ __forceinline__ int token(int i, int e, int lane) {
    return TURN ? (lane >> 3) + (lane & 4) + 8 * e : 8 * (i & 1) + (lane & 3) + 4 * e;
  }
  // Largest of, or sum over, the lanes that have the same head.
  template <class F>
  static __device__ __forceinline__ float over_head(float x, F f) {
#pragma unroll
    for (int o = TURN ? 4 : 1; o <= (TURN ? 16 : 2); o <<= 1) x = f(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }

  // Scores of a step: s[i][e] of head g and block i / 2 (turned: head t and block i).
  // stage: its keys; frag: the queries' fragments, [KS][32 lanes]; frag_lo: the third parts'.
  __device__ __forceinline__ void scores(float (&s)[S][2], const unsigned char* stage, const Frag* frag, const uint2* frag_lo, int lane) {
    const int g = lane >> 2, t = lane & 3, tok = (g >> 1) + 4 * (g & 1);
    const unsigned char* at[2] = {stage + L::place(tok, t * L::KB), stage + L::place(tok, L::KP > 1 ? (4 + t) * L::KB : 0)};
    float acc[S][4];
    uint32_t sc[2 * L::TB], by[2 * L::TB];                            // 4-bit: scale bytes; the scale of 16 channels as FP16 pairs
    constexpr int PS = L::KS / L::KP;                                 // MMA steps of a piece
#pragma unroll
    for (int p = 0; p < L::KP; ++p) {
      uint32_t k[2 * L::TB][L::KB / 4];
#pragma unroll
      for (int i = 0; i < 2 * L::TB; ++i) lds(k[i], at[p & 1] + (i / 2) * L::UNIT + (i & 1) * 8 * L::ROW + p / 2 * 128);
      if constexpr (KV == KV_FP4) {
        const unsigned char* sb = stage + kBlockTokens * L::ROW + tok * (D / 16) + t * (D / 64);
#pragma unroll
        for (int i = 0; i < 2 * L::TB; ++i) {
          const unsigned char* x = sb + (i / 2) * L::UNIT + (i & 1) * 8 * (D / 16);
          sc[i] = D == 128 ? *reinterpret_cast<const uint16_t*>(x) : *x;
        }
      }
      // of the two keys of a lane in block b
      auto product = [&](int st, int b, const uint32_t (&x)[2], const uint32_t (&y)[2], const Frag& a, const uint2& z) {
        if constexpr (TURN) {
          if (st == 0) mma<BF, true>(acc[b], x[0], y[0], x[1], y[1], a.x, a.y);
          else mma<BF>(acc[b], x[0], y[0], x[1], y[1], a.x, a.y);
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t b0 = n ? y[0] : x[0], b1 = n ? y[1] : x[1];
            if (st == 0) mma<BF, true>(acc[2 * b + n], a.x, a.y, a.z, a.w, b0, b1);
            else mma<BF>(acc[2 * b + n], a.x, a.y, a.z, a.w, b0, b1);
            if constexpr (LOW) mma<BF>(acc[2 * b + n], z.x, 0u, z.y, 0u, b0, b1);
          }
        }
      };
      if constexpr (KV == KV_FP4) {
#pragma unroll
        for (int q = 0; q < PS; q += 2) {                             // a word: two steps
          const Frag a0 = frag[q * 32 + lane], a1 = frag[(q + 1) * 32 + lane];
#pragma unroll
          for (int b = 0; b < L::TB; ++b) {
            uint32_t y[2][2][2];                                      // [step][key]
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int i = 2 * b + n;
              if (q % 4 == 0) {
                const uint32_t byte = sc[i] >> (8 * (q / 4)) & 0xffu;
                by[i] = e4m3x2_h2(byte * 0x0101u);
              }
              uint32_t x[4];
              e2m1x8_to_h2(k[i][q / 2], x);
#pragma unroll
              for (int c = 0; c < 4; ++c) y[c >> 1][n][c & 1] = hmul2(x[c], by[i]);
            }
            product(q, b, y[0][0], y[0][1], a0, make_uint2(0, 0));
            product(q + 1, b, y[1][0], y[1][1], a1, make_uint2(0, 0));
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < PS; ++q) {
          const int st = p * PS + q;
          const Frag a = frag[st * 32 + lane];
          uint2 z = make_uint2(0, 0);
          if constexpr (LOW) z = frag_lo[st * 32 + lane];
#pragma unroll
          for (int b = 0; b < L::TB; ++b) {
            uint32_t x[2][2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int i = 2 * b + n;
              if constexpr (BF) {
                x[n][0] = k[i][2 * q];
                x[n][1] = k[i][2 * q + 1];
              } else {
                e4m3x4_to_h2(k[i][q], x[n][0], x[n][1]);
              }
            }
            product(st, b, x[0], x[1], a, z);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[i][e] = TURN ? acc[i][2 * e] + acc[i][2 * e + 1] : acc[i][e] + acc[i][e + 2];
        if constexpr (FEW && BF) s[i][e] += __shfl_xor_sync(0xffffffffu, s[i][e], 16);
        if constexpr (BF) s[i][e] += s[i][e] - s[i][e];               // of a key that is not finite: NaN
      }
  }

  // Softmax over the lane's tokens: probabilities as A fragments of P V (turned: as B
  // fragments, pa[b][0 .. 1]), and what the output so far is to be multiplied by.
  // live: tokens of each block that the row sees.
  __device__ __forceinline__ float soften(float (&s)[S][2], uint32_t (&pa)[S][3], const int (&live)[L::TB], float fac, int lane) {
    constexpr float UP = BF ? 0.f : 14.f;
    float mx = -INFINITY;
#pragma unroll
    for (int b = 0; b < L::TB; ++b)
      if (live[b] < kBlockTokens) {                                   // the same for the whole warp
#pragma unroll
        for (int i = b * S / L::TB; i < (b + 1) * S / L::TB; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (token(i, e, lane) >= live[b]) s[i][e] = -INFINITY;
      }
#pragma unroll
    for (int i = 0; i < S; ++i) mx = fmaxf(mx, fmaxf(s[i][0], s[i][1]));
    mx = over_head(mx, [](float x, float y) { return fmaxf(x, y); });
    // differences of scores first: equal ones stay equal however large they are
    const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn, al = ex2((m - mu) * fac);
    m = mn;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float p0 = ex2(fmaf(s[i][0] - mu, fac, UP)), p1 = ex2(fmaf(s[i][1] - mu, fac, UP));
      sum += p0 + p1;
      if constexpr (TURN) {
        pa[i][0] = transposed(parts(p0));
        pa[i][1] = transposed(parts(p1));
      } else {
        split<BF>(p0, p1, pa[i][0], pa[i][1], pa[i][2]);
        if constexpr (FEW) rows(pa[i][0], pa[i][1], pa[i][2], lane);
      }
    }
    l = fmaf(l, al, sum);
    return al;
  }

  // O = O * al + P V for a step whose values are in the stage. spec: where values
  // that are not finite go (null: they are not looked for).
  __device__ __forceinline__ void values(const uint32_t (&pa)[S][3], const unsigned char* stage, const int (&live)[L::TB], float al, float* spec, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t v[L::TB][4][L::VP][L::VB / 4], vs[KV == KV_FP4 ? L::TB : 1][2];
    const unsigned char* at[2] = {stage + L::place(t, g * L::VB), stage + L::place(t + 4, g * L::VB)};
#pragma unroll
    for (int b = 0; b < L::TB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < L::VP; ++p) lds(v[b][i][p], at[i & 1] + b * L::UNIT + 8 * (i >> 1) * L::ROW + p * 128);
      if constexpr (KV == KV_FP4) {
        const unsigned char* x = stage + b * L::UNIT + kBlockTokens * L::ROW + t * (D / 16) + g * (D / 8) / 16;
#pragma unroll
        for (int n = 0; n < 2; ++n) vs[b][n] = x[8 * n * (D / 16)] | (uint32_t)x[(8 * n + 4) * (D / 16)] << 8;
      }
    }
#pragma unroll
    for (int b = 0; b < L::TB; ++b) {
      if (live[b] < kBlockTokens) {                                   // the same for the whole warp
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (t + 4 * (i & 1) + 8 * (i >> 1) < live[b]) continue;
          if constexpr (KV == KV_FP4) {
            vs[b][i >> 1] &= (i & 1) ? 0x00ffu : 0xff00u;
          } else {
#pragma unroll
            for (int p = 0; p < L::VP; ++p)
#pragma unroll
              for (int w = 0; w < L::VB / 4; ++w) v[b][i][p][w] = 0;
          }
        }
      }
      if constexpr (BF) {
        if (spec) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int p = 0; p < L::VP; ++p)
#pragma unroll
              for (int w = 0; w < L::VB / 4; ++w) {
                uint32_t& x = v[b][i][p][w];
                if ((x & 0x7f80u) == 0x7f80u) { atomicAdd(spec + L::v_channel(g, p * L::VC + 2 * w), bf16_lo(x)); x &= 0xffff0000u; }
                if ((x & 0x7f800000u) == 0x7f800000u) { atomicAdd(spec + L::v_channel(g, p * L::VC + 2 * w + 1), bf16_hi(x)); x &= 0xffffu; }
              }
        }
      }
    }
    auto add = [&](int c, const uint32_t (&f0)[L::TB], const uint32_t (&f1)[L::TB]) {
      float acc[4];
#pragma unroll
      for (int b = 0; b < L::TB; ++b) {
        if (b == 0) mma<BF, true>(acc, pa[0][0], pa[0][1], pa[1][0], pa[1][1], f0[0], f1[0]);
        else mma<BF>(acc, pa[2 * b][0], pa[2 * b][1], pa[2 * b + 1][0], pa[2 * b + 1][1], f0[b], f1[b]);
        if constexpr (LOW) mma<BF>(acc, pa[2 * b][2], 0u, pa[2 * b + 1][2], 0u, f0[b], f1[b]);
      }
      o[c][0] = fmaf(o[c][0], al, acc[0] + acc[2]);
      o[c][1] = fmaf(o[c][1], al, acc[1] + acc[3]);
    };
    // the same for the n-tiles (turned: halves of an m-tile) c and d
    auto add2 = [&](int c, int d, const uint32_t (&f0)[L::TB], const uint32_t (&f1)[L::TB], const uint32_t (&h0)[L::TB], const uint32_t (&h1)[L::TB]) {
      if constexpr (TURN) {
        float acc[4];
#pragma unroll
        for (int b = 0; b < L::TB; ++b) {
          if (b == 0) mma<BF, true>(acc, f0[0], h0[0], f1[0], h1[0], pa[0][0], pa[0][1]);
          else mma<BF>(acc, f0[b], h0[b], f1[b], h1[b], pa[b][0], pa[b][1]);
        }
        o[c][0] = fmaf(o[c][0], al, acc[0] + acc[1]);
        o[d][0] = fmaf(o[d][0], al, acc[2] + acc[3]);
      } else {
        add(c, f0, f1);
        add(d, h0, h1);
      }
    };
    uint32_t f[4][L::TB], f2[4][L::TB];
    if constexpr (KV == KV_BF16) {
#pragma unroll
      for (int p = 0; p < L::VP; ++p)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
#pragma unroll
            for (int b = 0; b < L::TB; ++b) {
              f[0][b] = __byte_perm(v[b][0][p][w], v[b][1][p][w], odd ? 0x7632 : 0x5410);
              f2[0][b] = __byte_perm(v[b][2][p][w], v[b][3][p][w], odd ? 0x7632 : 0x5410);
            }
            add(8 * p + 2 * w + odd, f[0], f2[0]);
          }
    } else if constexpr (KV == KV_E4M3) {
#pragma unroll
      for (int w = 0; w < L::VB / 4; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int b = 0; b < L::TB; ++b) {
            const uint32_t x = __byte_perm(v[b][0][0][w], v[b][1][0][w], half ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v[b][2][0][w], v[b][3][0][w], half ? 0x7362 : 0x5140);
            e4m3x4_to_h2(x, f[0][b], f[1][b]);
            e4m3x4_to_h2(y, f2[0][b], f2[1][b]);
          }
          add2(4 * w + 2 * half, 4 * w + 2 * half + 1, f[0], f2[0], f[1], f2[1]);
        }
    } else {
      uint32_t sc[L::TB][2];
#pragma unroll
      for (int b = 0; b < L::TB; ++b) { sc[b][0] = e4m3x2_h2(vs[b][0]); sc[b][1] = e4m3x2_h2(vs[b][1]); }
#pragma unroll
      for (int w = 0; w < L::VB / 4; ++w)
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
#pragma unroll
          for (int b = 0; b < L::TB; ++b) {
            uint32_t x[4], y[4];
            auto pairs = [&](uint32_t p, uint32_t q) {
              return odd ? ((p >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u) : (p & 0x0f0f0f0fu) | ((q << 4) & 0xf0f0f0f0u);
            };
            e2m1x8_to_h2(pairs(v[b][0][0][w], v[b][1][0][w]), x);
            e2m1x8_to_h2(pairs(v[b][2][0][w], v[b][3][0][w]), y);
#pragma unroll
            for (int c = 0; c < 4; ++c) { f[c][b] = hmul2(x[c], sc[b][0]); f2[c][b] = hmul2(y[c], sc[b][1]); }
          }
#pragma unroll
          for (int c = 0; c < 4; c += 2) add2(8 * w + 2 * c + odd, 8 * w + 2 * c + 2 + odd, f[c], f2[c], f[c + 1], f2[c + 1]);
        }
    }
  }

  // The warp's state to shared memory: so [head][D], sm_m and sm_l [head].
  __device__ __forceinline__ void leave(float* so, float* sm_m, float* sm_l, const float* spec, int lane) {
    const int g = lane >> 2, t = lane & 3;
    if constexpr (TURN) {
      if (g == 0) { sm_m[t] = m; sm_l[t] = l; }
#pragma unroll
      for (int c = 0; c < L::NT; ++c) so[t * D + L::v_channel(g, c)] = o[c][0];
      return;
    }
    if (t == 0) { sm_m[g] = m; sm_l[g] = l; }
#pragma unroll
    for (int c = 0; c < L::NT; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int ch = L::v_channel(2 * t + e, c);
        float x = o[c][e];
        if constexpr (FEW) x += __shfl_xor_sync(0xffffffffu, x, 16);
        so[g * D + ch] = spec ? x + spec[ch] : x;
      }
  }
};

// One cluster of 1..8 CTAs per (row, KV head, group of eight query heads); its
// warps take the row's blocks in turn and the CTAs' parts merge through
// distributed shared memory. One launch, no scratch.
template <int D, int KV, bool FEW>
__global__ void __launch_bounds__(32 * kBaWarps, ba_per_sm(D) / kBaWarps) block_attention_kernel(const BlockAttnArgs a) {
  using L = Lay<D, KV>;
  using Warp = BlockWarp<D, KV, FEW>;
  constexpr bool BF = L::BF;
  __shared__ __align__(16) typename Warp::Frag frag[L::KS * 32];
  __shared__ __align__(16) uint2 frag_lo[Warp::LOW ? L::KS * 32 : 1];
  extern __shared__ __align__(128) unsigned char ring[];              // [warp][K stages, V stages]
  float* so = reinterpret_cast<float*>(ring);                         // then [warp][head][D]
  __shared__ float sm_m[kBaWarps][kBaHeads], sm_l[kBaWarps][kBaHeads], cta_m[kBaHeads], cta_l[kBaHeads], sm_fac[kBaHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int sp = (int)(blockIdx.x % (unsigned)a.cluster), pair = (int)(blockIdx.x / (unsigned)a.cluster);
  const int hb = pair % a.hblocks, h = pair / a.hblocks % a.nkv, row = pair / a.hblocks / a.nkv;
  const int G = a.nq / a.nkv, gn = min(kBaHeads, G - hb * kBaHeads);
  const size_t head0 = (size_t)row * a.nq + (size_t)h * G + hb * kBaHeads;
  const int g = Warp::TURN ? lane >> 3 : (lane >> 2) & (FEW ? 3 : 7), t = lane & 3;   // the head whose query the lane splits

  pdl_enter();
  Picks pk;
  const int pos = a.positions[row], seq = a.row_seq ? a.row_seq[row] : row;
  pk.sel = a.sel + ((size_t)row * a.nkv + h) * a.k;
  pk.k = a.k;
  pk.stride = a.cluster * warps;
  const int first = sp * warps + warp + lane * pk.stride;
  pk.at = first;
  pk.e2 = pk.entry();
  float x[D / 4];                                                     // head g's channels of this lane
#pragma unroll
  for (int i = 0; i < D / 4; i += 4) {
    const float4 q = g < gn ? __ldg(reinterpret_cast<const float4*>(a.q + (head0 + g) * D + L::q_channel(t, i)))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    x[i] = q.x; x[i + 1] = q.y; x[i + 2] = q.z; x[i + 3] = q.w;
  }
  const bool ok = pos >= 0 && pos / kBlockTokens < a.bt_stride && seq >= 0 && seq < a.nseq;
  if (!ok && tid == 0 && sp == 0 && h == 0 && hb == 0) set_err(a.err, MBT_DEV_POS_RANGE);
  pk.last = ok ? pos / kBlockTokens : -1;
  if (!ok) { pk.at = pk.k; pk.e2 = -1; }                              // no entry counts
  pk.table = a.bt + (size_t)(ok ? seq : 0) * a.bt_stride;
  pk.num_blocks = a.num_blocks;
  pk.err = a.err;
  pk.mask = 0;
  const unsigned char* kpool = reinterpret_cast<const unsigned char*>(a.kpool);
  const unsigned char* vpool = reinterpret_cast<const unsigned char*>(a.vpool);
  Warp w;
  unsigned char* mine = ring + warp * L::RING;
  const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(mine);
  // Steps in one body of code, or one for each stage. The former saves fetches of
  // instructions where a step is long or BF16 is read for few heads, the latter
  // registers. In a graph, us, one body against one per stage: 4-bit blocks of d = 64,
  // 510 rows of 32 + 2 x 8 heads over 48 59.7 and 63.6, 256 rows of 64 + 2 x 8 over 64 58.0
  // and 59.0; BF16 blocks of d = 128, 32 + 2 x 8 heads over 64, one row 8.2 and 8.6, 64
  // rows 48.1 and 47.8. The other way about, d = 128: 64 rows of 64 + 2 x 8 heads over 128
  // e4m3 blocks 52.8 and 52.1, 128 4-bit blocks 55.8 and 54.7, 64 BF16 blocks 51.8 and 51.5.
  constexpr bool ROLLED = L::TB == 4 || (BF && FEW);
  int blk[L::TB], live[kBaStages][L::TB];                             // of the last step and of those under way
  bool on[kBaStages];
  auto step = [&](int i) {                                            // the next step's blocks
    on[i] = pk.any();
#pragma unroll
    for (int b = 0; b < L::TB; ++b)
      if (on[i]) pk.take(blk[b], live[i][b], pos);
  };
  auto request = [&](bool there, int stage, bool v) {
    if (there) w.request(mine_at + ((v ? kBaStages : 0) + stage) * L::STAGE, v ? vpool : kpool, blk, a.nkv, h, lane);
    else asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto begin = [&]() {
#pragma unroll
    for (int i = 0; i < kBaStages; ++i) {
      step(i);
      request(on[i], i, false);
      request(on[i], i, true);
    }
  };
  begin();

  // The queries' fragments, while the first blocks are under way. A power of two
  // per head brings the largest into FP16's range, or (BF16) a tiny one away from
  // the smallest numbers: below 2^-9, so that D products with keys below 2^128, and
  // differences of such sums, stay in fp32's range, and no further than `fac`, which
  // takes scores back to the log2 domain, is a normal number.
  uint32_t big = 0;                                                   // largest magnitude's bits; a NaN's are larger than inf's
#pragma unroll
  for (int i = 0; i < D / 4; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
  const int ex = (int)(big >> 23), ks = (int)(__float_as_uint(a.k_scale) >> 23) - 127;
  const int e = BF ? (ex < 87 ? min(117 - ex, 122 + ks) : 0) : min(120, 140 - ex);
  const float up = __int_as_float((e + 127) << 23);
  float fac = 1.4426950408889634f / sqrtf((float)D) * a.k_scale * __int_as_float((127 - e) << 23);
  fac = fmaxf(fac, 1.2e-38f);                                         // masked scores (-inf) stay -inf
  if (big >= 0x7f800000u) fac = __int_as_float(0x7fc00000);           // a non-finite query: its row is NaN
  if (t == 0) sm_fac[g] = fac;                                        // every warp the same
  if constexpr (Warp::TURN) fac = __shfl_sync(0xffffffffu, fac, 8 * t);   // scores are of head t
#pragma unroll
  for (int st = 0; st < L::KS; ++st) {
    uint32_t h0, h1, m0, m1, l0, l1;
    split<BF>(x[4 * st] * up, x[4 * st + 1] * up, h0, m0, l0);
    split<BF>(x[4 * st + 2] * up, x[4 * st + 3] * up, h1, m1, l1);
    if constexpr (FEW && BF) {
      Warp::rows(h0, m0, l0, lane);
      Warp::rows(h1, m1, l1, lane);
    }
    if (st % warps == warp) {
      if constexpr (Warp::TURN) frag[st * 32 + lane] = lane & 4 ? make_uint2(m0, m1) : make_uint2(h0, h1);
      else frag[st * 32 + lane] = make_uint4(h0, m0, h1, m1);
      if constexpr (Warp::LOW) frag_lo[st * 32 + lane] = make_uint2(l0, l1);
    }
  }
  __syncthreads();

  float* spec = nullptr;
  w.start();
#pragma unroll 1
  while (true) {
    auto turn = [&](int at, int slot) {                               // the step in this stage and place of `live`
      float s[Warp::S][2];
      uint32_t pa[Warp::S][3];
      int now[L::TB];
      asm volatile("cp.async.wait_group %0;" ::"n"(2 * kBaStages - 1) : "memory");
      __syncwarp();
      w.scores(s, mine + at * L::STAGE, frag, frag_lo, lane);
#pragma unroll
      for (int b = 0; b < L::TB; ++b) now[b] = live[slot][b];
      if constexpr (ROLLED) {
        slot = kBaStages - 1;
#pragma unroll
        for (int i = 0; i < kBaStages - 1; ++i) {
          on[i] = on[i + 1];
#pragma unroll
          for (int b = 0; b < L::TB; ++b) live[i][b] = live[i + 1][b];
        }
      }
      __syncwarp();                                                   // the keys' stage may be refilled
      step(slot);
      request(on[slot], at, false);
      const float al = w.soften(s, pa, now, fac, lane);
      asm volatile("cp.async.wait_group %0;" ::"n"(2 * kBaStages - 1) : "memory");
      __syncwarp();
      w.values(pa, mine + (kBaStages + at) * L::STAGE, now, al, spec, lane);
      __syncwarp();
      request(on[slot], at, true);
    };
    if constexpr (ROLLED) {
      int at = 0;
#pragma unroll 1
      while (on[0]) {
        turn(at, 0);
        at = at == kBaStages - 1 ? 0 : at + 1;
      }
    } else {
      bool more = true;
#pragma unroll 1
      while (more) {
#pragma unroll
        for (int i = 0; i < kBaStages; ++i) {
          if (!on[i]) { more = false; break; }
          turn(i, i);
        }
      }
    }
    w.l = Warp::over_head(w.l, [](float x, float y) { return x + y; });
    if constexpr (!BF) break;
    // BF16 values may be infinite or NaN, and a product with a part that is 0 is
    // then NaN: such a warp goes through its blocks again and adds them apart.
    bool odd = false;
    if (!spec) {
#pragma unroll
      for (int c = 0; c < L::NT; ++c)
#pragma unroll
        for (int e = 0; e < Warp::E; ++e) odd |= !(fabsf(w.o[c][e]) <= 3.4e38f);
      odd = odd && w.l <= 3.4e38f;
    }
    if (!__any_sync(0xffffffffu, odd)) break;
    spec = reinterpret_cast<float*>(ring + warps * L::RING) + warp * D;
    for (int i = lane; i < D; i += 32) spec[i] = 0.f;
    __syncwarp();
    pk.at = first;
    pk.e2 = pk.entry();
    pk.mask = 0;
    w.start();
    begin();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                                                    // every ring is drained
  w.leave(so + warp * kBaHeads * D, sm_m[warp], sm_l[warp], spec, lane);
  __syncthreads();
  // an infinity counts whatever its share
  auto share = [](float x, float f) { return x * (fabsf(x) > 3.4e38f ? 1.f : f); };
  // What a part with maximum m counts by. fmaxf turns a NaN into nothing: a part without
  // a token is 0 then, also where the query makes the factor of its scores NaN (one
  // with tokens is NaN itself).
  auto weight = [](float m, float mu, float fac) { return ex2(fmaxf((m - mu) * fac, -INFINITY)); };
  for (int i = tid; i < gn * D; i += blockDim.x) {
    const int hr = i / D;
    float M = -INFINITY, Ls = 0.f, acc = 0.f;
    for (int v = 0; v < warps; ++v) M = fmaxf(M, sm_m[v][hr]);
    const float mu = M == -INFINITY ? 0.f : M;
    for (int v = 0; v < warps; ++v) {
      const float f = weight(sm_m[v][hr], mu, sm_fac[hr]);
      Ls = fmaf(sm_l[v][hr], f, Ls);
      acc += share(so[v * kBaHeads * D + i], f);
    }
    if (a.cluster == 1) {
      a.out[head0 * D + i] = Ls == 0.f ? 0.f : acc * (a.v_scale / Ls);
    } else {
      so[i] = acc;                                                    // of warp 0's part: read by this thread only
      if (i % D == 0) { cta_m[hr] = M; cta_l[hr] = Ls; }
    }
  }
  if (a.cluster == 1) return;
  cluster_sync_all();
  for (int i = sp * blockDim.x + tid; i < gn * D; i += a.cluster * blockDim.x) {
    float pm[kBaCluster], pl[kBaCluster], po[kBaCluster], M = -INFINITY, Ls = 0.f, acc = 0.f;
#pragma unroll
    for (int r = 0; r < kBaCluster; ++r) {
      const bool in = r < a.cluster;
      pm[r] = in ? ld_dsmem_f32(&cta_m[i / D], r) : -INFINITY;
      pl[r] = in ? ld_dsmem_f32(&cta_l[i / D], r) : 0.f;
      po[r] = in ? ld_dsmem_f32(&so[i], r) : 0.f;
      M = fmaxf(M, pm[r]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int r = 0; r < kBaCluster; ++r) {
      const float f = weight(pm[r], mu, sm_fac[i / D]);
      Ls = fmaf(pl[r], f, Ls);
      acc += share(po[r], f);
    }
    a.out[head0 * D + i] = Ls == 0.f ? 0.f : acc * (a.v_scale / Ls);
  }
  cluster_sync_all();                                                 // stay resident until the others have read
}

// CTAs of so many warps that an SM holds, by registers and by shared memory.
template <int D, int KV, bool FEW>
long long ba_places(int warps, int num_sms) {
  using L = Lay<D, KV>;
  using Warp = BlockWarp<D, KV, FEW>;
  constexpr int FIXED = L::KS * 32 * ((int)sizeof(typename Warp::Frag) + (Warp::LOW ? 8 : 0)) + 512 + 1024;   // fragments; sums; what a CTA is charged
  return (long long)num_sms * std::min(ba_per_sm(D) / warps, (228 << 10) / (warps * L::WARP + FIXED));
}

template <int D, int KV, bool FEW>
cudaError_t ba_launch(const BlockAttnArgs& in, long long pairs, int num_sms, cudaStream_t s) {
  using L = Lay<D, KV>;
  BlockAttnArgs a = in;
  // Four warps a CTA while one wave holds all pairs, then two, then one, and two again for
  // several waves. In a graph, us, four, three, two and one warps, 8 KV heads of 128, 64
  // blocks: BF16, 32 query heads, 40 rows 36, 34, 35, 48; 64 rows 61, 52, 49, 53; 112 rows
  // 83, 82, 95, 79; 256 rows 168, 169, 165, 181. e4m3, 64 query heads, 40 rows 25, 28, 29,
  // 41; 64 rows 44, 35, 32, 43; 128 rows 68, 61, 75, 58.
  a.warps = pairs <= ba_places<D, KV, FEW>(4, num_sms) ? 4 : pairs <= ba_places<D, KV, FEW>(2, num_sms) ? 2
          : pairs <= ba_places<D, KV, FEW>(1, num_sms) ? 1 : 2;
  // Clusters of a power of two while pairs are few: up to 4/3 CTAs per SM over BF16
  // caches, which bound by memory, 8/3 over the others, no warp with less than a step, or
  // from 33 pairs on than four blocks. In a graph, us, one, two, four and eight CTAs a
  // pair, 32 + 2 x 8 heads of 128 over 64 blocks (* taken; seven CTAs for 64 pairs 23):
  //   rows  BF16                      e4m3                     4-bit
  //   1     15.7 12.1  9.2  8.1*      9.6  8.2  6.7  5.6*      10.6  8.8  7.1  6.0*
  //   4     16.2 12.5 10.1* 11.7     10.6  9.4  7.9  8.6*      11.8 10.1  8.5  8.4*
  //   8     16.4 13.2* 14.1 23.6     10.8  9.8  9.9* 15.4      12.0 10.3  9.7* 15.9
  //   16    17.5* 19.4 30.1 36.1     11.5 12.8* 18.3 23.4      12.2 12.4* 18.5 24.1
  //   24    23.4* 26.7 33.3 48.3     14.6 15.9* 20.7 31.2      15.3 14.8* 20.3 32.0
  // and of shorter lists: 4 rows over 16 blocks 8.5 8.5 7.7* 9.8, 5.6 6.1* 5.7 7.0, 6.2 6.4*
  // 6.2 7.4; 6 rows over 16 blocks 8.6* 8.8 10.0 11.6, 6.0* 6.4 7.2 8.1, 6.3* 6.5 7.3 8.3; 8 over
  // 32 11.3 10.4* 11.7 21.1, 8.0 8.3* 8.5 14.7, 8.8 8.7* 8.4 15.5. d = 64, 8 rows over 256 4-bit
  // blocks: 20.7 13.4 11.4* 11.7.
  const long long room = (L::BF ? 4LL : 8LL) * num_sms / 3 / pairs, least = std::max(L::TB, pairs > 32 ? 4 : 1);
  const long long most = std::min(room, a.k / (kBaWarps * least));
  a.cluster = 1;
  while (a.warps == kBaWarps && 2 * a.cluster <= std::min<long long>(kBaCluster, most)) a.cluster *= 2;
  void* p[] = {&a};
  return launch_ex((const void*)block_attention_kernel<D, KV, FEW>, dim3((unsigned)(pairs * a.cluster)), dim3(32 * a.warps),
                   a.warps * L::WARP, s, p, pdl_pays(pairs * a.cluster, num_sms), 100, a.cluster > 1 ? a.cluster : 0);
}

template <int D, int KV, bool FEW>
cudaError_t ba_init() {
  return cudaFuncSetAttribute((const void*)block_attention_kernel<D, KV, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kBaWarps * Lay<D, KV>::WARP);
}

}  // namespace

cudaError_t launch_block_attention(const BlockAttnArgs& in, int num_sms, cudaStream_t s) {
  BlockAttnArgs a = in;
  a.hblocks = (a.nq / a.nkv + kBaHeads - 1) / kBaHeads;
  const long long pairs = (long long)a.n * a.nkv * a.hblocks;
  if (pairs * kBaCluster > 0x7fffffffLL || a.k > 0x7fffffff - 32 * kBaWarps * kBaCluster) return cudaErrorInvalidValue;
  const bool wide = a.d == 128;
  const bool few = a.nq / a.nkv <= 4;
  auto go = [&](auto kv) {
    constexpr int KV = decltype(kv)::value;
    return wide ? few ? ba_launch<128, KV, true>(a, pairs, num_sms, s) : ba_launch<128, KV, false>(a, pairs, num_sms, s)
                : few ? ba_launch<64, KV, true>(a, pairs, num_sms, s) : ba_launch<64, KV, false>(a, pairs, num_sms, s);
  };
  if (a.kv == KV_BF16) return go(std::integral_constant<int, KV_BF16>());
  if (a.kv == KV_E4M3) return go(std::integral_constant<int, KV_E4M3>());
  return go(std::integral_constant<int, KV_FP4>());
}

cudaError_t block_attention_init() {
  for (auto init : {ba_init<64, KV_BF16, false>, ba_init<128, KV_BF16, false>, ba_init<64, KV_BF16, true>, ba_init<128, KV_BF16, true>,
                    ba_init<64, KV_E4M3, false>, ba_init<128, KV_E4M3, false>, ba_init<64, KV_E4M3, true>, ba_init<128, KV_E4M3, true>,
                    ba_init<64, KV_FP4, false>, ba_init<128, KV_FP4, false>, ba_init<64, KV_FP4, true>, ba_init<128, KV_FP4, true>}) {
    const cudaError_t e = init();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mbt
