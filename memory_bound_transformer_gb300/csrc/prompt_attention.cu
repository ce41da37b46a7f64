// Causal attention of packed prompts over the paged KV cache (BF16, e4m3 or
// 4-bit), on the tcgen05 tensor cores:
//   o = sum_{t <= p} softmax_t(q . K_t / sqrt(d)) V_t   for the row at position p,
// one pass with the running maximum and sum of the softmax ("GPU Inference
// Internals", "Kernels: FlashAttention and the Memory Hierarchy": K and V tiles
// in on-chip memory, no score matrix in HBM).
//
// A CTA takes 128 query rows: T = 128 / G neighbouring tokens x the G query heads
// of one KV head, so grouped heads share every K and V tile and a short prompt
// fills the MMA's rows. Keys come in tiles of 128 tokens with two score buffers:
// while the softmax of tile j runs, the tensor cores do P V of tile j - 1 and the
// scores of tile j + 1.
//   warps 0-7        softmax and output: two threads per row, half of a tile's
//                    columns and half of the output channels each
//   warps 8-11       K loader: raw cache blocks to FP16 tiles in shared memory
//   warps 12-15      V loader
//   warps 16, 17     MMA issue of even and odd tiles (one issuing thread reaches
//                    an M = 128 MMA per ~100 cycles, two reach the pipe's 64)
// Accuracy is that of single-token attention: queries and probabilities enter
// as FP16 high and low parts (2^-22), two MMAs per product, low part first. So
// the floor is twice the formula's operations at the tensor rate. Probabilities
// are relative to 2^-14 of the row's largest so far (the factor cancels in o / l),
// which puts FP16's smallest steps at 2^-39 of it: many small ones behind one
// large one keep their share. e4m3 and 4-bit
// values widen to FP16 exactly. BF16 values get one exponent per 16 tokens (a
// cache block of a head) that puts the largest just below 2^16: exact down to
// 2^-29 of it, 2^-30 of it off below; scores take the exponent with the query
// scale, probabilities with the softmax's offset, both for free. In tiles of keys
// that some query row does not see whole, the last one or two, the exponent is
// per token and of the largest value up to it, and a row takes V relative to the
// largest exponent of what it attends to: nothing depends on later tokens.
// Queries and probabilities are the A operand in tensor memory (the tile of K
// or V is then the only operand read from shared memory: an M = N = 128 MMA with
// both there needs all of its bandwidth); probabilities take the place of the
// scores they came from. P V of each tile goes to a fresh accumulator that the
// softmax threads add to fp32 registers (IEEE adds; the tensor core's own
// accumulation truncates), which also makes the rescaling a fused multiply-add.
//
// Tensor memory (512 columns): scores / probabilities of even and odd tiles (128
// each: for 16 keys 8 columns of high and 8 of low parts), P V (128), queries
// (D / 2 high, D / 2 low).
//
// What bounds it: a key tile costs an SM 2550 cycles with a 4-bit cache, 2700
// with e4m3, 3900 with BF16 (widening takes that much more), the MMAs 2048 of
// them; the softmax warps' chain is the longer one (maximum 620 to 750,
// exponentials and split 1250, adding P V 500). A CTA's start (its place, its
// queries, the first scores) and its end cost 13,000 cycles and the launch of the
// next 2,000; at one CTA an SM nothing overlaps them, which is a third of the
// time at eight key tiles a CTA. 1000 tokens after 8200, 64 + 2 x 8 heads of 128,
// 4-bit: 389 us, 730 TFLOP/s of the formula's operations; 2048 tokens, 32 + 2 x 8
// heads: 72 us, 475; 4096, 64 + 2 x 8, e4m3: 424 us, 650; the same over BF16: 562.
// The keys of a tile of queries are not split: few tokens over a long context run
// on as many SMs as they have tiles (33 after 8200, 32 + 2 x 8 heads: 16 CTAs).
// CTAs that stay for all their query tiles were slower in each form tried (the
// next queries loaded by the softmax warps 443 us, by the V loaders 418, against
// 391 for the first of these at the time): the state they carry takes the loop's
// registers.
//
// A value of V that is not finite at a token some rows of the tile do not attend
// to would reach them as 0 x inf, and an infinity those that do as inf + 0 x inf
// (a probability's low part): the loader stores 0 for it and notes its block, and
// the rows that attend to it add it at the end. Of the tiles that every row sees
// whole they are added up once for all rows (the order of infinities and NaN does
// not matter); NaN, all that e4m3 and 4-bit caches have, can stay where it is
// there. BF16 keys that are not finite become zeros, too, and the rows that attend
// to them NaN.
#include <algorithm>
#include <climits>

#include "fp4.cuh"
#include "internal.h"
#include "pair_loop.h"
#include "tcgen05.cuh"

namespace mbt {

namespace {

constexpr int kPaRows = 128;                // query rows and keys per tile
constexpr int kPaThreads = 640;
constexpr uint32_t kPaO = 256, kPaQ = 384;  // TMEM columns (scores at 0 and 128)
constexpr int kPaIssueRegs = 32;
constexpr float kPaUp = 14.f;               // probabilities go up to 2^14

template <int D, int KV>
struct PaShape {
  static constexpr bool BF = KV == KV_BF16;           // tiles carry an exponent per block
  static constexpr int UNIT = KV == KV_FP4 ? fp4_unit_bytes(D) : kBlockTokens * D * (KV == KV_E4M3 ? 1 : 2);
  static constexpr int CPC = KV == KV_FP4 ? 32 : KV == KV_E4M3 ? 16 : 8;   // channels of a 16-byte raw chunk
  static constexpr int ROWB = D / CPC * 16;           // raw bytes of a token's codes
  static constexpr int PP = 64 / CPC;                 // chunks of a row in a 64-channel panel
  static constexpr int NCH = kBlockTokens * (D / CPC) / 32;   // chunks of a block per lane
  static constexpr int PANEL = kPaRows * 128;         // 128 tokens x 64 channels, 128-byte swizzle
  static constexpr int TILE = D / 64 * PANEL;
  // registers: 256 x 168 + 256 x 56 + 128 x 32 (BF16: 152 and 72, its loader holds
  // a raw block) = 640 x 96, what the block is launched with
  static constexpr int SOFTMAX_REGS = BF ? 152 : 168, LOAD_REGS = BF ? 72 : 56;
  static constexpr int LDO = D + 4;                   // output staging row, floats
  static constexpr int STAGES = BF ? 1 : 2;           // raw pairs of blocks of a loader warp
  static constexpr int SMEM = 4 * TILE + 8 * STAGES * 2 * UNIT + 1024;
  static_assert(kPaRows * LDO * 4 <= 4 * TILE, "the output fits in the drained tiles");
};

struct PaBars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], ofull[2], done[2], ofree, qfull;
};

// One try that may sleep in hardware for up to about a millisecond.
__device__ __forceinline__ bool pa_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(b)), "r"(parity), "r"(1000000u) : "memory");
  return ok != 0;
}
// Bounded wait; once any wait of the CTA has run out, the others give up too.
__device__ __forceinline__ bool pa_wait(uint64_t* b, uint32_t parity, volatile int* stop) {
  if (pa_try(b, parity)) return true;
  const long long t0 = clock64();
  while (!pa_try(b, parity)) {
    if (*stop) return false;
    if (clock64() - t0 > kTcWaitCycles) { *stop = 1; return false; }
  }
  return true;
}

__device__ __forceinline__ float pa_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values per register pair: one instruction for both.
__device__ __forceinline__ uint64_t pa_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 pa_unpair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t pa_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pa_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float pa_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// x = hi + lo as FP16 pairs (first value in the low half).
__device__ __forceinline__ void pa_split(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
  const float2 h = h2_to_float2(hi);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x1 - h.y), "f"(x0 - h.x));
}
__device__ __forceinline__ uint32_t pa_hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// tensor memory: 32 or 16 columns of this thread's lane to registers, 8 from them
__device__ __forceinline__ void pa_ld32(uint32_t t, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                 "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(t));
}
// Wait for the loads into r (threaded through, so no use moves before it).
__device__ __forceinline__ void pa_ld_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :: "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void pa_st8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void pa_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread of the (converged) warp.
__device__ __forceinline__ bool pa_elect() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}
// D += A B with A from tensor memory (rows in lanes, two 16-bit K elements per column).
__device__ __forceinline__ void pa_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Shared-memory descriptor of a tile whose rows are K (tokens) and whose
// 64-channel panels are N: 8-row groups 1024 bytes apart, panels `panel` bytes.
__device__ __forceinline__ uint64_t pa_mn_desc(uint32_t saddr, uint32_t panel) {
  return (sw128_desc(saddr) & ~((uint64_t)0x3fff << 16)) | ((uint64_t)(panel >> 4) << 16);
}

// One query tile: where its rows are and how far they see.
struct PaTile { int seq, row0, tokens, pos0, ctx; };   // pos0: position of the first token's row

// The tile of index `idx` among all sequences' tiles of T tokens, in order of
// the sequences; false past the last. One warp; every lane gets the result.
__device__ __forceinline__ bool pa_find(const PromptArgs& a, int T, long long idx, int lane, PaTile* t) {
  auto rows_of = [&](int s, int& lo, int& hi) {
    lo = hi = 0;
    if (s >= a.nseq) return;
    lo = min(max(a.cu[s], 0), a.n);
    hi = min(max(a.cu[s + 1], lo), a.n);
  };
  long long before = 0;
  int s0 = 0;
  for (; s0 + 256 < a.nseq; s0 += 256) {                             // many sequences: 256 per round trip
    int sum = 0, lo, hi;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      rows_of(s0 + 32 * k + lane, lo, hi);
      sum += (hi - lo + T - 1) / T;
    }
    const long long all = __reduce_add_sync(0xffffffffu, sum);
    if (before + all > idx) break;
    before += all;
  }
  for (; s0 < a.nseq; s0 += 32) {
    const int s = s0 + lane;
    int lo, hi;
    rows_of(s, lo, hi);
    const int ctx = s < a.nseq ? a.lens[s] : 0;
    const int mine = (hi - lo + T - 1) / T;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > idx);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int first = (int)(idx - before) - __shfl_sync(0xffffffffu, inc - mine, src);
      const int count = __shfl_sync(0xffffffffu, mine, src);
      lo = __shfl_sync(0xffffffffu, lo, src);
      hi = __shfl_sync(0xffffffffu, hi, src);
      const int at = (count - 1 - first) * T;                        // a sequence's last tiles (the longest) first
      t->seq = s0 + src;
      t->row0 = lo + at;
      t->tokens = min(T, hi - lo - at);
      t->ctx = __shfl_sync(0xffffffffu, ctx, src);
      t->pos0 = t->ctx - (hi - lo) + at;
      return true;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// ---------------------------------------------------------------------------
// loader

// A lane's chunk q of a block: panel, token and part of the token's panel row.
template <int D, int KV>
__device__ __forceinline__ void pa_chunk(int q, int lane, int& panel, int& row, int& part) {
  using S = PaShape<D, KV>;
  const int id = q * 32 + lane;
  panel = id / (kBlockTokens * S::PP);
  row = id / S::PP % kBlockTokens;
  part = id % S::PP;
}

// Requests one raw block.
template <int UNIT>
__device__ __forceinline__ void pa_request(uint32_t dst, const unsigned char* src, int lane) {
#pragma unroll
  for (int c = 0; c < UNIT; c += 512)
    if (c + 512 <= UNIT || c + lane * 16 < UNIT)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + c + lane * 16), "l"(src + c + lane * 16) : "memory");
}

// A lane's chunks of a raw block.
template <int D, int KV>
struct PaRaw {
  uint4 c[PaShape<D, KV>::NCH];
  uint16_t sc[PaShape<D, KV>::NCH];                                  // 4-bit: the two groups' scales
  __device__ __forceinline__ void read(const unsigned char* u, int lane) {
    using S = PaShape<D, KV>;
#pragma unroll
    for (int q = 0; q < S::NCH; ++q) {
      int panel, row, part;
      pa_chunk<D, KV>(q, lane, panel, row, part);
      c[q] = *reinterpret_cast<const uint4*>(u + row * S::ROWB + (panel * S::PP + part) * 16);
      if (KV == KV_FP4)
        sc[q] = *reinterpret_cast<const uint16_t*>(u + kBlockTokens * (D / 2) + row * (D / 16) + panel * 4 + part * 2);
    }
  }
};

__device__ __forceinline__ uint32_t pa_max2(uint32_t a, uint32_t b) {   // of two unsigned 16-bit pairs
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Exponent base of a BF16 block: FP16 exponent field = BF16 field - base, the
// largest value's at 30. `high` (uniform): some value is not finite, and the base
// is not to be used.
template <int D>
__device__ __forceinline__ int pa_block_base(const PaRaw<D, KV_BF16>& raw, bool& high) {
  uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
  for (int q = 0; q < PaShape<D, KV_BF16>::NCH; ++q) {
    m[0] = pa_max2(m[0], raw.c[q].x & 0x7fff7fffu);
    m[1] = pa_max2(m[1], raw.c[q].y & 0x7fff7fffu);
    m[2] = pa_max2(m[2], raw.c[q].z & 0x7fff7fffu);
    m[3] = pa_max2(m[3], raw.c[q].w & 0x7fff7fffu);
  }
  const uint32_t x = pa_max2(pa_max2(m[0], m[1]), pa_max2(m[2], m[3]));
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(x >> 16, x & 0xffffu));
  high = top >= 0x7f80u;
  return max(0, (int)(top >> 7) - 30);
}
// The same per token of a raw block's first `keep`, each over the tokens up to it.
// Two lanes per token, half of its channels each. Returns the first token with a
// value that is not finite, 16 where there is none.
template <int D>
__device__ __forceinline__ int pa_token_bases(const unsigned char* u, int keep, int lane, int* out) {
  constexpr int N = D / 16;                                          // 16-byte chunks per lane
  const int token = lane >> 1, half = lane & 1;
  const unsigned char* row = u + token * (2 * D) + half * N * 16;
  auto largest = [&](bool finite) {                                  // chunks in an order that keeps eight lanes in different banks
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 c = *reinterpret_cast<const uint4*>(row + ((i + token + 4 * half) & (N - 1)) * 16);
      const uint32_t w[4] = {c.x & 0x7fff7fffu, c.y & 0x7fff7fffu, c.z & 0x7fff7fffu, c.w & 0x7fff7fffu};
#pragma unroll
      for (int e = 0; e < 4; ++e) x = pa_max2(x, finite ? w[e] & ~__vcmpgeu2(w[e], 0x7f807f80u) : w[e]);
    }
    return token < keep ? max(x >> 16, x & 0xffffu) : 0u;
  };
  uint32_t m = largest(false);
  const uint32_t high = __ballot_sync(0xffffffffu, m >= 0x7f80u);
  if (high) m = largest(true);                                       // rare
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
#pragma unroll
  for (int o = 2; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m = max(m, t);
  }
  if (!half) out[token] = max(0, (int)(m >> 7) - 30);
  return high ? (__ffs(high) - 1) >> 1 : kBlockTokens;
}

// Values of a BF16 block that are not finite become zeros (rare).
template <int D>
__device__ __forceinline__ void pa_clear(PaRaw<D, KV_BF16>& raw) {
  auto clear = [](uint32_t& w) { w &= ~__vcmpgeu2(w & 0x7fff7fffu, 0x7f807f80u); };
#pragma unroll
  for (int q = 0; q < PaShape<D, KV_BF16>::NCH; ++q) { clear(raw.c[q].x); clear(raw.c[q].y); clear(raw.c[q].z); clear(raw.c[q].w); }
}

// Raw chunks to FP16 values in the tile (rows R0 .. R0 + 15). Tokens from `keep`
// on are stored as zeros; where `guard`, values that are not finite are too, and
// the return value says whether there were any. BF16: `base` is the block's
// exponent base, `tok` its tokens'; all values are finite (pa_clear).
// MODE: PA_WHOLE converts a block with no branch inside, which would keep the
// loop's chains from interleaving; PA_KEEP takes `keep`, `guard` and `tok`.
enum { PA_WHOLE, PA_KEEP };
template <int D, int KV, int MODE>
__device__ __forceinline__ bool pa_store(const PaRaw<D, KV>& raw, unsigned char* tile, int R0, int keep, bool guard, int lane, int base, const int* tok) {
  using S = PaShape<D, KV>;
  bool found = false;
#pragma unroll
  for (int q = 0; q < S::NCH; ++q) {
    int panel, row, part;
    pa_chunk<D, KV>(q, lane, panel, row, part);
    const uint32_t w[4] = {raw.c[q].x, raw.c[q].y, raw.c[q].z, raw.c[q].w};
    const int R = R0 + row;
    unsigned char* dst = tile + panel * S::PANEL + R * 128;
    const int b = MODE != PA_WHOLE && S::BF ? tok[row] : base;
    const uint32_t low = (uint32_t)((b + 1) << 7) * 0x10001u;        // BF16: smallest magnitude kept, FP16 exponent field 1
    const uint32_t shift = 0u - (uint32_t)(b << 10) * 0x10001u;
    uint32_t sc[2];
    if (KV == KV_FP4) {
      uint32_t s2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(raw.sc[q]));
      sc[0] = __byte_perm(s2, s2, 0x1010);
      sc[1] = __byte_perm(s2, s2, 0x3232);
    }
#pragma unroll
    for (int k = 0; k < S::CPC / 8; ++k) {                           // 8 channels = 16 bytes of the tile
      uint32_t v[4];
      if (KV == KV_FP4) {
        e2m1x8_to_h2(w[k], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pa_hmul2(v[e], sc[k >> 1]);
      } else if (KV == KV_E4M3) {
        v[0] = e4m3x2_to_h2bits(w[2 * k]); v[1] = e4m3x2_to_h2bits(w[2 * k] >> 16);
        v[2] = e4m3x2_to_h2bits(w[(2 * k + 1) & 3]); v[3] = e4m3x2_to_h2bits(w[(2 * k + 1) & 3] >> 16);
      } else {
        // (magnitude - (base << 7)) << 3 in both halves at once, sign kept
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = (pa_max2(w[e] & 0x7fff7fffu, low) * 8u + shift) | (w[e] & 0x80008000u);
      }
      if (MODE != PA_WHOLE && row >= keep) v[0] = v[1] = v[2] = v[3] = 0u;   // whatever the raw block's place held
      if (MODE != PA_WHOLE && !S::BF && guard) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bad = __vcmpeq2(v[e] & 0x7c007c00u, 0x7c007c00u);
          found |= bad != 0;
          v[e] &= ~bad;
        }
      }
      *reinterpret_cast<uint4*>(dst + (((part * (S::CPC / 8) + k) ^ (R & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  return found;
}

__device__ __forceinline__ float pa_exponent(int base) { return __int_as_float((base + 15) << 23); }   // 2^(base - 112)

// One cached value as fp32 (the slow path's).
template <int D, int KV>
__device__ float pa_value(const unsigned char* unit, int slot, int ch) {
  if (KV == KV_FP4) {
    uint32_t h[4];
    e2m1x8_to_h2(unit[slot * (D / 2) + ch / 2], h);
    const float2 f = h2_to_float2(h[0]);
    return (ch & 1 ? f.y : f.x) * e4m3_to_f32(unit[kBlockTokens * (D / 2) + slot * (D / 16) + ch / 16]);
  }
  if (KV == KV_E4M3) return e4m3_to_f32(unit[slot * D + ch]);
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(unit)[slot * D + ch] << 16);
}

// ---------------------------------------------------------------------------

template <int D, int KV>
__global__ void __launch_bounds__(kPaThreads, 1) prompt_attention_kernel(const PromptArgs a) {
  using S = PaShape<D, KV>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) PaBars bars;
  __shared__ uint32_t tmem_slot, sm_big[2][kPaRows];
  __shared__ float sm_mx[2][2][kPaRows];                             // halves' maxima: even and odd tiles
  __shared__ PaTile sm_tile;
  // first and last cache block with values of V replaced by zeros, of BF16's whole
  // tiles and of the others; first token whose K was
  __shared__ int sm_ok, sm_bad_whole[2], sm_bad_last_tiles[2], sm_bad_key;
  __shared__ float sm_bad_sum[S::BF ? D : 1];
  // BF16 exponent bases of the tiles' blocks, and of their tokens; a K tile's outlive its buffer
  __shared__ int sm_kbase[4][8], sm_vbase[2][8];
  __shared__ __align__(16) int sm_ktok[S::BF ? 4 : 1][kPaRows], sm_vtok[S::BF ? 2 : 1][kPaRows];
  __shared__ volatile int sm_stop;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int G = a.nq / a.nkv, T = kPaRows / G, h = (int)(blockIdx.x % (unsigned)a.nkv);

  if (warp == 0) {
    PaTile t;
    const bool ok = pa_find(a, T, blockIdx.x / (unsigned)a.nkv, lane, &t);
    if (lane == 0) {
      sm_ok = ok;
      if (ok) sm_tile = t;
      sm_stop = 0;
      sm_bad_whole[0] = sm_bad_last_tiles[0] = sm_bad_key = INT_MAX;
      sm_bad_whole[1] = sm_bad_last_tiles[1] = -1;
    }
  } else if (warp == 2) {
    if (S::BF)
      for (int i = lane; i < D; i += 32) sm_bad_sum[i] = 0.f;
  } else if (warp == 1) {
    if (lane == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars.kfull[s], 4); mbar_init(&bars.vfull[s], 4); mbar_init(&bars.pfull[s], 8);
        mbar_init(&bars.kempty[s], 1); mbar_init(&bars.vempty[s], 1); mbar_init(&bars.sfull[s], 1);
        mbar_init(&bars.ofull[s], 1); mbar_init(&bars.done[s], 1);
      }
      mbar_init(&bars.ofree, 8);
      mbar_init(&bars.qfull, 8);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  } else if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto release = [&]() {
    if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  };
  if (!sm_ok) { release(); return; }                                 // past the last tile
  const PaTile t = sm_tile;
  const bool bad_len = t.ctx < 0 || t.ctx > (long long)a.bt_stride * kBlockTokens;
  if (bad_len && tid == 0) set_err(a.err, MBT_DEV_SEQLEN_RANGE);
  const int last = bad_len ? -1 : t.pos0 + t.tokens - 1;             // the tile's last position
  const int ntiles = last < 0 ? 0 : last / kPaRows + 1;
  // row r of the tile is row r / G nq + r % G from here: a token's G heads are neighbours
  const size_t qrow0 = (size_t)t.row0 * a.nq + (size_t)h * G;
  if (!ntiles) {                                                     // nothing to attend to
    for (int i = tid; i < t.tokens * G * D; i += kPaThreads)
      a.out[(qrow0 + (size_t)(i / D / G) * a.nq + i / D % G) * D + i % D] = 0.f;
    release();
    return;
  }
  // BF16: the tiles that every row sees whole have an exponent per block, those after them one per token
  const int whole = S::BF ? min(max(t.pos0 + 1, 0) / kPaRows, ntiles) : ntiles;
  unsigned char* kbuf = smem;
  unsigned char* vbuf = smem + 2 * S::TILE;

  if (warp < 8) {
    // ---- softmax and output: row r of the tile, half `s` of the columns of
    // every tile and of the output channels ------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::SOFTMAX_REGS));
    const int s = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    // r / G for r < 128 and G <= 16 by a multiplication (exact: 128 * 16 < 2^16)
    const uint32_t inv = (0x10000u + G - 1) / G;
    auto row_of = [&](int rr) { return qrow0 + rr + (size_t)((rr * inv) >> 16) * (a.nq - G); };
    const int rows = t.tokens * G;
    const int pos = r < rows ? t.pos0 + (int)((r * inv) >> 16) : -1;
    constexpr int RL = D / 4, RW = 32 / RL;                          // lanes of a row's 16-byte chunks, rows per warp and access
    float fac, f1, f2;                                               // fac = f1 f2 above a lower limit
    constexpr float kFacMin = 1.2e-38f;                              // masked scores (-inf) stay -inf
    {
      // the query rows, whole rows at a time, into the V tiles' place (the V
      // loader waits), chunks swizzled by row
#pragma unroll 4
      for (int i = 0; i < kPaRows / 8; i += RW) {
        const int rr = warp * (kPaRows / 8) + i + lane / RL, ch = lane % RL;
        if (rr < rows)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                       ::"r"(smem_u32(vbuf) + rr * D * 4 + ((ch ^ (rr & 7)) << 4)),
                       "l"(a.q + row_of(rr) * D + ch * 4) : "memory");
      }
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
      named_bar(1, 256);
      // this half of the row's channels: scaled by a power of two that puts the
      // row's largest in [2^13, 2^14), high and low parts to tensor memory; fac
      // takes scores back to the log2 domain
      float x[D / 2];
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float4 v = r >= rows ? make_float4(0.f, 0.f, 0.f, 0.f)
            : *reinterpret_cast<const float4*>(vbuf + r * D * 4 + (((s * (D / 8) + i) ^ (r & 7)) << 4));
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < D / 2; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
      sm_big[s][r] = big;
      named_bar(2 + (warp & 3), 64);
      big = max(big, sm_big[s ^ 1][r]);
      const int e = min(120, 140 - (int)(big >> 23));
      const float up = __int_as_float((e + 127) << 23);
      // in two parts of about the same size: a product with a block's exponent
      // then leaves fp32's range only where the whole does
      f1 = 1.4426950408889634f / sqrtf((float)D) * a.k_scale;
      const int half = ((__float_as_int(f1) >> 23) - 127 - e) >> 1;
      f1 *= __int_as_float((127 - e - half) << 23);
      f2 = __int_as_float((127 + half) << 23);
      fac = fmaxf(f1 * f2, kFacMin);
#pragma unroll
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) pa_split(x[c + 2 * i] * up, x[c + 2 * i + 1] * up, hi[i], lo[i]);
        const uint32_t col = tmem + lanes + kPaQ + (uint32_t)(s * (D / 2) + c) / 2;
        pa_st8(col, hi);
        pa_st8(col + D / 2, lo);
      }
      pa_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.qfull);
    }
    float m = -INFINITY, l = 0.f, al_prev = 0.f;
    int vbase = -1000;                                               // BF16: o is in units of 2^(vbase - 112)
    constexpr int C = kPaRows / 2, E = D / 2;                        // columns and channels of this thread
    uint64_t o[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) o[i] = 0;
    // BF16: the factor of scores whose keys have this exponent base
    auto factor = [&](int base) { return pa_exponent(base) * f2 * f1; };
    // adds tile j's P V, rescaling what is there by `al`
    auto drain = [&](int j, float al) {
      if (!__all_sync(0xffffffffu, pa_wait(&bars.ofull[j & 1], (j >> 1) & 1, &sm_stop))) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < E; c += 32) {
        uint32_t v[32];
        pa_ld32(tmem + lanes + kPaO + s * E + c, v);
        pa_ld_wait32(v);
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          o[(c + k) / 2] = pa_fma2(o[(c + k) / 2], pa_pair(al, al), pa_pair(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.ofree);
      return true;
    };
    auto wait_all = [&](uint64_t* b, int j) { return __all_sync(0xffffffffu, pa_wait(b + (j & 1), (j >> 1) & 1, &sm_stop)); };
    auto columns = [&](int j) { return tmem + lanes + 128u * (j & 1) + s * C; };   // of tile j's scores
    float mx, al;
    // exchanges maxima with the rows' other warp; al: what the sum and the output are rescaled by
    auto meet = [&](int j, bool ok) {
      sm_mx[j & 1][s][r] = mx;
      ok = named_bar_and(2 + (warp & 3), 64, ok);
      mx = fmaxf(mx, sm_mx[j & 1][s ^ 1][r]);
      const float mn = fmaxf(m, S::BF ? mx - kPaUp : fmaf(mx, fac, -kPaUp));
      al = pa_ex2(m - (mn == -INFINITY ? 0.f : mn));
      m = mn;
      l *= al;
      return ok;
    };
    // probabilities are in place: their tile's P V may start; adds the one before it, done meanwhile
    auto next = [&](int j, float sum) {
      l += sum;
      pa_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.pfull[j & 1]);
      const bool ok = !j || drain(j - 1, al_prev);
      al_prev = al;
      return ok;
    };
    // P = 2^(score - maximum + 14), for BF16 times 2^(V's base - vbase)
    uint32_t v[2][32];
    float fcs[4];
    bool ok = pair_tiles(0, whole, true, [&](int j, bool ok) {
      ok = ok && wait_all(bars.sfull, j);
      tc_fence_after();
      const uint32_t sc = columns(j);
      pa_ld32(sc, v[0]);
      pa_ld32(sc + 32, v[1]);
      pa_ld_wait32(v[0]);
      pa_ld_wait32(v[1]);
      const int lim = pos - j * kPaRows - s * C;                     // columns 0..lim are seen
      if (!S::BF && __any_sync(0xffffffffu, lim < C - 1)) {
#pragma unroll
        for (int k = 0; k < C; ++k) if (k > lim) v[k / 32][k % 32] = 0xff800000u;
      }
      mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < C; c += 16) {                              // 16 columns: a cache block
        auto at = [&](int k) { return __uint_as_float(v[(c + k) / 32][(c + k) % 32]); };
        const float x0 = pa_max3(pa_max3(at(0), at(1), at(2)), at(3), at(4)), x1 = pa_max3(pa_max3(at(5), at(6), at(7)), at(8), at(9));
        const float y = pa_max3(pa_max3(x0, x1, at(10)), pa_max3(at(11), at(12), at(13)), fmaxf(at(14), at(15)));
        if (S::BF) fcs[c / 16] = factor(sm_kbase[j & 3][(s * C + c) / 16]);
        mx = fmaxf(mx, S::BF ? y * fcs[c / 16] : y);
      }
      return ok;
    }, meet, [&](int j) {
      const uint32_t sc = columns(j);
      if (S::BF) {                                                   // V's largest exponent so far
        if (!wait_all(bars.vfull, j)) return false;
        int top = vbase;
#pragma unroll
        for (int c = 0; c < kPaRows / 16; ++c) top = max(top, sm_vbase[j & 1][c]);
        al *= pa_ex2((float)(vbase - top));
        vbase = top;
      }
      const float mu = m == -INFINITY ? 0.f : m;
      uint64_t ls[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < C; c += 16) {
        const int blk = (s * C + c) / 16;
        const float fc = S::BF ? fcs[c / 16] : fac;
        const float off = S::BF ? (float)max(sm_vbase[j & 1][blk] - vbase, -80) : 0.f;   // below: nothing beside the largest
        uint64_t part[2] = {0, 0};
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float2 t2 = pa_unpair(pa_fma2(pa_pair(__uint_as_float(v[c / 32][(c + k) % 32]),
                                                      __uint_as_float(v[c / 32][(c + k + 1) % 32])),
                                              pa_pair(fc, fc), pa_pair(off - mu, off - mu)));
          const float p0 = pa_ex2(t2.x), p1 = pa_ex2(t2.y);
          uint64_t& sum = S::BF ? part[k / 2 & 1] : ls[k / 2 & 1];
          sum = pa_add2(sum, pa_pair(p0, p1));
          pa_split(p0, p1, hi[k / 2], lo[k / 2]);
        }
        if (S::BF) {
          const float back = pa_ex2(-off);
#pragma unroll
          for (int e = 0; e < 2; ++e) ls[e] = pa_fma2(part[e], pa_pair(back, back), ls[e]);
        }
        pa_st8(sc + c, hi);                                          // 16 keys: 8 columns high parts, 8 low parts
        pa_st8(sc + c + 8, lo);
      }
      const float2 l2 = pa_unpair(pa_add2(ls[0], ls[1]));
      return next(j, l2.x + l2.y);
    });
    // BF16: the tiles with tokens that some row does not see, an exponent per
    // token. 16 columns at a time, read twice, for the sake of registers: one loop
    // that held 64 with both kinds of exponents spilled in the whole tiles, too
    // (1000 tokens after 8200: 812 us against 570)
    if constexpr (S::BF) {
      auto tokens = [](const int* from, int (&to)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int4 x = reinterpret_cast<const int4*>(from)[i];
          to[4 * i] = x.x; to[4 * i + 1] = x.y; to[4 * i + 2] = x.z; to[4 * i + 3] = x.w;
        }
      };
      auto limit = [&](int j) { return pos - j * kPaRows - s * C; };  // columns 0..limit are seen
      auto most_of = [&](int j) { return min(last - j * kPaRows - s * C + 1, C); };   // those that some row sees
      ok = pair_tiles(whole, ntiles, ok, [&](int j, bool ok) {
        ok = ok && wait_all(bars.sfull, j);
        tc_fence_after();
        const uint32_t sc = columns(j);
        const int lim = limit(j), most = most_of(j), *ktok = sm_ktok[j & 3] + s * C;
        mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < most; c += 16) {
          uint32_t x[16];
          int kt[16];
          tmem_ld16_async(sc + c, x);
          tokens(ktok + c, kt);
          tmem_ld_wait16(x);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float y = __uint_as_float(x[k]) * factor(kt[k]);
            mx = fmaxf(mx, c + k <= lim ? y : -INFINITY);
          }
        }
        return ok;
      }, meet, [&](int j) {
        if (!wait_all(bars.vfull, j)) return false;
        const uint32_t sc = columns(j);
        const int lim = limit(j), most = most_of(j), *ktok = sm_ktok[j & 3] + s * C, *vtok = sm_vtok[j & 1];
        int top = vbase;
        const int seen = min(pos - j * kPaRows, kPaRows - 1);        // the row's last token in this tile
#pragma unroll
        for (int c = 0; c < kPaRows; c += kBlockTokens)
          if (c <= seen) top = max(top, vtok[min(c + kBlockTokens - 1, seen)]);
        al *= pa_ex2((float)(vbase - top));
        vbase = top;
        const float mu = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll 1
        for (int c = 0; c < C; c += 16) {
          uint32_t hi[8] = {}, lo[8] = {};
          if (c < most) {
            uint32_t x[16];
            int kt[16], vt[16];
            tmem_ld16_async(sc + c, x);
            tokens(ktok + c, kt);
            tokens(vtok + s * C + c, vt);
            tmem_ld_wait16(x);
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              float p[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float y = pa_ex2(fmaf(__uint_as_float(x[k + e]), factor(kt[k + e]), -mu));
                p[e] = c + k + e <= lim ? y : 0.f;
              }
              part += p[0] + p[1];
#pragma unroll
              for (int e = 0; e < 2; ++e) p[e] *= __int_as_float(max(127 + min(vt[k + e] - vbase, 0), 0) << 23);
              pa_split(p[0], p[1], hi[k / 2], lo[k / 2]);
            }
            sum += part;
          }
          pa_st8(sc + c, hi);
          pa_st8(sc + c + 8, lo);
        }
        return next(j, sum);
      });
    }
    if (ok) drain(ntiles - 1, al_prev);

    // all products and copies are done: rows through the drained tiles, stored whole
    sm_mx[0][s][r] = l;
    named_bar(1, 256);
    const float L = l + sm_mx[0][s ^ 1][r];
    // BF16: o / L, the exponent and the scale one after the other (the product of
    // the last two with 1 / L can be too small for fp32 where the output is not)
    // the query and (BF16) all keys; NaN where they are not
    const bool finite = max(sm_big[0][r], sm_big[1][r]) < 0x7f800000u && pos < sm_bad_key;
    const float wgt = pos < 0 ? 0.f : !finite ? __int_as_float(0x7fc00000) : S::BF ? 1.f / L : a.v_scale / L;
    const float unit = pa_exponent(max(vbase, 0));
    auto result = [&](float x) { return S::BF ? x * wgt * unit * a.v_scale : x * wgt; };
    float* stage = reinterpret_cast<float*>(smem) + r * S::LDO + s * E;
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float2 x = pa_unpair(o[i / 2]), y = pa_unpair(o[i / 2 + 1]);
      *reinterpret_cast<float4*>(stage + i) = make_float4(result(x.x), result(x.y), result(y.x), result(y.y));
    }
    auto unit_of = [&](int blk) {
      int id = a.bt[(size_t)t.seq * a.bt_stride + blk];
      if ((uint32_t)id > (uint32_t)a.num_blocks) id = a.num_blocks;
      return reinterpret_cast<const unsigned char*>(a.vpool) + ((size_t)id * a.nkv + h) * S::UNIT;
    };
    if (S::BF && sm_bad_whole[1] >= 0) {                             // rare: the same for all rows, so all threads search
      constexpr int N = S::UNIT / 16;                                // 16-byte chunks of a block
#pragma unroll 1
      for (long long i = tid; i < (sm_bad_whole[1] - sm_bad_whole[0] + 1LL) * N; i += 256) {
        const int at = (int)(i % N) * 8;
        const uint4 c = *reinterpret_cast<const uint4*>(unit_of(sm_bad_whole[0] + (int)(i / N)) + at * 2);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __uint_as_float(w[e / 2] << (e & 1 ? 0 : 16) & 0xffff0000u);
          if (!isfinite(x)) atomicAdd(&sm_bad_sum[(at + e) % D], x);
        }
      }
      named_bar(1, 256);
      for (int ch = 0; pos >= 0 && ch < E; ++ch) stage[ch] += sm_bad_sum[s * E + ch];
    }
    if (sm_bad_last_tiles[1] >= 0) {                                 // rare: at most two tiles
      const int end = min(pos, sm_bad_last_tiles[1] * kBlockTokens + kBlockTokens - 1);
      for (int tok = sm_bad_last_tiles[0] * kBlockTokens; tok <= end; ++tok) {
        const unsigned char* u = unit_of(tok / kBlockTokens);
        for (int ch = 0; ch < E; ++ch) {
          const float x = pa_value<D, KV>(u, tok % kBlockTokens, s * E + ch);
          if (!isfinite(x)) stage[ch] += x;
        }
      }
    }
    named_bar(1, 256);
#pragma unroll 4
    for (int i = 0; i < kPaRows / 8; i += RW) {
      const int rr = warp * (kPaRows / 8) + i + lane / RL, ch = lane % RL;
      if (rr < rows)
        *reinterpret_cast<float4*>(a.out + row_of(rr) * D + ch * 4) =
            *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + rr * S::LDO + ch * 4);
    }
  } else if (warp < 16) {
    // ---- loaders: two blocks of every K (or V) tile per warp; raw blocks are
    // requested as their stage of the ring falls free, block ids (lanes 0..7
    // hold a tile's) a tile before that
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::LOAD_REGS));
    const bool is_k = warp < 12;
    const int lw = warp & 3, nblk = (t.ctx + kBlockTokens - 1) / kBlockTokens;
    constexpr int BT = kPaRows / kBlockTokens;
    const int* bt = a.bt + (size_t)t.seq * a.bt_stride;
    const unsigned char* pool = reinterpret_cast<const unsigned char*>(is_k ? a.kpool : a.vpool) + (size_t)h * S::UNIT;
    unsigned char* ring = smem + 4 * S::TILE + (warp - 8) * S::STAGES * 2 * S::UNIT;
    uint64_t* full = is_k ? bars.kfull : bars.vfull;
    uint64_t* empty = is_k ? bars.kempty : bars.vempty;
    auto ids_of = [&](int j) { return lane < BT && j * BT + lane < nblk ? __ldg(bt + j * BT + lane) : 0; };
    int ids = ids_of(0);
    // one block of the warp's two in tile j, a copy group of its own
    auto request = [&](int j, int half) {
      if (j < ntiles) {
        if (half == 0 && lane < BT && j * BT + lane < nblk && (uint32_t)ids > (uint32_t)a.num_blocks) {   // out of range: the null block
          set_err(a.err, MBT_DEV_BLOCK_RANGE);
          ids = a.num_blocks;
        }
        const int at = half * 4 + lw;
        const unsigned char* src = pool + (size_t)__shfl_sync(0xffffffffu, ids, at) * a.nkv * S::UNIT;
        if (j * BT + at < nblk) pa_request<S::UNIT>(smem_u32(ring) + ((j % S::STAGES) * 2 + half) * S::UNIT, src, lane);
        if (half) ids = ids_of(j + 1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < 2 * S::STAGES; ++i) request(i / 2, i & 1);
    const bool go = is_k || __all_sync(0xffffffffu, pa_wait(&bars.qfull, 0, &sm_stop));   // the queries sit in V's place
    auto raw_block = [&](int j, int half) {                          // in its place of the ring, once it has arrived
      asm volatile("cp.async.wait_group %0;" ::"n"(2 * S::STAGES - 1) : "memory");
      __syncwarp();
      return ring + ((j % S::STAGES) * 2 + half) * S::UNIT;
    };
    auto wait_empty = [&](int j) {
      return j < 2 || __all_sync(0xffffffffu, pa_wait(&empty[j & 1], (j / 2 - 1) & 1, &sm_stop));
    };
    auto arrive_full = [&](int j) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[j & 1]);
    };
    auto note_bad = [&](bool bad, int tok0, int (&range)[2]) {
      if (bad) { atomicMin(&range[0], tok0 / kBlockTokens); atomicMax(&range[1], tok0 / kBlockTokens); }
    };
#pragma unroll 1
    for (int j = 0; go && j < whole; ++j) {
      if (!wait_empty(j)) break;
      unsigned char* tile = (is_k ? kbuf : vbuf) + (j & 1) * S::TILE;
#pragma unroll (S::BF ? 1 : 2)
      for (int half = 0; half < 2; ++half) {
        const int at = half * 4 + lw, tok0 = j * kPaRows + at * kBlockTokens;
        const bool guard = !S::BF && !is_k && tok0 + kBlockTokens - 1 > t.pos0;
        PaRaw<D, KV> raw;
        raw.read(raw_block(j, half), lane);
        __syncwarp();                                                // every lane has read: the place is free
        request(j + S::STAGES, half);
        const int keep = S::BF ? kBlockTokens : t.ctx - tok0;
        int base = 0;
        if constexpr (S::BF) {
          bool high;
          base = pa_block_base<D>(raw, high);
          if (high) {
            pa_clear<D>(raw);
            base = pa_block_base<D>(raw, high);
            if (is_k) atomicMin(&sm_bad_key, tok0);
            else note_bad(true, tok0, sm_bad_whole);
          }
          if (lane == 0) (is_k ? sm_kbase[j & 3] : sm_vbase[j & 1])[at] = base;
        }
        if (guard || keep < kBlockTokens) {
          note_bad(pa_store<D, KV, PA_KEEP>(raw, tile, at * kBlockTokens, keep, guard, lane, base, nullptr), tok0, sm_bad_last_tiles);
        } else {
          pa_store<D, KV, PA_WHOLE>(raw, tile, at * kBlockTokens, kBlockTokens, false, lane, base, nullptr);
        }
      }
      arrive_full(j);
    }
    if constexpr (S::BF) {
#pragma unroll 1
      for (int j = whole; go && j < ntiles; ++j) {
        if (!wait_empty(j)) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int at = half * 4 + lw, tok0 = j * kPaRows + at * kBlockTokens;
          int* tok = (is_k ? sm_ktok[j & 3] : sm_vtok[j & 1]) + at * kBlockTokens;
          unsigned char* tile = (is_k ? kbuf : vbuf) + (j & 1) * S::TILE;
          const int keep = last + 1 - tok0;                          // tokens that some row of the tile sees
          const unsigned char* place = raw_block(j, half);
          if (keep <= 0) {
            request(j + S::STAGES, half);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {                       // 16 rows of D / 64 panels, in any order
              const int id = i * 32 + lane;
              *reinterpret_cast<uint4*>(tile + id / 128 * S::PANEL + at * (kBlockTokens * 128) + id % 128 * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            continue;
          }
          PaRaw<D, KV> raw;
          const int bad = pa_token_bases<D>(place, keep, lane, tok);
          raw.read(place, lane);
          __syncwarp();
          request(j + S::STAGES, half);
          if (bad < kBlockTokens) {
            pa_clear<D>(raw);
            if (is_k) atomicMin(&sm_bad_key, tok0 + bad);
            else note_bad(true, tok0, sm_bad_last_tiles);
          }
          pa_store<D, KV, PA_KEEP>(raw, tile, at * kBlockTokens, keep, false, lane, 0, tok);
        }
        arrive_full(j);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPaIssueRegs));
    if (warp < 18) {
      // ---- MMA issue of tiles s, s + 2, ...: the whole warp follows, one elected
      // thread issues (with uniform control flow the descriptors stay in uniform
      // registers) ----------------------------------------------------------------
      const int s = warp - 16;
      const uint32_t sacc = tmem + 128u * s;
      constexpr uint32_t id_s = idesc_16(128, kPaRows, 1), id_o = idesc_16(128, D, 1) | (1u << 16);
      const uint64_t kt = sw128_desc(smem_u32(kbuf) + s * S::TILE), vt = pa_mn_desc(smem_u32(vbuf) + s * S::TILE, S::PANEL);
      bool ok = __all_sync(0xffffffffu, pa_wait(&bars.qfull, 0, &sm_stop));
      tc_fence_after();
#pragma unroll 1
      for (int i = 0, j = s; ok && j < ntiles; ++i, j += 2) {
        if (!(ok = __all_sync(0xffffffffu, pa_wait(&bars.kfull[s], i & 1, &sm_stop)))) break;
        tc_fence_after();
        if (pa_elect()) {
#pragma unroll
          for (int part = 1; part >= 0; --part)                      // low parts, then high
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              pa_mma(sacc, tmem + kPaQ + part * (D / 2) + 8 * k, kt + (((k >> 2) * S::PANEL + (k & 3) * 32) >> 4), id_s,
                     part == 0 || k > 0);
          umma_commit(&bars.sfull[s]);
          umma_commit(&bars.kempty[s]);
        }
        __syncwarp();
        ok = pa_wait(&bars.pfull[s], i & 1, &sm_stop) && pa_wait(&bars.vfull[s], i & 1, &sm_stop) &&
             (!j || pa_wait(&bars.ofree, (j - 1) & 1, &sm_stop));
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        if (pa_elect()) {
#pragma unroll
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < kPaRows / 16; ++k)
              pa_mma(tmem + kPaO, sacc + 16 * k + 8 * part, vt + ((k * 2048) >> 4), id_o, part == 0 || k > 0);
          umma_commit(&bars.ofull[s]);
          umma_commit(&bars.vempty[s]);
        }
        __syncwarp();
      }
      if (pa_elect()) umma_commit(&bars.done[s]);
      __syncwarp();
      if (!mbar_wait(&bars.done[s], 0)) sm_stop = 1;
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && sm_stop) set_err(a.err, MBT_DEV_WAIT_LIMIT);       // some warp's wait ran out
  release();
}

template <int D, int KV>
cudaError_t pa_launch(const PromptArgs& a, unsigned grid, cudaStream_t s) {
  PromptArgs args = a;
  void* p[] = {&args};
  return launch_ex((const void*)prompt_attention_kernel<D, KV>, dim3(grid), dim3(kPaThreads), PaShape<D, KV>::SMEM, s, p, false, -1);
}
template <int D>
cudaError_t pa_launch_d(const PromptArgs& a, unsigned grid, cudaStream_t s) {
  if (a.kv == KV_FP4) return pa_launch<D, KV_FP4>(a, grid, s);
  return a.kv == KV_E4M3 ? pa_launch<D, KV_E4M3>(a, grid, s) : pa_launch<D, KV_BF16>(a, grid, s);
}
template <int D, int KV>
cudaError_t pa_init() {
  return cudaFuncSetAttribute((const void*)prompt_attention_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              PaShape<D, KV>::SMEM);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s) {
  // as many CTAs as there can be tiles: a sequence's last may be short
  const int T = kPaRows / (a.nq / a.nkv);
  const long long grid = ((long long)a.n / T + std::min(a.nseq, a.n)) * a.nkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return a.d == 64 ? pa_launch_d<64>(a, (unsigned)grid, s) : pa_launch_d<128>(a, (unsigned)grid, s);
}

cudaError_t prompt_attention_init() {
  cudaError_t e = pa_init<64, KV_BF16>();
  if (e == cudaSuccess) e = pa_init<64, KV_E4M3>();
  if (e == cudaSuccess) e = pa_init<64, KV_FP4>();
  if (e == cudaSuccess) e = pa_init<128, KV_BF16>();
  if (e == cudaSuccess) e = pa_init<128, KV_E4M3>();
  if (e == cudaSuccess) e = pa_init<128, KV_FP4>();
  return e;
}

}  // namespace mbt
