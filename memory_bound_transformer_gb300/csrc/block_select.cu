// Ranges of the keys in a cache block and the choice of blocks by them.
//
// key_bounds_kernel: per (block, KV head) and channel the smallest and largest
// key as 8-bit codes, rounded outwards on a power-of-two grid. Reads the keys of
// the blocks written to once; bound by latency for a step's rows (64 rows of 8
// heads of 128, BF16: 2.3 us in a graph) and short prompts (4084 rows of 8 x 128, e4m3:
// 5.2 us, of which an SM is at work 2600 to 9500 cycles: the look-up of the rows, few
// blocks a CTA, instructions fetched for the first time), and for long ones by
// the instructions per key (50021 rows of 8 x 64, 4-bit: 12.1 us, 1.5 TB/s, ALU pipe 64 %
// while active; with every lane encoding eight channels and no keys under way 53).
//
// block_select_kernel: for integers u = rint(q 2^(10 - x)) of the group's
// queries, P_i and N_i the sums of the positive and negative ones,
//   sum_g u_g . k <= sum_i P_i max k_i + N_i min k_i
// for every key of the block; the right side with the 8-bit codes is an exact
// integer (|.| < 2^29: P - N <= 2^14, codes <= 127, 128 channels), so that no
// order of summation can move a block over the border of the chosen ones. The
// codes only loosen the bound, by up to 1/63 of the block's largest key a channel; u
// moves it by up to 2^-10 of the group's largest query times the key. 8 bits and 11
// keep a range at 1/32 of a BF16 block's bytes and the sum inside 32 bits. What is
// attended to is not rounded.
// Bound by the gather of the ranges, 2 d bytes each (6.2 TB/s alone for 256): four
// byte products per instruction, on two bytes of each weight. Measured in a graph,
// us, 32 + 2 x 8 heads of 128: one row over 2048 blocks 8.1 (five round trips, the
// choice 2.6 of them); 64 rows over 1000 to 2048 blocks 40 (64 heads; 5.0 TB/s, the
// scores alone 35); two rows over 62500 blocks 55.5 (4.7 TB/s), one 40.
#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "../../include/mbt_ops.h"

namespace mbt {

namespace {

// Row i's sequence if its position and sequence are inside the table, else -1.
__device__ __forceinline__ int row_in_table(const int* positions, const int* row_seq, int nseq, int bt_stride, int i, int& pos) {
  pos = positions[i];
  const int seq = row_seq ? row_seq[i] : i;
  return pos >= 0 && pos / kBlockTokens < bt_stride && seq >= 0 && seq < nseq ? seq : -1;
}

// ---------------------------------------------------------------------------
// ranges

__device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b, bool bf) {
  uint32_t r;
  if (bf) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b, bool bf) {
  uint32_t r;
  if (bf) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Channels 8 c .. 8 c + 7 of a token's key as they lie in the cache, and as four
// 16-bit pairs, exactly: BF16 values as they are, e4m3 and 4-bit ones as FP16
// (e2m1 * e4m3 has at most six significant bits and lies in FP16's range).
template <int D, int KV>
struct Key8 {
  uint32_t w[KV == KV_BF16 ? 4 : KV == KV_E4M3 ? 2 : 1], scale;
  __device__ __forceinline__ void load(const unsigned char* unit, int token, int c) {
    if constexpr (KV == KV_BF16) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(unit + token * 2 * D + 16 * c));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (KV == KV_E4M3) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(unit + token * D + 8 * c));
      w[0] = v.x; w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(unit + token * (D / 2) + 4 * c));
      scale = __ldg(unit + kBlockTokens * (D / 2) + token * (D / kFp4Group) + c / 2);
    }
  }
  __device__ __forceinline__ void pairs(uint32_t (&p)[4]) const {
    if constexpr (KV == KV_BF16) {
      p[0] = w[0]; p[1] = w[1]; p[2] = w[2]; p[3] = w[3];
    } else if constexpr (KV == KV_E4M3) {
      p[0] = e4m3x2_to_h2bits(w[0]); p[1] = e4m3x2_to_h2bits(w[0] >> 16);
      p[2] = e4m3x2_to_h2bits(w[1]); p[3] = e4m3x2_to_h2bits(w[1] >> 16);
    } else {
      e2m1x8_to_h2(w[0], p);
      const uint32_t g = e4m3x2_to_h2bits(scale | scale << 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(g));
    }
  }
};

constexpr int kBoundsWarps = 8;
constexpr int kBoundsRows = 256;             // most rows of a CTA

// A CTA looks through `rows` neighbouring rows for those that their block is left
// to, then a warp takes a (block, KV head) at a time, the next one's keys under
// way: a lane holds eight channels, the lanes cover 256 / D tokens (those past the
// row's are replaced by its own). Smallest and largest stay 16-bit pairs; lanes of
// the same channels halve them among each other, so that each encodes its own.
template <int D, int KV>
__global__ void __launch_bounds__(32 * kBoundsWarps) key_bounds_kernel(const KeyBoundsArgs a) {
  constexpr int LANES = D / 8, TOK = 32 / LANES;
  constexpr bool BF = KV == KV_BF16;
  __shared__ int sm_blk[kBoundsRows], sm_upto[kBoundsRows], sm_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.x * a.rows + tid;
  pdl_enter();
  if (tid == 0) sm_count = 0;
  __syncthreads();
  if (tid < a.rows && row < a.n) {
    int pos, next;
    const int seq = row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, row, pos);
    const bool left = row + 1 < a.n && row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, row + 1, next) == seq &&
                      next / kBlockTokens == pos / kBlockTokens;      // to the next row
    if (seq < 0) {
      set_err(a.err, MBT_DEV_POS_RANGE);
    } else if (!left) {
      const int blk = a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens];
      if (blk < 0 || blk > a.num_blocks) {
        set_err(a.err, MBT_DEV_BLOCK_RANGE);
      } else {
        const int at = atomicAdd(&sm_count, 1);
        sm_blk[at] = blk;
        sm_upto[at] = pos % kBlockTokens;
      }
    }
  }
  __syncthreads();
  constexpr size_t UNIT = KV == KV_BF16 ? kBlockTokens * D * 2 : KV == KV_E4M3 ? kBlockTokens * D : fp4_unit_bytes(D);
  constexpr int LOADS = kBlockTokens / TOK, OWN = 4 / TOK;            // pairs that a lane encodes
  const int c = lane % LANES, count = sm_count;
  Key8<D, KV> key[LOADS];
  size_t next = 0;                                                    // the (block, head) whose keys are under way
  auto load = [&](int b, int h) {
    next = (size_t)sm_blk[b] * a.nkv + h;
    const unsigned char* unit = reinterpret_cast<const unsigned char*>(a.kpool) + next * UNIT;
#pragma unroll
    for (int t = 0; t < LOADS; ++t) key[t].load(unit, min(t * TOK + lane / LANES, sm_upto[b]), c);
  };
  int b = 0, h = warp;                                                // the heads of all blocks, over the warps in turn
  auto settle = [&]() { while (h >= a.nkv) { h -= a.nkv; ++b; } };
  settle();
  if (b < count) load(b, h);
  while (b < count) {
    const size_t at = next;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < LOADS; ++t) {
      uint32_t p[4];
      key[t].pairs(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo[k] = t ? min_nan(lo[k], p[k], BF) : p[k];
        hi[k] = t ? max_nan(hi[k], p[k], BF) : p[k];
      }
    }
    h += kBoundsWarps;
    settle();
    if (b < count) load(b, h);
    int ch = 8 * c;                                                   // the lane's first channel
#pragma unroll
    for (int o = 16, n = 2; o >= LANES; o >>= 1, n >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const uint32_t l = __shfl_xor_sync(0xffffffffu, up ? lo[k] : lo[n + k], o);
        const uint32_t h = __shfl_xor_sync(0xffffffffu, up ? hi[k] : hi[n + k], o);
        lo[k] = min_nan(up ? lo[n + k] : lo[k], l, BF);
        hi[k] = max_nan(up ? hi[n + k] : hi[k], h, BF);
      }
      ch += up ? 2 * n : 0;
    }
    float l[2 * OWN], u[2 * OWN];
    uint32_t big = 0;                                                 // a NaN's bits are larger than an infinity's
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const float2 x = BF ? make_float2(bf16_lo(lo[k]), bf16_hi(lo[k])) : h2_to_float2(lo[k]);
      const float2 y = BF ? make_float2(bf16_lo(hi[k]), bf16_hi(hi[k])) : h2_to_float2(hi[k]);
      l[2 * k] = x.x; l[2 * k + 1] = x.y;
      u[2 * k] = y.x; u[2 * k + 1] = y.y;
    }
#pragma unroll
    for (int k = 0; k < 2 * OWN; ++k)
      big = max(big, max(__float_as_uint(l[k]) & 0x7fffffffu, __float_as_uint(u[k]) & 0x7fffffffu));
    big = __reduce_max_sync(0xffffffffu, big);
    const bool bad = big >= 0x7f800000u;
    // big = f 2^x with f in [1/2, 1): 127 * 2^(x - 7) holds it up to f = 127 / 128
    const int e = max((int)(big >> 23) - 126 - ((big & 0x7fffffu) <= 0x7e0000u ? 7 : 6), -100);
    const float down = bad || big == 0 ? 0.f : __int_as_float((127 - e) << 23);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2 * OWN; ++k) {
      // a product too small for fp32 is still on its side of 0
      float x = bad ? 0.f : floorf(l[k] * down), y = bad ? 0.f : ceilf(u[k] * down);
      if (down != 0.f && l[k] < 0.f) x = fminf(x, -1.f);
      if (down != 0.f && u[k] > 0.f) y = fmaxf(y, 1.f);
      w[0] |= ((uint32_t)(int)x & 0xffu) << (8 * k);
      w[1] |= ((uint32_t)(int)y & 0xffu) << (8 * k);
    }
    int8_t* dst = a.bounds + at * 2 * D + ch;
    if constexpr (OWN == 2) {
      *reinterpret_cast<uint32_t*>(dst) = w[0];
      *reinterpret_cast<uint32_t*>(dst + D) = w[1];
    } else {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w[0];
      *reinterpret_cast<uint16_t*>(dst + D) = (uint16_t)w[1];
    }
    if (lane == 0) a.scales[at] = bad ? __int_as_float(0x7f800000) : big == 0 ? 0.f : __int_as_float((e + 127) << 23);
  }
}

// ---------------------------------------------------------------------------
// choice

constexpr int kSelWarps = 8;                 // warps of a CTA that chooses from one context
constexpr int kSelPerSm = 4;                 // such CTAs per SM (64 registers a thread)
constexpr int kSelCluster = 8;               // most CTAs of a cluster
// Widest table for which one CTA has all keys. One row of 8 KV heads over 2048 blocks
// 8.4 us (two launches 14.2), 4096 12.4 (14.6), 8192 20.3 (16.0); 64 rows over 4096 87
// (101), 8192 251 (183). By the table's width, which the host knows, not the contexts:
// in a wider table 48 rows over 2048 blocks take 54 us, not 39, one row 14.0, not 8.1.
constexpr int kSelOne = 4096;
constexpr int kPartWarps = 16;               // warps of a CTA that scores a part of a long context, two per SM
constexpr int kMergeWarps = 32;              // of one that chooses among the parts' candidates
constexpr int kPartMost = 8192;              // most blocks of a part
constexpr int kMergeSmem = 192 << 10;        // shared memory for the candidates of all parts
constexpr int kSelLoads = 8;                 // 16-byte loads that a lane has under way
constexpr int kBins = 1024;
constexpr uint32_t kKept = 0xffffffffu;      // key of a block that is taken in any case; scores' are lower, and not 0

// 16 bytes read once, past L1. Volatile: such loads are issued in a row.
__device__ __forceinline__ uint4 ld_range(const unsigned char* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}
// Dot product of four unsigned with four signed bytes, added to c.
__device__ __forceinline__ int dp4a_us(uint32_t u, uint32_t s, int c) {
  int r;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(s), "r"(c));
  return r;
}
__device__ __forceinline__ void st_dsmem_u32(const void* p, uint32_t rank, uint32_t x) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(r), "r"(x) : "memory");
}
// The two halves of a cluster barrier: past the second all its CTAs have started.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Order-preserving bits of a float that is not NaN; -0 counts as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// v[0 .. N - 1] of each lane, to sums over groups of LANES neighbouring lanes: a
// lane is left with the sum of v[its place in the group / (LANES / N)]. Half of the
// values change hands in each step.
template <int LANES, int N>
__device__ __forceinline__ int group_sums(int (&v)[N], int lane) {
  int o = LANES / 2;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int mine = lane & o ? v[n + i] : v[i], other = lane & o ? v[i] : v[n + i];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// A (row, KV head) and its context.
struct SelRow {
  int row, h, held;                          // held: blocks of the context, 0 for a row outside its table
  const int* table;
  bool bad;
};
__device__ __forceinline__ SelRow sel_row(const BlockSelectArgs& a, int pair) {
  SelRow r;
  r.h = pair % a.nkv;
  r.row = pair / a.nkv;
  int pos;
  const int seq = row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, r.row, pos);
  r.bad = seq < 0;
  r.held = r.bad ? 0 : pos / kBlockTokens + 1;
  r.table = a.bt + (size_t)max(seq, 0) * a.bt_stride;
  return r;
}

// Shared memory of the scores: the group's queries, then the two bytes of the
// weights, of -N for the low codes and of P for the high ones.
template <int D>
struct SelQuery {
  float q[16 * D];
  __align__(16) uint8_t digit[2][2 * D];
  uint32_t red[kPartWarps];
};

// Requests the group's queries (nothing depends on where the row is).
template <int D, int WARPS>
__device__ __forceinline__ uint32_t load_group(SelQuery<D>& m, const BlockSelectArgs& a, int row, int h) {
  const int G = a.nq / a.nkv;
  const float* q = a.q + ((size_t)row * a.nq + (size_t)h * G) * D;
  uint32_t big = 0;
  for (int i = threadIdx.x; i < G * D; i += 32 * WARPS) {
    const float x = __ldg(q + i);
    m.q[i] = x;
    big = max(big, __float_as_uint(x) & 0x7fffffffu);
  }
  return big;
}
// The weights from them; all threads call it, `big` from load_group.
template <int D, int WARPS>
__device__ __forceinline__ void weigh(SelQuery<D>& m, uint32_t big, int G) {
  const int tid = threadIdx.x, lane = tid & 31;
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) m.red[tid >> 5] = big;
  __syncthreads();
  big = __reduce_max_sync(0xffffffffu, lane < WARPS ? m.red[lane] : 0);
  int e;
  frexpf(__uint_as_float(big), &e);
  // 2^(10 - e) in two factors that fp32 holds; rint takes care of what is too small for it
  const float m1 = ldexpf(1.f, (10 - e) / 2), m2 = ldexpf(1.f, (10 - e) - (10 - e) / 2);
  for (int i = tid; i < D; i += 32 * WARPS) {
    int up = 0, down = 0;
    if (big != 0 && big < 0x7f800000u) {
      for (int g = 0; g < G; ++g) {
        const int u = (int)rintf(m.q[g * D + i] * m1 * m2);
        up += max(u, 0);
        down += max(-u, 0);
      }
    }
    m.digit[0][i] = (uint8_t)down; m.digit[1][i] = (uint8_t)(down >> 8);
    m.digit[0][D + i] = (uint8_t)up; m.digit[1][D + i] = (uint8_t)(up >> 8);
  }
  __syncthreads();
}

// Table entry i + lane of a run of cnt from j0 on; past its end block 0, not used.
__device__ __forceinline__ int sel_entry(const SelRow& w, int j0, int cnt, int i) {
  i += threadIdx.x & 31;
  return i < cnt ? __ldg(w.table + j0 + i) : 0;
}
__device__ __forceinline__ int first_entry(const SelRow& w, int j0, int cnt) { return sel_entry(w, j0, cnt, threadIdx.x & ~31); }

// Keys of the context's blocks [j0, j0 + cnt), 32 at a time per warp: a range is
// read by 16 or 8 neighbouring lanes. next: first_entry. put(place, key).
template <int D, int WARPS, class Put>
__device__ __forceinline__ void score_blocks(const SelQuery<D>& m, const BlockSelectArgs& a, const SelRow& w, int j0, int cnt, int next, Put put) {
  constexpr int REC = 2 * D, LANES = REC / 16, PER = 32 / LANES;      // bytes of a range, lanes on one, ranges per load
  constexpr int BATCH = kSelLoads * PER, SAME = LANES / kSelLoads;    // ranges per round of loads, lanes left with one's sum
  const int lane = threadIdx.x & 31, l = lane % LANES, side = l < LANES / 2 ? -1 : 1;
  const unsigned char* ranges = reinterpret_cast<const unsigned char*>(a.bounds) + 16 * l;
  const uint4 w0 = *reinterpret_cast<const uint4*>(m.digit[0] + 16 * l), w1 = *reinterpret_cast<const uint4*>(m.digit[1] + 16 * l);
#pragma unroll 1
  for (int i0 = threadIdx.x & ~31; i0 < cnt; i0 += 32 * WARPS) {
    int id = next;
    next = sel_entry(w, j0, cnt, i0 + 32 * WARPS);
    if ((uint32_t)id > (uint32_t)a.num_blocks) {
      set_err(a.err, MBT_DEV_BLOCK_RANGE);
      id = a.num_blocks;
    }
    const float scale = __ldg(a.scales + (size_t)id * a.nkv + w.h);
#pragma unroll
    for (int b = 0; b < 32; b += BATCH) {
      if (i0 + b >= cnt) break;
      uint4 v[kSelLoads];
#pragma unroll
      for (int u = 0; u < kSelLoads; ++u) {
        const int from = __shfl_sync(0xffffffffu, id, b + u * PER + lane / LANES);
        v[u] = ld_range(ranges + ((size_t)from * a.nkv + w.h) * REC);
      }
      int dot[kSelLoads];
#pragma unroll
      for (int u = 0; u < kSelLoads; ++u) {
        const int lo = dp4a_us(w0.w, v[u].w, dp4a_us(w0.z, v[u].z, dp4a_us(w0.y, v[u].y, dp4a_us(w0.x, v[u].x, 0))));
        const int hi = dp4a_us(w1.w, v[u].w, dp4a_us(w1.z, v[u].z, dp4a_us(w1.y, v[u].y, dp4a_us(w1.x, v[u].x, 0))));
        dot[u] = side * (hi * 256 + lo);
      }
      const int total = group_sums<LANES, kSelLoads>(dot, lane);
      const int r = b + l / SAME * PER + lane / LANES, i = i0 + r, j = j0 + i;
      const float sc = __shfl_sync(0xffffffffu, scale, r);
      if (i < cnt && l % SAME == 0) {
        const float inf = __int_as_float(0x7f800000);
        // no scale that is not finite: 0 times -infinity would be a NaN, whose bits are kKept
        put(i, j < a.keep_first || j >= w.held - a.keep_last ? kKept : key_of(fabsf(sc) < inf ? (float)total * sc : inf));
      }
    }
  }
}

// Adds one to bin off >> shift where off <= span.
__device__ __forceinline__ void count_in(uint32_t* bins, uint32_t off, uint32_t span, int shift) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(bins + (off >> shift));
  asm volatile("{\n .reg .pred p;\n setp.le.u32 p, %1, %2;\n @p red.shared.add.u32 [%0], 1;\n}\n" ::"r"(at), "r"(off), "r"(span) : "memory");
}

// The bin that holds the need-th of all counted ones from the highest bin down,
// its count, and the count above it. Every warp calls it for itself.
__device__ __forceinline__ void find_bin(const uint32_t* bins, uint32_t need, int lane, uint32_t& bin, uint32_t& in_bin, uint32_t& above) {
  constexpr int N = kBins / 128;                                      // groups of 128 bins, four to a lane
  uint4 c[N];
  uint32_t total[N];
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = *reinterpret_cast<const uint4*>(bins + 128 * i + 4 * lane);
#pragma unroll
  for (int i = 0; i < N; ++i) total[i] = __reduce_add_sync(0xffffffffu, c[i].x + c[i].y + c[i].z + c[i].w);
  uint4 v = c[0];
  uint32_t before = 0;
  int group = 0;
  bool done = false;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    if (!done && before + total[i] >= need) {
      done = true;
      group = i;
      v = c[i];
    }
    if (!done) before += total[i];
  }
  const uint32_t s = v.x + v.y + v.z + v.w;
  uint32_t upto = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_down_sync(0xffffffffu, upto, o);
    if (lane + o < 32) upto += u;
  }
  before += upto - s;
  const int owner = __ffs(__ballot_sync(0xffffffffu, before < need && need <= before + s)) - 1;
  const uint32_t q[4] = {v.w, v.z, v.y, v.x};
  uint32_t b = 0, n = 0, up = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (before < need && need <= before + q[i]) { b = 128 * group + 4 * lane + 3 - i; n = q[i]; up = before; }
    before += q[i];
  }
  bin = __shfl_sync(0xffffffffu, b, owner);
  in_bin = __shfl_sync(0xffffffffu, n, owner);
  above = __shfl_sync(0xffffffffu, up, owner);
}

// Shared memory of the choice.
struct Chooser {
  __align__(16) uint32_t hist[2][kBins];
  uint32_t red[kMergeWarps][3], list[2][32], listed;
};
__device__ __forceinline__ void clear(Chooser& m, int threads) {      // before the first barrier ahead of choose()
  for (int i = threadIdx.x; i < kBins / 2; i += threads) reinterpret_cast<uint4*>(m.hist)[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) m.listed = 0;
}

// The k largest of n > k keys get(i), of equal ones the first; keys kKept are
// among them, and at most k. put(place among the taken, i), in order. Histograms
// over the range that is left narrow down the k-th largest until at most 32
// candidates are left, which are ranked, or a single value, of which the first are
// taken. All threads call it.
template <int WARPS, class Get, class Put>
__device__ __forceinline__ void choose(Chooser& m, int n, int k, Get get, Put put) {
  constexpr int threads = 32 * WARPS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seg = (n + threads - 1) / threads * 32;                   // a warp's run of keys, eight times 32 at a time
  const int s0 = min(warp * seg, n), s1 = min(s0 + seg, n);
  auto eight = [&](int i, uint32_t (&k8)[8]) {                        // keys past the run read as 0
#pragma unroll
    for (int u = 0; u < 8; ++u) k8[u] = i + 32 * u + lane < s1 ? get(i + 32 * u + lane) : 0;
  };
  // The last `need` are to be found among the `left` keys in [base, top]; all above
  // are taken. First the range of all keys but 0 and kKept.
  uint32_t base = 0xffffffffu, top = 0, kept = 0;
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      base = min(base, k8[u] - 1);
      top = max(top, k8[u] + 1);
      kept += k8[u] == kKept;
    }
  }
  base = __reduce_min_sync(0xffffffffu, base);
  top = __reduce_max_sync(0xffffffffu, top);
  kept = __reduce_add_sync(0xffffffffu, kept);
  if (lane == 0) { m.red[warp][0] = base; m.red[warp][1] = top; m.red[warp][2] = kept; }
  __syncthreads();
  base = __reduce_min_sync(0xffffffffu, lane < WARPS ? m.red[lane][0] : 0xffffffffu) + 1;
  top = __reduce_max_sync(0xffffffffu, lane < WARPS ? m.red[lane][1] : 0) - 1;
  kept = __reduce_add_sync(0xffffffffu, lane < WARPS ? m.red[lane][2] : 0);
  uint32_t need = k - kept, left = n - kept;
  if (need == 0) base = top = kKept - 1;                              // no key; only kept ones are above
#pragma unroll 1
  for (int turn = 0; need > 0 && left > 32 && base < top; ++turn) {
    uint32_t* mine = m.hist[turn & 1];
    const uint32_t span = top - base;
    const int shift = max(22 - __clz(span), 0);
    for (int i = s0; i < s1; i += 256) {
      uint32_t k8[8];
      eight(i, k8);
#pragma unroll
      for (int u = 0; u < 8; ++u) count_in(mine, k8[u] - base, span, shift);
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += threads) m.hist[(turn + 1) & 1][i] = 0;   // read before this turn's barrier
    uint32_t bin, above;
    find_bin(mine, need, lane, bin, left, above);
    need -= above;
    base += bin << shift;
    top = min(top, base + ((1u << shift) - 1));
    if (need == left) break;                                          // all of them
    __syncthreads();                                                  // the other histogram is clear
  }
  __syncthreads();                                                    // `red` has been read by all
  // Count the keys above the range, and list the candidates in it.
  const bool ranked = left <= 32 && need > 0;
  uint32_t sure = 0, tied = 0;
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      sure += k8[u] > top;
      if (k8[u] - base <= top - base) {
        ++tied;
        if (ranked) {
          const uint32_t at = atomicAdd(&m.listed, 1u);
          m.list[0][at] = k8[u];
          m.list[1][at] = i + 32 * u + lane;
        }
      }
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  tied = __reduce_add_sync(0xffffffffu, tied);
  if (lane == 0) { m.red[warp][0] = sure; m.red[warp][1] = tied; }
  __syncthreads();
  uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? m.red[lane][0] : 0);   // taken before this warp's run
  uint32_t tied_before = __reduce_add_sync(0xffffffffu, lane < warp ? m.red[lane][1] : 0);
  // Taken are keys above last_key, and those equal to it up to place last_i.
  const bool cut = !ranked && need < left;                            // equal keys: the first `need`
  uint32_t last_key = base, last_i = 0xffffffffu;
  if (ranked) {
    const bool in = lane < left;
    const uint32_t key = in ? m.list[0][lane] : 0, i = in ? m.list[1][lane] : 0;
    uint32_t ahead = 0;
    for (int c = 0; c < (int)left; ++c) {
      const uint32_t kc = m.list[0][c], ic = m.list[1][c];
      ahead += kc > key || (kc == key && ic < i);
    }
    const int it = __ffs(__ballot_sync(0xffffffffu, in && ahead == need - 1)) - 1;
    last_key = __shfl_sync(0xffffffffu, key, it);
    last_i = __shfl_sync(0xffffffffu, i, it);
    at += __popc(__ballot_sync(0xffffffffu, in && ahead < need && i < (uint32_t)s0));
  } else {
    at += min(tied_before, need);
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t j = i + 32 * u + lane;
      bool same = k8[u] == last_key && j <= last_i;
      if (cut) {
        const uint32_t m1 = __ballot_sync(0xffffffffu, same);
        same = same && tied_before + __popc(m1 & below) < need;
        tied_before += __popc(m1);
      }
      const bool taken = k8[u] > last_key || same;
      const uint32_t t = __ballot_sync(0xffffffffu, taken);
      if (taken) put(at + __popc(t & below), j);
      at += __popc(t);
    }
  }
}

// Contexts of at most kSelOne blocks: a CTA per (row, KV head), or where those are
// few a cluster that shares the scores and leaves the choice to its first CTA, to
// whose shared memory the others write their keys.
template <int D>
__global__ void __launch_bounds__(32 * kSelWarps, kSelPerSm) block_select_kernel(const BlockSelectArgs a) {
  constexpr int threads = 32 * kSelWarps;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelQuery<D> mem;
  __shared__ Chooser chooser;
  const int tid = threadIdx.x;
  const int rank = (int)(blockIdx.x % (unsigned)a.cluster), pair = (int)(blockIdx.x / (unsigned)a.cluster);
  pdl_enter();
  const uint32_t big = load_group<D, kSelWarps>(mem, a, pair / a.nkv, pair % a.nkv);
  const SelRow w = sel_row(a, pair);
  int* sel = a.sel + (size_t)pair * a.k;
  if (w.bad && tid == 0 && rank == 0 && w.h == 0) set_err(a.err, MBT_DEV_POS_RANGE);
  if (w.held <= a.k) {                                                // all of them; the cluster's CTAs agree
    for (int j = rank * threads + tid; j < a.k; j += a.cluster * threads) {
      if (j < w.held && (uint32_t)w.table[j] > (uint32_t)a.num_blocks) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      sel[j] = j < w.held ? j : -1;
    }
    return;
  }
  const bool shared = a.cluster > 1;
  if (shared) cluster_arrive();
  const int share = (w.held + a.cluster - 1) / a.cluster, j0 = min(rank * share, w.held), cnt = min(share, w.held - j0);
  const int first = first_entry(w, j0, cnt);                          // under way while the weights are made
  clear(chooser, threads);
  weigh<D, kSelWarps>(mem, big, a.nq / a.nkv);
  if (shared) cluster_wait();
  score_blocks<D, kSelWarps>(mem, a, w, j0, cnt, first, [&](int i, uint32_t key) {
    if (shared) st_dsmem_u32(keys + j0 + i, 0, key);
    else keys[i] = key;
  });
  if (shared) {
    cluster_sync_all();
    if (rank) return;
  } else {
    __syncthreads();
  }
  choose<kSelWarps>(chooser, w.held, a.k, [&](int i) { return keys[i]; }, [&](uint32_t at, uint32_t j) { sel[at] = (int)j; });
}

// Longer ones, in two launches: each CTA scores a part of a context and leaves the
// k best of it, in order, in memory; then a CTA per (row, KV head) chooses among
// those. (A context's k best are among its parts' k best, and in the same order.)
__device__ __forceinline__ int part_blocks(const BlockSelectArgs& a, int held) { return (held + a.parts - 1) / a.parts; }

template <int D>
__global__ void __launch_bounds__(32 * kPartWarps, 2) block_candidates_kernel(const BlockSelectArgs a) {
  constexpr int threads = 32 * kPartWarps;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelQuery<D> mem;
  __shared__ Chooser chooser;
  const int part = (int)(blockIdx.x % (unsigned)a.parts), pair = (int)(blockIdx.x / (unsigned)a.parts);
  pdl_enter();
  const uint32_t big = load_group<D, kPartWarps>(mem, a, pair / a.nkv, pair % a.nkv);
  const SelRow w = sel_row(a, pair);
  if (w.held <= a.k) return;
  const int share = part_blocks(a, w.held), j0 = min(part * share, w.held), cnt = min(share, w.held - j0);
  const int take = min(a.k, share);
  uint32_t* ck = a.keys + (size_t)pair * a.cand + (size_t)part * take;
  int* cj = a.places + (size_t)pair * a.cand + (size_t)part * take;
  const int first = first_entry(w, j0, cnt);
  clear(chooser, threads);
  weigh<D, kPartWarps>(mem, big, a.nq / a.nkv);
  score_blocks<D, kPartWarps>(mem, a, w, j0, cnt, first, [&](int i, uint32_t key) { keys[i] = key; });
  __syncthreads();
  if (cnt <= take) {
    for (int i = threadIdx.x; i < cnt; i += threads) { ck[i] = keys[i]; cj[i] = j0 + i; }
    return;
  }
  choose<kPartWarps>(chooser, cnt, take, [&](int i) { return keys[i]; },
                     [&](uint32_t at, uint32_t i) { ck[at] = keys[i]; cj[at] = j0 + (int)i; });
}

__global__ void __launch_bounds__(32 * kMergeWarps) block_merge_kernel(const BlockSelectArgs a) {
  constexpr int threads = 32 * kMergeWarps;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ Chooser chooser;
  const int pair = (int)blockIdx.x;
  pdl_enter();
  const SelRow w = sel_row(a, pair);
  int* sel = a.sel + (size_t)pair * a.k;
  if (w.bad && threadIdx.x == 0 && w.h == 0) set_err(a.err, MBT_DEV_POS_RANGE);
  if (w.held <= a.k) {
    for (int j = threadIdx.x; j < a.k; j += threads) {
      if (j < w.held && (uint32_t)w.table[j] > (uint32_t)a.num_blocks) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      sel[j] = j < w.held ? j : -1;
    }
    return;
  }
  // every part but the last ones is full, so the candidates are one run
  const int share = part_blocks(a, w.held), take = min(a.k, share), full = w.held / share;
  const int n = full * take + min(take, w.held - full * share);
  const uint32_t* ck = a.keys + (size_t)pair * a.cand;
  const int* cj = a.places + (size_t)pair * a.cand;
  clear(chooser, threads);
  auto put = [&](uint32_t at, uint32_t i) { sel[at] = cj[i]; };
  if (n * 4LL <= kMergeSmem) {
    for (int i = threadIdx.x; i < n; i += 8 * threads) {
      uint32_t k8[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) k8[u] = i + u * threads < n ? ck[i + u * threads] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u * threads < n) keys[i + u * threads] = k8[u];
    }
    __syncthreads();
    if (n == a.k) {                                                   // cannot be fewer: the k best are among them
      for (int i = threadIdx.x; i < n; i += threads) put(i, i);
      return;
    }
    choose<kMergeWarps>(chooser, n, a.k, [&](int i) { return keys[i]; }, put);
  } else {
    __syncthreads();
    choose<kMergeWarps>(chooser, n, a.k, [&](int i) { return ck[i]; }, put);
  }
}

}  // namespace

cudaError_t launch_key_bounds(const KeyBoundsArgs& in, int num_sms, cudaStream_t s) {
  KeyBoundsArgs a = in;
  // all CTAs resident at once, four per SM (eight: 4084 rows 6.1 us against 5.2, 50021 rows
  // 13.6 against 12.6): most of a prompt's rows leave their block to the next
  a.rows = (int)std::min<long long>(kBoundsRows, (a.n + 4LL * num_sms - 1) / (4LL * num_sms));
  auto go = [&](auto kernel) {
    void* p[] = {&a};
    const unsigned ctas = (unsigned)((a.n + (long long)a.rows - 1) / a.rows);
    return launch_ex((const void*)kernel, dim3(ctas), dim3(32 * kBoundsWarps), 0, s, p, pdl_pays(ctas, num_sms), -1);
  };
  if (a.d == 64)
    return a.kv == KV_BF16 ? go(key_bounds_kernel<64, KV_BF16>) : a.kv == KV_E4M3 ? go(key_bounds_kernel<64, KV_E4M3>)
                                                                                  : go(key_bounds_kernel<64, KV_FP4>);
  return a.kv == KV_BF16 ? go(key_bounds_kernel<128, KV_BF16>) : a.kv == KV_E4M3 ? go(key_bounds_kernel<128, KV_E4M3>)
                                                                                 : go(key_bounds_kernel<128, KV_FP4>);
}

cudaError_t block_select_init() {
  for (const void* f : {(const void*)block_candidates_kernel<64>, (const void*)block_candidates_kernel<128>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kPartMost * 4);
    if (e != cudaSuccess) return e;
  }
  return cudaFuncSetAttribute((const void*)block_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMergeSmem);
}

cudaError_t block_select_plan(BlockSelectArgs* a, int num_sms) {
  const long long pairs = (long long)a->n * a->nkv, blocks = a->bt_stride;
  a->cluster = 1;
  a->parts = 0;
  a->cand = 0;
  if (blocks <= kSelOne) {
    // Clusters of a power of two, so that their CTAs have 256 blocks of a full table or
    // less, while one wave holds them with room to spare. One row over 2048 blocks: one
    // CTA per KV head 27.7 us, two 17.0, four 11.4, eight 8.6; over 600: 8.6, 8.1, 6.7, 6.7.
    // 12 rows over 2048: two 19.6, four 16.0, six 17.5, eight 20.1; 48 rows: one 39, two 47.
    while (a->cluster < kSelCluster && a->cluster * 32LL * kSelWarps < blocks && 2LL * a->cluster * pairs <= 7LL * num_sms / 2)
      a->cluster *= 2;
    return pairs * a->cluster > 0x7fffffffLL ? cudaErrorInvalidValue : cudaSuccess;
  }
  // One wave of parts, two per SM, none with less than 32 blocks per warp. One row over
  // 62500 blocks: 19 parts 39 us, 38 37, 57 47, 76 44; 4 rows over 8000: 4 parts 27, 9 24, 14 34.
  const long long least = (blocks + kPartMost - 1) / kPartMost, most = (blocks + 32 * kPartWarps - 1) / (32 * kPartWarps);
  a->parts = (int)std::max(least, std::min(most, 2LL * num_sms / pairs));
  const long long share = (blocks + a->parts - 1) / a->parts;
  a->cand = a->parts * std::min<long long>(a->k, share);
  return pairs * a->parts > 0x7fffffffLL ? cudaErrorInvalidValue : cudaSuccess;
}

size_t block_select_scratch(const BlockSelectArgs& a) {
  return (size_t)a.n * a.nkv * a.cand * (sizeof(uint32_t) + sizeof(int));
}

cudaError_t launch_block_select(const BlockSelectArgs& in, void* scratch, int num_sms, cudaStream_t s) {
  BlockSelectArgs a = in;
  void* p[] = {&a};
  const long long pairs = (long long)a.n * a.nkv;
  if (!a.parts) {
    const size_t smem = (size_t)a.bt_stride * sizeof(uint32_t);
    return launch_ex(a.d == 64 ? (const void*)block_select_kernel<64> : (const void*)block_select_kernel<128>,
                     dim3((unsigned)(pairs * a.cluster)), dim3(32 * kSelWarps), smem, s, p, pdl_pays(pairs * a.cluster, num_sms), -1, a.cluster > 1 ? a.cluster : 0);
  }
  a.keys = (uint32_t*)scratch;
  a.places = (int*)(a.keys + (size_t)pairs * a.cand);
  const size_t share = (a.bt_stride + a.parts - 1) / a.parts;
  const cudaError_t e =
      launch_ex(a.d == 64 ? (const void*)block_candidates_kernel<64> : (const void*)block_candidates_kernel<128>,
                dim3((unsigned)(pairs * a.parts)), dim3(32 * kPartWarps), share * sizeof(uint32_t), s, p, pdl_pays(pairs * a.parts, num_sms), -1);
  if (e != cudaSuccess) return e;
  return launch_pdl((const void*)block_merge_kernel, dim3((unsigned)pairs), dim3(32 * kMergeWarps),
                    (size_t)std::min<long long>(a.cand * 4LL, kMergeSmem), s, p);
}

}  // namespace mbt
