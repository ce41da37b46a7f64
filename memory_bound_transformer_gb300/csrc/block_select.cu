// Ranges of the keys in a cache block and the choice of blocks by them.
//
// key_bounds_kernel: per (block, KV head) and channel the smallest and largest
// key as 8-bit codes, rounded outwards on a power-of-two grid.
//
// block_select_kernel: for integers u = rint(q 2^(10 - x)) of the group's
// queries, P_i and N_i the sums of the positive and negative ones,
//   sum_g u_g . k <= sum_i P_i max k_i + N_i min k_i
// for every key of the block; the right side with the 8-bit codes is an exact
// integer (|.| < 2^29: P - N <= 2^14, codes <= 127, 128 channels), so that no
// order of summation can move a block over the border of the chosen ones.
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

// Channels 8 c .. 8 c + 7 of a token's key as four 16-bit pairs, exactly: BF16
// values as they are, e4m3 and 4-bit ones as FP16 (e2m1 * e4m3 has at most six
// significant bits and lies in FP16's range).
template <int D, int KV>
__device__ __forceinline__ void key_pairs(const unsigned char* unit, int token, int c, uint32_t (&p)[4]) {
  if constexpr (KV == KV_BF16) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(unit + token * 2 * D + 16 * c));
    p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
  } else if constexpr (KV == KV_E4M3) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(unit + token * D + 8 * c));
    p[0] = e4m3x2_to_h2bits(v.x); p[1] = e4m3x2_to_h2bits(v.x >> 16);
    p[2] = e4m3x2_to_h2bits(v.y); p[3] = e4m3x2_to_h2bits(v.y >> 16);
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(unit + token * (D / 2) + 4 * c));
    const uint32_t s = __ldg(unit + kBlockTokens * (D / 2) + token * (D / kFp4Group) + c / 2), g = e4m3x2_to_h2bits(s | s << 8);
    e2m1x8_to_h2(w, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(g));
  }
}

constexpr int kBoundsWarps = 8;

// One row per CTA, its KV heads over the warps. A lane holds eight channels; the
// lanes of a warp cover 256 / D tokens at a time. Tokens past the row's are
// replaced by its own.
template <int D, int KV>
__global__ void __launch_bounds__(32 * kBoundsWarps) key_bounds_kernel(const KeyBoundsArgs a) {
  constexpr int LANES = D / 8, TOK = 32 / LANES;
  constexpr bool BF = KV == KV_BF16;
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int pos, next;
  const int seq = row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, row, pos);
  if (seq < 0) {
    if (threadIdx.x == 0) set_err(a.err, MBT_DEV_POS_RANGE);
    return;
  }
  if (row + 1 < a.n && row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, row + 1, next) == seq &&
      next / kBlockTokens == pos / kBlockTokens)
    return;                                                          // the next row's work
  const int blk = a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens];
  if (blk < 0 || blk > a.num_blocks) {
    if (threadIdx.x == 0) set_err(a.err, MBT_DEV_BLOCK_RANGE);
    return;
  }
  constexpr size_t UNIT = KV == KV_BF16 ? kBlockTokens * D * 2 : KV == KV_E4M3 ? kBlockTokens * D : fp4_unit_bytes(D);
  const int c = lane % LANES, upto = pos % kBlockTokens;
  for (int h = warp; h < a.nkv; h += kBoundsWarps) {
    const size_t at = (size_t)blk * a.nkv + h;
    const unsigned char* unit = reinterpret_cast<const unsigned char*>(a.kpool) + at * UNIT;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < kBlockTokens / TOK; ++t) {
      uint32_t p[4];
      key_pairs<D, KV>(unit, min(t * TOK + lane / LANES, upto), c, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = t ? min_nan(lo[i], p[i], BF) : p[i];
        hi[i] = t ? max_nan(hi[i], p[i], BF) : p[i];
      }
    }
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = min_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o), BF);
        hi[i] = max_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o), BF);
      }
    float l[8], u[8];
    uint32_t big = 0;                                                // a NaN's bits are larger than an infinity's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = BF ? make_float2(bf16_lo(lo[i]), bf16_hi(lo[i])) : h2_to_float2(lo[i]);
      const float2 y = BF ? make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])) : h2_to_float2(hi[i]);
      l[2 * i] = x.x; l[2 * i + 1] = x.y;
      u[2 * i] = y.x; u[2 * i + 1] = y.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, max(__float_as_uint(l[i]) & 0x7fffffffu, __float_as_uint(u[i]) & 0x7fffffffu));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
    const bool bad = big >= 0x7f800000u;
    // big = f 2^x with f in [1/2, 1): 127 * 2^(x - 7) holds it up to f = 127 / 128
    const int e = max((int)(big >> 23) - 126 - ((big & 0x7fffffu) <= 0x7e0000u ? 7 : 6), -100);
    const float down = bad || big == 0 ? 0.f : __int_as_float((127 - e) << 23);
    uint32_t w[2][2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a product too small for fp32 is still on its side of 0
      float x = bad ? 0.f : floorf(l[i] * down), y = bad ? 0.f : ceilf(u[i] * down);
      if (down != 0.f && l[i] < 0.f) x = fminf(x, -1.f);
      if (down != 0.f && u[i] > 0.f) y = fmaxf(y, 1.f);
      w[0][i / 4] |= ((uint32_t)(int)x & 0xffu) << (8 * (i % 4));
      w[1][i / 4] |= ((uint32_t)(int)y & 0xffu) << (8 * (i % 4));
    }
    if (lane < LANES) {
      uint2* dst = reinterpret_cast<uint2*>(a.bounds + at * 2 * D) + c;
      dst[0] = make_uint2(w[0][0], w[0][1]);
      dst[LANES] = make_uint2(w[1][0], w[1][1]);
    }
    if (lane == 0) a.scales[at] = bad ? __int_as_float(0x7f800000) : big == 0 ? 0.f : __int_as_float((e + 127) << 23);
  }
}

// ---------------------------------------------------------------------------
// choice

constexpr int kSelWarps = 16;                // most warps of a CTA
constexpr int kSelFew = 8;                   // of one with up to 2048 blocks
constexpr int kSelLoads = 8;                 // 16-byte loads that a lane has under way
constexpr int kSelPerSm = 4;                 // such CTAs per SM
constexpr int kSelCluster = 8;               // most CTAs of a cluster
constexpr int kSelShare = MBT_SELECT_MAX_BLOCKS / kSelCluster;   // most blocks of a CTA
constexpr int kSelCollect = 2048;            // blocks up to which one CTA of a cluster chooses
constexpr int kBins = 256;
constexpr uint32_t kKept = 0xffffffffu;      // key of a block that is taken in any case; scores' are lower

// Dot product of four unsigned with four signed bytes, added to c.
__device__ __forceinline__ int dp4a_us(uint32_t u, uint32_t s, int c) {
  int r;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(s), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* p, uint32_t rank) {
  return __float_as_uint(ld_dsmem_f32(p, rank));
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

// A cluster per (row, KV head); its CTAs take equal runs of the context's blocks
// and leave their keys in shared memory. Histograms of 256 bins over the range
// that is left, summed over the cluster, narrow down the k-th largest key until at
// most 32 candidates are left, which are ranked, or a single value, of which the
// first are taken.
template <int D, int WARPS, int LOADS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) block_select_kernel(const BlockSelectArgs a) {
  constexpr int REC = 2 * D, LANES = REC / 16, PER = 32 / LANES;      // bytes of a range, lanes on one, ranges per load
  constexpr int BATCH = LOADS * PER, SAME = LANES / LOADS;            // ranges per round of loads, lanes left with one's sum
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint8_t digit[2][REC];                     // weights' low and high bytes
  __shared__ __align__(16) uint32_t hist[2][kBins], sum[kBins];
  __shared__ float group[16 * D];                                     // the group's queries
  __shared__ uint32_t red[kSelWarps][2], per_warp[kSelWarps][2];
  __shared__ uint32_t ends[2], counts[3], list[2][32];                // read by the cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int warps = WARPS, threads = 32 * WARPS;
  const int rank = (int)(blockIdx.x % (unsigned)a.cluster), pair = (int)(blockIdx.x / (unsigned)a.cluster);
  const int h = pair % a.nkv, row = pair / a.nkv, G = a.nq / a.nkv;
  int* sel = a.sel + (size_t)pair * a.k;
  int pos;
  const int seq = row_in_table(a.positions, a.row_seq, a.nseq, a.bt_stride, row, pos);
  const int held = seq < 0 ? 0 : pos / kBlockTokens + 1;
  const int* table = a.bt + (size_t)max(seq, 0) * a.bt_stride;
  if (seq < 0 && tid == 0 && rank == 0 && h == 0) set_err(a.err, MBT_DEV_POS_RANGE);
  if (held <= a.k) {                                                  // all of them; the cluster's CTAs agree
    for (int j = rank * threads + tid; j < a.k; j += a.cluster * threads) {
      if (j < held && (uint32_t)table[j] > (uint32_t)a.num_blocks) set_err(a.err, MBT_DEV_BLOCK_RANGE);
      sel[j] = j < held ? j : -1;
    }
    return;
  }
  // Few blocks: all keys go to the first CTA, which does the rest alone.
  const bool collect = a.cluster > 1 && held <= kSelCollect;
  if (collect) cluster_arrive();
  // this CTA's blocks are [j0, j0 + cnt), a warp's 32 at a time
  const int share = (held + a.cluster - 1) / a.cluster, j0 = min(rank * share, held), cnt = min(share, held - j0);
  const int l = lane % LANES;
  const unsigned char* ranges = reinterpret_cast<const unsigned char*>(a.bounds) + 16 * l;
  auto entry = [&](int i) { return i + lane < cnt ? __ldg(table + j0 + i + lane) : 0; };   // past the share: block 0, not used
  auto checked = [&](int id) {
    if ((uint32_t)id <= (uint32_t)a.num_blocks) return id;
    set_err(a.err, MBT_DEV_BLOCK_RANGE);
    return a.num_blocks;
  };
  uint4 v[LOADS];
  int i0 = 32 * warp, id = entry(i0), next = entry(i0 + 32 * warps);
  auto request = [&](int b) {
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int from = __shfl_sync(0xffffffffu, id, b + u * PER + lane / LANES);
      v[u] = ld_stream(ranges + ((size_t)from * a.nkv + h) * REC);
    }
  };
  id = checked(id);
  float scale = 0.f;
  if (i0 < cnt) {
    scale = __ldg(a.scales + (size_t)id * a.nkv + h);
  }

  // weights: the group's rounded queries
  const float* q = a.q + ((size_t)row * a.nq + (size_t)h * G) * D;
  uint32_t big = 0;
  for (int i = tid; i < G * D; i += threads) {
    const float x = __ldg(q + i);
    group[i] = x;
    big = max(big, __float_as_uint(x) & 0x7fffffffu);
  }
  big = __reduce_max_sync(0xffffffffu, big);
  if (lane == 0) red[warp][0] = big;
  for (int i = tid; i < kBins; i += threads) hist[0][i] = hist[1][i] = 0;
  if (tid == 0) counts[2] = 0;
  __syncthreads();
  big = __reduce_max_sync(0xffffffffu, lane < warps ? red[lane][0] : 0);
  int e;
  frexpf(__uint_as_float(big), &e);
  // 2^(10 - e) in two factors that fp32 holds; rint takes care of what is too small for it
  const float m1 = ldexpf(1.f, (10 - e) / 2), m2 = ldexpf(1.f, (10 - e) - (10 - e) / 2);
  for (int i = tid; i < D; i += threads) {
    int up = 0, down = 0;
    if (big != 0 && big < 0x7f800000u) {
      for (int g = 0; g < G; ++g) {
        const int u = (int)rintf(group[g * D + i] * m1 * m2);
        up += max(u, 0);
        down += max(-u, 0);
      }
    }
    digit[0][i] = (uint8_t)down; digit[1][i] = (uint8_t)(down >> 8);
    digit[0][D + i] = (uint8_t)up; digit[1][D + i] = (uint8_t)(up >> 8);
  }
  __syncthreads();
  const uint4 w0 = *reinterpret_cast<const uint4*>(digit[0] + 16 * l), w1 = *reinterpret_cast<const uint4*>(digit[1] + 16 * l);
  const int side = l < LANES / 2 ? -1 : 1;

  if (collect) cluster_wait();
#pragma unroll 1
  while (i0 < cnt) {
    const float scale_now = scale;
    const int ahead = i0 + 32 * warps;
#pragma unroll
    for (int b = 0; b < 32; b += BATCH) {
      if (i0 + b >= cnt) break;
      request(b);
      int dot[LOADS];
#pragma unroll
      for (int u = 0; u < LOADS; ++u) {
        const int lo = dp4a_us(w0.w, v[u].w, dp4a_us(w0.z, v[u].z, dp4a_us(w0.y, v[u].y, dp4a_us(w0.x, v[u].x, 0))));
        const int hi = dp4a_us(w1.w, v[u].w, dp4a_us(w1.z, v[u].z, dp4a_us(w1.y, v[u].y, dp4a_us(w1.x, v[u].x, 0))));
        dot[u] = side * (hi * 256 + lo);
      }
      const int total = group_sums<LANES, LOADS>(dot, lane);
      const int r = b + l / SAME * PER + lane / LANES, i = i0 + r, j = j0 + i;
      const float sc = __shfl_sync(0xffffffffu, scale_now, r);
      if (i < cnt && l % SAME == 0) {
        const float inf = __int_as_float(0x7f800000);
        const bool kept = j < a.keep_first || j >= held - a.keep_last;
        const uint32_t key = kept ? kKept : key_of(sc < inf ? (float)total * sc : inf);
        if (collect) st_dsmem_u32(keys + j, 0, key);
        else keys[i] = key;
      }
    }
    i0 = ahead;
    if (ahead < cnt) {
      id = checked(next);
      next = entry(ahead + 32 * warps);
      scale = __ldg(a.scales + (size_t)id * a.nkv + h);
    }
  }

  // From here on: the CTA's keys [0, n) of the blocks from `origin` on.
  int n = cnt, origin = j0;
  bool solo = a.cluster == 1;
  if (collect) {
    cluster_sync_all();
    if (rank) return;
    n = held;
    origin = 0;
    solo = true;
  } else {
    __syncthreads();
  }
  const int seg = (n + threads - 1) / threads * 32;                   // a warp's run of keys, eight times 32 at a time
  const int s0 = min(warp * seg, n), s1 = min(s0 + seg, n);
  auto eight = [&](int i, uint32_t (&k8)[8]) {                        // keys past the run read as 0, below all scores'
#pragma unroll
    for (int u = 0; u < 8; ++u) k8[u] = i + 32 * u + lane < s1 ? keys[i + 32 * u + lane] : 0;
  };

  // the range of keys
  uint32_t lowest = 0xffffffffu, highest = 0;
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k8[u] != kKept && k8[u]) { lowest = min(lowest, k8[u]); highest = max(highest, k8[u]); }
  }
  lowest = __reduce_min_sync(0xffffffffu, lowest);
  highest = __reduce_max_sync(0xffffffffu, highest);
  if (lane == 0) { red[warp][0] = lowest; red[warp][1] = highest; }
  __syncthreads();
  lowest = __reduce_min_sync(0xffffffffu, lane < warps ? red[lane][0] : 0xffffffffu);
  highest = __reduce_max_sync(0xffffffffu, lane < warps ? red[lane][1] : 0);
  if (!solo) {
    if (tid == 0) { ends[0] = lowest; ends[1] = highest; }
    cluster_sync_all();
    lowest = __reduce_min_sync(0xffffffffu, lane < a.cluster ? ld_dsmem_u32(&ends[0], lane) : 0xffffffffu);
    highest = __reduce_max_sync(0xffffffffu, lane < a.cluster ? ld_dsmem_u32(&ends[1], lane) : 0);
  }
  // The last `need` are to be found among the `left` keys in [base, base + 2^bits);
  // all above are taken.
  uint32_t base = lowest, need = a.k - a.keep_first - a.keep_last, left = held - a.keep_first - a.keep_last;
  int bits = highest > lowest ? 32 - __clz(highest - lowest) : 0;
  auto below_top = [&](uint32_t key) { return key - base <= (bits >= 32 ? 0xffffffffu : (1u << bits) - 1); };
#pragma unroll 1
  for (int turn = 0; bits > 0 && need > 0 && left > 32; ++turn) {
    uint32_t* mine = hist[turn & 1];
    const int shift = max(bits - 8, 0);
    for (int i = s0; i < s1; i += 256) {
      uint32_t k8[8];
      eight(i, k8);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (k8[u] != kKept && k8[u] >= base && below_top(k8[u])) atomicAdd(&mine[(k8[u] - base) >> shift], 1u);
    }
    if (solo) __syncthreads();
    else cluster_sync_all();
    if (tid < kBins) {
      if (!solo) {
        uint32_t c[kSelCluster], t = 0;
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) c[r] = r < a.cluster ? ld_dsmem_u32(&mine[tid], r) : 0;
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) t += c[r];
        sum[tid] = t;
      }
      hist[(turn + 1) & 1][tid] = 0;                                  // read by all before this turn's barrier
    }
    if (!solo) __syncthreads();
    // every warp: counts from the highest bin down
    const uint4* bins = reinterpret_cast<const uint4*>(solo ? mine : sum) + (31 - lane) * (kBins / 128);
    const uint4 c1 = bins[0], c0 = bins[1];
    const uint32_t c[8] = {c0.w, c0.z, c0.y, c0.x, c1.w, c1.z, c1.y, c1.x};
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += c[i];
    uint32_t before = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += u;
    }
    before -= t;
    const int owner = __ffs(__ballot_sync(0xffffffffu, before < need && need <= before + t)) - 1;
    uint32_t bin = 0, in_bin = 0, above = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (before < need && need <= before + c[i]) { bin = kBins - 1 - (lane * 8 + i); in_bin = c[i]; above = before; }
      before += c[i];
    }
    need -= __shfl_sync(0xffffffffu, above, owner);
    base += __shfl_sync(0xffffffffu, bin, owner) << shift;
    left = __shfl_sync(0xffffffffu, in_bin, owner);
    bits = shift;
    if (need == left) break;                                          // all of them
    __syncthreads();                                                  // the other histogram is clear
  }
  // Count the keys above the range (or kept), and list the candidates in it.
  const bool ranked = left <= 32 && need > 0;
  auto kind = [&](uint32_t key) {                                     // 2 taken, 1 in the last range, 0 not
    if (key == kKept) return 2;
    if (need == 0 || key < base) return 0;
    return below_top(key) ? 1 : 2;
  };
  uint32_t sure = 0, tied = 0;                                        // of this lane, then of the warp
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = kind(k8[u]);
      sure += t == 2;
      tied += t == 1;
      if (ranked && t == 1) {
        const uint32_t at = atomicAdd(&counts[2], 1u);
        list[0][at] = k8[u];
        list[1][at] = origin + i + 32 * u + lane;
      }
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  tied = __reduce_add_sync(0xffffffffu, tied);
  if (lane == 0) { per_warp[warp][0] = sure; per_warp[warp][1] = tied; }
  __syncthreads();
  const uint32_t ps = lane < warps ? per_warp[lane][0] : 0, pt = lane < warps ? per_warp[lane][1] : 0;
  uint32_t sure_before = __reduce_add_sync(0xffffffffu, lane < warp ? ps : 0);
  uint32_t tied_before = __reduce_add_sync(0xffffffffu, lane < warp ? pt : 0);
  if (!solo) {
    const uint32_t cs = __reduce_add_sync(0xffffffffu, ps), ct = __reduce_add_sync(0xffffffffu, pt);
    if (tid == 0) { counts[0] = cs; counts[1] = ct; }
    cluster_sync_all();
    sure_before += __reduce_add_sync(0xffffffffu, lane < rank ? ld_dsmem_u32(&counts[0], lane) : 0);
    tied_before += __reduce_add_sync(0xffffffffu, lane < rank ? ld_dsmem_u32(&counts[1], lane) : 0);
  }
  // The last one taken: candidate (key, place), ranked by key, then by place.
  uint32_t last_key = base, last_j = 0xffffffffu, at = sure_before;
  if (ranked) {
    uint32_t first = 0;                                               // of CTA r's candidates
    int r = 0;
    if (!solo) {
      uint32_t upto = lane < a.cluster ? ld_dsmem_u32(&counts[2], lane) : 0;
#pragma unroll
      for (int o = 1; o < kSelCluster; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
#pragma unroll
      for (int i = 0; i < kSelCluster - 1; ++i) {
        const uint32_t u = __shfl_sync(0xffffffffu, upto, i);
        if (i + 1 < a.cluster && lane >= u) { r = i + 1; first = u; }
      }
    }
    const bool in = lane < left;
    uint32_t key = 0, j = 0;
    if (in) {
      key = solo ? list[0][lane] : ld_dsmem_u32(&list[0][lane - first], r);
      j = solo ? list[1][lane] : ld_dsmem_u32(&list[1][lane - first], r);
    }
    uint32_t ahead = 0;
    for (int i = 0; i < (int)left; ++i) {
      const uint32_t ki = __shfl_sync(0xffffffffu, key, i), ji = __shfl_sync(0xffffffffu, j, i);
      ahead += ki > key || (ki == key && ji < j);
    }
    const int it = __ffs(__ballot_sync(0xffffffffu, in && ahead == need - 1)) - 1;
    last_key = __shfl_sync(0xffffffffu, key, it);
    last_j = __shfl_sync(0xffffffffu, j, it);
    at += __popc(__ballot_sync(0xffffffffu, in && ahead < need && j < (uint32_t)(origin + s0)));
  } else {
    at += min(tied_before, need);
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = s0; i < s1; i += 256) {
    uint32_t k8[8];
    eight(i, k8);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t j = origin + i + 32 * u + lane;
      const int t = kind(k8[u]);
      bool one = ranked && (k8[u] > last_key || (k8[u] == last_key && j <= last_j));
      if (!ranked) {                                                  // equal keys: the first ones
        const uint32_t m1 = __ballot_sync(0xffffffffu, t == 1);
        one = tied_before + __popc(m1 & below) < need;
        tied_before += __popc(m1);
      }
      const bool taken = t == 2 || (t == 1 && one);
      const uint32_t m = __ballot_sync(0xffffffffu, taken);
      if (taken) sel[at + __popc(m & below)] = (int)j;
      at += __popc(m);
    }
  }
  if (!solo) cluster_sync_all();                                      // stay resident until the others have read
}

}  // namespace

cudaError_t launch_key_bounds(const KeyBoundsArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)a.n, 32 * kBoundsWarps, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.d == 64)
    return a.kv == KV_BF16 ? go(key_bounds_kernel<64, KV_BF16>) : a.kv == KV_E4M3 ? go(key_bounds_kernel<64, KV_E4M3>)
                                                                                  : go(key_bounds_kernel<64, KV_FP4>);
  return a.kv == KV_BF16 ? go(key_bounds_kernel<128, KV_BF16>) : a.kv == KV_E4M3 ? go(key_bounds_kernel<128, KV_E4M3>)
                                                                                 : go(key_bounds_kernel<128, KV_FP4>);
}

cudaError_t block_select_init() {
  for (const void* f : {(const void*)block_select_kernel<64, kSelWarps, kSelLoads>, (const void*)block_select_kernel<128, kSelWarps, kSelLoads>}) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelShare * 4);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_block_select(const BlockSelectArgs& a, int num_sms, cudaStream_t s) {
  BlockSelectArgs args = a;
  const long long pairs = (long long)a.n * a.nkv;
  if (pairs * kSelCluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  // four CTAs of eight warps per SM; no CTA with less than 32 blocks of a full table per warp
  const long long want = std::min<long long>((a.bt_stride + 255) / 256, (long long)kSelPerSm * num_sms / pairs);
  args.cluster = (int)std::max<long long>(want, (a.bt_stride + kSelShare - 1) / kSelShare);
  args.cluster = std::max(1, std::min(args.cluster, kSelCluster));
  const int share = (a.bt_stride + args.cluster - 1) / args.cluster;
  const bool few = share <= 2048;
  const void* f = a.d == 64 ? few ? (const void*)block_select_kernel<64, kSelFew, kSelLoads> : (const void*)block_select_kernel<64, kSelWarps, kSelLoads>
                            : few ? (const void*)block_select_kernel<128, kSelFew, kSelLoads> : (const void*)block_select_kernel<128, kSelWarps, kSelLoads>;
  void* p[] = {&args};
  return launch_ex(f, dim3((unsigned)(pairs * args.cluster)), dim3(32 * (few ? kSelFew : kSelWarps)),
                   (size_t)std::max(share, std::min(a.bt_stride, kSelCollect)) * 4, s, p, false, -1, args.cluster > 1 ? args.cluster : 0);
}

}  // namespace mbt
