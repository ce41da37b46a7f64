// Writing and reading the 4-bit paged KV cache (format in fp4.cuh).
//
// rope_kv_write_fp4_kernel: "RoPE + KV-cache write: rotate, then copy into
// paged blocks ... One read, one write" ("Kernels, Fusion & CUDA Graphs", "Fix
// 1: kernel fusion"), for a 4-bit cache. Rotate-half pairing: element i pairs
// with i + d/2 and turns by its position's table angle. Over each 16 channels
// of a key or value row x, with the tensor's scale g,
//   s = e4m3(max |x| / (6 g)),   code_i = e2m1(x_i / (s g)),
// both rounded to nearest (ties to even) and saturating.
//
// The codes are those of the exact real x: fp32 arithmetic moves a value that
// lies next to a border of the 4-bit grid, or a maximum next to a border of the
// e4m3 grid, to the other side (a few per million values). So every rounding
// is done for both ends of the interval that the fp32 error leaves; where the
// two differ, that code (or that block's scale) is decided again in 64 bits by
// exact comparisons with the borders: a code in about one warp in 500, a scale
// in one in 1500 for N(0, 1) rows.
//
// Bound by memory: one read of the projection's rows (4 bytes a value), one
// write of the rotated queries and of 9/16 byte a cached value. Its loads are a
// chain (position, then angles), so what counts is how many threads an SM
// holds: 4084 rows of 64 + 2 x 8 heads of 128 take 52.7 us (5.8 TB/s) at 32
// registers, 55.1 at 56; one thread per item of all rows and heads, with 64-bit
// divisions and the exact path's values kept, took 87. Heads that share a
// thread (2 or 4) load the angles once but finish together: 60 to 63 us. 64
// rows of 32 + 2 x 8 heads: 3.3 us.
#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

// e4m3 value of a non-negative code as a double.
__device__ __forceinline__ double e4m3_f64(int c) { return (double)e4m3_to_f32((uint32_t)c); }

// Where a thread's four channels and their partners lie: x is the channels' own
// address, y their partners' (the other half of the head), cs their angles
// (cos, sin interleaved); sign is -1 for channels of the first half, 1 for the
// second's, 0 where nothing is rotated.
struct Source { const float *x, *y, *cs; float sign; };

// One channel in 64 bits: both products are exact, their sum is rounded once.
__device__ __forceinline__ double exact_value(const Source& q, int i) {
  const double x = __ldg(q.x + i);
  if (q.sign == 0.f) return x;
  return fma((double)(q.sign * __ldg(q.y + i)), (double)__ldg(q.cs + 2 * i + 1), x * (double)__ldg(q.cs + 2 * i));
}

// The scale code of the block of four neighbouring lanes from exact values:
// the e4m3 code nearest to m / (6 g), ties to the even code, where `sc` is the
// code of the upper end of the interval. 6 g times the midpoint of two
// neighbouring e4m3 values is exact in a double (5 + 2 + 24 bits). Every lane
// of the warp calls it; blocks whose code is `sure` keep theirs.
__device__ __noinline__ int exact_scale(const Source q, float g, int sc, bool sure) {
  double m = 0.0;
  if (!sure)
    for (int i = 0; i < 4; ++i) m = fmax(m, fabs(exact_value(q, i)));
  for (int o = 1; o < 4; o <<= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (sure) return sc;
  const double g6 = 6.0 * g;
  for (; sc > 0; --sc) {
    const double mid = 0.5 * (e4m3_f64(sc - 1) + e4m3_f64(sc)) * g6;
    if (m > mid || (m == mid && !(sc & 1))) break;
  }
  return sc;
}

// Replaces the codes marked in `unsure` by those of the exact values: the e2m1
// code nearest to x / u (u = s g > 0), ties to the even code.
__device__ __noinline__ uint32_t exact_codes(const Source q, float g, int sc, uint32_t codes, uint32_t unsure) {
  const double u = e4m3_f64(sc) * g;
  for (int i = 0; i < 4; ++i) {
    const uint32_t mask = 0xfu << (4 * i);
    if (!(unsure & mask)) continue;
    const double x = exact_value(q, i), a = fabs(x);
    uint32_t c = 0;
    c += a > 0.25 * u;
    c += a >= 0.75 * u;
    c += a > 1.25 * u;
    c += a >= 1.75 * u;
    c += a > 2.5 * u;
    c += a >= 3.5 * u;
    c += a > 5.0 * u;
    codes = (codes & ~mask) | (c | (x < 0.0 ? 8u : 0u)) << (4 * i);
  }
  return codes;
}

struct Quad { float x[4]; float err; };                 // four neighbouring channels and a bound on their fp32 error
constexpr float kRel = 1.f / (1 << 21);                 // room for the roundings of the scaled values below

// Scale code of one 16-channel block held by four neighbouring lanes, for the
// upper end of the interval; 0x7f for a block with a NaN, 0x7e with an
// infinity. `sure`: the lower end has the same.
__device__ __forceinline__ int scale_code(const Quad& q, float inv6g, bool& sure) {
  float m = 0.f, e = q.err;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = fmaxf(m, fabsf(q.x[i]));
    nan |= q.x[i] != q.x[i];
  }
  if (nan) m = __uint_as_float(0x7fffffff);             // as bits, above every number
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m = __uint_as_float(max(__float_as_uint(m), __shfl_xor_sync(0xffffffffu, __float_as_uint(m), o)));
    e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
  }
  if (m != m) return 0x7f;
  if (!(m <= 3.0e38f)) return 0x7e;
  const int sc = f32_to_e4m3((m + e) * inv6g * (1.f + kRel));
  sure &= f32_to_e4m3(fmaxf(m - e, 0.f) * inv6g * (1.f - kRel)) == (uint8_t)sc;
  return sc;
}

// Codes of a lane's four channels (4 bits each, first channel lowest) for a
// scale code. `unsure` marks those that the fp32 error could move over a border
// (all bits that differ).
__device__ __forceinline__ uint32_t value_codes(const Quad& q, float g, int sc, uint32_t& unsure) {
  unsure = 0;
  if (sc == 0 || sc == 0x7f) return 0;                  // too small for the scale's grid, or a NaN
  const float inv = __fdiv_rn(1.f, e4m3_to_f32((uint32_t)sc) * g);
  float lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = q.x[i] * inv, d = fabsf(r) * kRel + q.err * inv;
    const bool fin = d <= 3.0e38f;                      // an infinity keeps its code
    lo[i] = fin ? r - d : r;
    hi[i] = fin ? r + d : r;
  }
  const uint32_t c = f32x2_to_e2m1x2(hi[0], hi[1]) | (f32x2_to_e2m1x2(hi[2], hi[3]) << 8);
  unsure = c ^ (f32x2_to_e2m1x2(lo[0], lo[1]) | (f32x2_to_e2m1x2(lo[2], lo[3]) << 8));
  return c;
}

constexpr int kWriteThreads = 128;

// A CTA takes one row and 128 / T of its heads. A thread holds channels
// 4i..4i+3 of a head and the same of its other half, requested before the
// position whose angles turn them. The four lanes of a 16-channel block are
// neighbours. The exact path loads its values again, so that it costs the
// other lanes no registers; 14 CTAs an SM, with a few spills, beat 9 without.
template <int D>
__global__ void __launch_bounds__(kWriteThreads, 14) rope_kv_write_fp4_kernel(const RopeKvFp4Args a) {
  constexpr int T = D / 8, H2 = D / 2, SL = kWriteThreads / T;       // threads per head row, channels per half, heads
  const int nh = a.nq + 2 * a.nkv, row = blockIdx.x;
  const int h0 = blockIdx.y * SL, hh = h0 + threadIdx.x / T, i4 = 4 * (threadIdx.x % T);
  const bool live = hh < nh, rotated = hh < a.nq + a.nkv, is_q = hh < a.nq;
  int pos = a.positions[row];
  const float* src = a.qkv + (size_t)row * a.ld_qkv + (size_t)min(hh, nh - 1) * D + i4;
  const float4 x1 = __ldg(reinterpret_cast<const float4*>(src)), x2 = __ldg(reinterpret_cast<const float4*>(src + H2));
  const bool pos_ok = pos >= 0 && pos < a.max_pos;
  if (!pos_ok) pos = 0;
  const float* cs = a.rope + (size_t)pos * D + 2 * i4;
  const float4 t0 = __ldg(reinterpret_cast<const float4*>(cs)), t1 = __ldg(reinterpret_cast<const float4*>(cs) + 1);
  int blk = -1;                                                      // the row's block, where the CTA has k or v heads
  if (h0 + SL > a.nq) {
    const int seq = a.row_seq ? a.row_seq[row] : row, jb = pos / kBlockTokens;
    if (pos_ok && seq >= 0 && seq < a.nseq && jb < a.bt_stride) blk = a.bt[(size_t)seq * a.bt_stride + jb];
    if (blk < 0 || blk > a.num_blocks) blk = -1;
  }
  const float in1[4] = {x1.x, x1.y, x1.z, x1.w}, in2[4] = {x2.x, x2.y, x2.z, x2.w};
  const float cc[4] = {t0.x, t0.z, t1.x, t1.z}, ss[4] = {t0.y, t0.w, t1.y, t1.w};
  Quad y1, y2;
  y1.err = y2.err = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a product and an fma: within 2^-24 of either's magnitude, with room
    constexpr float kE = 1.f / (1 << 22);
    y1.x[i] = rotated ? in1[i] * cc[i] - in2[i] * ss[i] : in1[i];
    y2.x[i] = rotated ? in2[i] * cc[i] + in1[i] * ss[i] : in2[i];
    if (rotated) {
      y1.err = fmaxf(y1.err, fabsf(in1[i] * cc[i]) * kE + fabsf(in2[i] * ss[i]) * kE);
      y2.err = fmaxf(y2.err, fabsf(in2[i] * cc[i]) * kE + fabsf(in1[i] * ss[i]) * kE);
    }
  }
  if (is_q) {
    float* q = a.q_out + ((size_t)row * a.nq + hh) * D + i4;
    *reinterpret_cast<float4*>(q) = make_float4(y1.x[0], y1.x[1], y1.x[2], y1.x[3]);
    *reinterpret_cast<float4*>(q + H2) = make_float4(y2.x[0], y2.x[1], y2.x[2], y2.x[3]);
  }
  const bool writes = live && !is_q;
  if (!__any_sync(0xffffffffu, writes)) return;

  const float g = rotated ? a.k_scale : a.v_scale, inv6g = rotated ? a.inv6_k : a.inv6_v;
  const Source q1 = {src, src + H2, cs, rotated ? -1.f : 0.f}, q2 = {src + H2, src, cs, rotated ? 1.f : 0.f};
  bool sure1 = true, sure2 = true;
  int s1 = scale_code(y1, inv6g, sure1), s2 = scale_code(y2, inv6g, sure2);
  if (__any_sync(0xffffffffu, writes && !(sure1 && sure2))) {
    s1 = exact_scale(q1, g, s1, sure1);
    s2 = exact_scale(q2, g, s2, sure2);
  }
  uint32_t u1, u2, c1 = value_codes(y1, g, s1, u1), c2 = value_codes(y2, g, s2, u2);
  if (!writes) return;
  if (u1) c1 = exact_codes(q1, g, s1, c1, u1);
  if (u2) c2 = exact_codes(q2, g, s2, c2, u2);
  if (blk < 0) {
    if (i4 == 0 && hh == a.nq) set_err(a.err, pos_ok ? MBT_DEV_BLOCK_RANGE : MBT_DEV_POS_RANGE);
    return;
  }
  const int kvh = rotated ? hh - a.nq : hh - a.nq - a.nkv, slot = pos % kBlockTokens;
  unsigned char* unit = reinterpret_cast<unsigned char*>(rotated ? a.kpool : a.vpool) +
                        ((size_t)blk * a.nkv + kvh) * fp4_unit_bytes(D);
  unsigned char* cod = unit + slot * (D / 2) + i4 / 2;
  *reinterpret_cast<uint16_t*>(cod) = (uint16_t)c1;
  *reinterpret_cast<uint16_t*>(cod + H2 / 2) = (uint16_t)c2;
  if (i4 % kFp4Group == 0) {
    unsigned char* scl = unit + kBlockTokens * (D / 2) + slot * (D / kFp4Group) + i4 / kFp4Group;
    scl[0] = (unsigned char)s1;
    scl[H2 / kFp4Group] = (unsigned char)s2;
  }
}

// Cached tokens as fp32 values: one row per blockIdx.x, four neighbouring
// channels of a head's K and V per thread (the position, the table's entry and
// the cached bytes are three loads in a row; both share the first two). Lanes
// store neighbouring 16 bytes: with eight channels a thread each store would
// fill half of every sector (10.8 us against 9.7, 4.0 TB/s, for 4084 rows of 8
// heads of 128).
template <int D>
__global__ void __launch_bounds__(kWriteThreads) kv_read_fp4_kernel(const KvReadFp4Args a) {
  constexpr int T = D / 4;
  const int row = blockIdx.x, h = blockIdx.y * (kWriteThreads / T) + threadIdx.x / T, i4 = 4 * (threadIdx.x % T);
  if (h >= a.nkv) return;
  const int pos = a.positions[row], seq = a.row_seq ? a.row_seq[row] : row;
  const bool pos_ok = pos >= 0 && pos / kBlockTokens < a.bt_stride && seq >= 0 && seq < a.nseq;
  int blk = pos_ok ? a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens] : -1;
  if (blk < 0 || blk > a.num_blocks) {
    if (i4 == 0 && h == 0) set_err(a.err, pos_ok ? MBT_DEV_BLOCK_RANGE : MBT_DEV_POS_RANGE);
    blk = -1;
  }
  const int slot = pos % kBlockTokens;
  const size_t unit = ((size_t)max(blk, 0) * a.nkv + h) * fp4_unit_bytes(D), out = ((size_t)row * a.nkv + h) * D + i4;
  uint32_t w[2] = {0, 0}, sb[2] = {0, 0};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const unsigned char* u = reinterpret_cast<const unsigned char*>(t ? a.vpool : a.kpool) + unit;
    if (blk >= 0) {
      w[t] = *reinterpret_cast<const uint16_t*>(u + slot * (D / 2) + i4 / 2);
      sb[t] = u[kBlockTokens * (D / 2) + slot * (D / kFp4Group) + i4 / kFp4Group];
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float s = e4m3_to_f32(sb[t]), g = t ? a.v_scale : a.k_scale;
    uint32_t p[2];
    e2m1x4_to_h2(w[t], p);
    const float2 f0 = h2_to_float2(p[0]), f1 = h2_to_float2(p[1]);   // code * scale is exact in fp32
    *reinterpret_cast<float4*>((t ? a.v_out : a.k_out) + out) =
        make_float4(f0.x * s * g, f0.y * s * g, f1.x * s * g, f1.y * s * g);
  }
}

}  // namespace

cudaError_t launch_rope_kv_write_fp4(const RopeKvFp4Args& a, cudaStream_t s) {
  const long long chunks = ((a.nq + 2LL * a.nkv) * (a.d / 8) + kWriteThreads - 1) / kWriteThreads;
  if (chunks > 65535) return cudaErrorInvalidValue;
  if (a.d == 64) rope_kv_write_fp4_kernel<64><<<dim3(a.n, (unsigned)chunks), kWriteThreads, 0, s>>>(a);
  else rope_kv_write_fp4_kernel<128><<<dim3(a.n, (unsigned)chunks), kWriteThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_fp4(const KvReadFp4Args& a, cudaStream_t s) {
  const long long chunks = ((long long)a.nkv * (a.d / 4) + kWriteThreads - 1) / kWriteThreads;
  if (chunks > 65535) return cudaErrorInvalidValue;
  if (a.d == 64) kv_read_fp4_kernel<64><<<dim3(a.n, (unsigned)chunks), kWriteThreads, 0, s>>>(a);
  else kv_read_fp4_kernel<128><<<dim3(a.n, (unsigned)chunks), kWriteThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mbt
