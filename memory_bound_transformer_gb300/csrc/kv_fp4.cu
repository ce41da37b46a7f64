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
// is done for both ends of the interval that the fp32 error leaves; where a
// warp meets two different results it repeats its values in 64 bits and
// decides by exact comparisons with the borders (about one warp in 500 for
// N(0, 1) rows).
//
// Bound by memory: one read of the projection's rows (4 bytes a value), one
// write of the rotated queries and of 9/16 byte a cached value.
#include "fp4.cuh"
#include "internal.h"

namespace mbt {

namespace {

// e4m3 value of a non-negative code as a double.
__device__ __forceinline__ double e4m3_f64(int c) { return (double)e4m3_to_f32((uint32_t)c); }

// The e4m3 code nearest to m / (6 g) (ties to the even code), m >= 0 exact.
// 6 g times the midpoint of two neighbouring e4m3 values is exact in a double
// (5 + 2 + 24 bits), so the decision is exact.
__device__ __noinline__ int scale_code_f64(double m, double g) {
  const double g6 = 6.0 * g;
  int c = f32_to_e4m3((float)(m / g6));
  if (c > 0) {
    const double mid = 0.5 * (e4m3_f64(c - 1) + e4m3_f64(c)) * g6;
    if (m < mid || (m == mid && (c & 1))) return c - 1;
  }
  if (c < 0x7e) {
    const double mid = 0.5 * (e4m3_f64(c) + e4m3_f64(c + 1)) * g6;
    if (m > mid || (m == mid && (c & 1))) return c + 1;
  }
  return c;
}

// The e2m1 code nearest to x / u (u = s g > 0), ties to the even code.
__device__ __noinline__ uint32_t value_code_f64(double x, double u) {
  const double a = fabs(x);
  uint32_t c = 0;
  c += a > 0.25 * u;
  c += a >= 0.75 * u;
  c += a > 1.25 * u;
  c += a >= 1.75 * u;
  c += a > 2.5 * u;
  c += a >= 3.5 * u;
  c += a > 5.0 * u;
  return c | (x < 0.0 ? 8u : 0u);
}

struct Quad { float x[4]; float err; };   // four neighbouring channels and a bound on their fp32 error

// Codes (4 bits each, first channel lowest) and scale code of one 16-channel
// block held by four neighbouring lanes, four channels each; `sure` is cleared
// where the fp32 error could change a rounding.
__device__ __forceinline__ void quantise(const Quad& q, float g, float inv6g, uint32_t& codes, int& sc, bool& sure) {
  float m = 0.f, e = q.err;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = fmaxf(m, fabsf(q.x[i]));
    nan |= q.x[i] != q.x[i];
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
    nan |= __shfl_xor_sync(0xffffffffu, (int)nan, o) != 0;
  }
  if (nan) { sc = 0x7f; codes = 0; return; }            // a block with a NaN reads as NaN
  constexpr float kRel = 1.f / (1 << 21);               // the roundings below, with room
  if (!(m <= 3.0e38f)) {                                // an infinity saturates the block's scale
    sc = 0x7e;
    e = 0.f;
  } else {
    sc = f32_to_e4m3((m + e) * inv6g * (1.f + kRel));
    if (f32_to_e4m3(fmaxf(m - e, 0.f) * inv6g * (1.f - kRel)) != (uint8_t)sc) sure = false;
  }
  if (sc == 0) { codes = 0; return; }                   // too small for the scale's grid
  const float inv = __fdiv_rn(1.f, e4m3_to_f32((uint32_t)sc) * g);
  float lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = q.x[i] * inv, d = fabsf(r) * kRel + (e > 0.f ? q.err : 0.f) * inv;
    const bool fin = fabsf(r) <= 3.0e38f;
    lo[i] = fin ? r - d : r;
    hi[i] = fin ? r + d : r;
  }
  codes = f32x2_to_e2m1x2(hi[0], hi[1]) | (f32x2_to_e2m1x2(hi[2], hi[3]) << 8);
  if ((f32x2_to_e2m1x2(lo[0], lo[1]) | (f32x2_to_e2m1x2(lo[2], lo[3]) << 8)) != codes) sure = false;
}

// The same in 64 bits.
__device__ __noinline__ void quantise_f64(const double (&x)[4], double g, uint32_t& codes, int& sc) {
  double m = 0.0;
  bool fin = true;
  for (int i = 0; i < 4; ++i) {
    m = fmax(m, fabs(x[i]));
    fin &= fabs(x[i]) <= 1.0e300;
  }
  for (int o = 1; o < 4; o <<= 1) {
    m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    fin &= __shfl_xor_sync(0xffffffffu, (int)fin, o) != 0;
  }
  if (!fin) return;                                     // decided in 32 bits
  sc = scale_code_f64(m, g);
  codes = 0;
  if (sc == 0) return;
  const double u = e4m3_f64(sc) * g;
  for (int i = 0; i < 4; ++i) codes |= value_code_f64(x[i], u) << (4 * i);
}

constexpr int kWriteThreads = 256;

// One thread holds channels 4i..4i+3 and the same of the other half of one
// head's row; the four lanes of a 16-channel block are neighbours.
template <int D>
__global__ void __launch_bounds__(kWriteThreads) rope_kv_write_fp4_kernel(const RopeKvFp4Args a) {
  constexpr int T = D / 8, H2 = D / 2;                  // threads per head row, channels per half
  const int nh = a.nq + 2 * a.nkv;
  const long long total = (long long)a.n * nh * T;
  const long long id = (long long)blockIdx.x * kWriteThreads + threadIdx.x;
  const bool live = id < total;                         // whole rows: T divides the warp size
  const long long item = (live ? id : 0) / T;
  const int i4 = 4 * (int)(id % T);
  const int row = (int)(item / nh), hh = (int)(item % nh);
  const bool rotated = hh < a.nq + a.nkv, is_q = hh < a.nq;

  int pos = a.positions[row];
  const bool pos_ok = pos >= 0 && pos < a.max_pos;
  if (!pos_ok) pos = 0;
  const float* src = a.qkv + (size_t)row * a.ld_qkv + (size_t)hh * D + i4;
  const float4 x1 = *reinterpret_cast<const float4*>(src), x2 = *reinterpret_cast<const float4*>(src + H2);
  const float in1[4] = {x1.x, x1.y, x1.z, x1.w}, in2[4] = {x2.x, x2.y, x2.z, x2.w};
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  Quad y1, y2;
  y1.err = y2.err = 0.f;
  if (rotated) {
    const float4* cs = reinterpret_cast<const float4*>(a.rope + (size_t)pos * D) + i4 / 2;
    const float4 t0 = cs[0], t1 = cs[1];
    c[0] = t0.x; s[0] = t0.y; c[1] = t0.z; s[1] = t0.w;
    c[2] = t1.x; s[2] = t1.y; c[3] = t1.z; s[3] = t1.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y1.x[i] = in1[i] * c[i] - in2[i] * s[i];
      y2.x[i] = in2[i] * c[i] + in1[i] * s[i];
      // two products and a sum: within 3 * 2^-24 of the products' magnitudes
      constexpr float kE = 1.f / (1 << 22);
      y1.err = fmaxf(y1.err, (fabsf(in1[i] * c[i]) + fabsf(in2[i] * s[i])) * kE);
      y2.err = fmaxf(y2.err, (fabsf(in2[i] * c[i]) + fabsf(in1[i] * s[i])) * kE);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) { y1.x[i] = in1[i]; y2.x[i] = in2[i]; }
  }
  if (live && is_q) {
    float* q = a.q_out + ((size_t)row * a.nq + hh) * D + i4;
    *reinterpret_cast<float4*>(q) = make_float4(y1.x[0], y1.x[1], y1.x[2], y1.x[3]);
    *reinterpret_cast<float4*>(q + H2) = make_float4(y2.x[0], y2.x[1], y2.x[2], y2.x[3]);
  }
  if (__all_sync(0xffffffffu, is_q)) return;

  const float g = rotated ? a.k_scale : a.v_scale, inv6g = rotated ? a.inv6_k : a.inv6_v;
  uint32_t c1 = 0, c2 = 0;
  int s1 = 0, s2 = 0;
  bool sure = true;
  quantise(y1, g, inv6g, c1, s1, sure);
  quantise(y2, g, inv6g, c2, s2, sure);
  if (__any_sync(0xffffffffu, !sure && live && !is_q)) {
    double d1[4], d2[4];
    for (int i = 0; i < 4; ++i) {
      d1[i] = rotated ? __dsub_rn((double)in1[i] * c[i], (double)in2[i] * s[i]) : (double)in1[i];
      d2[i] = rotated ? __dadd_rn((double)in2[i] * c[i], (double)in1[i] * s[i]) : (double)in2[i];
    }
    quantise_f64(d1, g, c1, s1);
    quantise_f64(d2, g, c2, s2);
  }
  if (!live || is_q) return;

  const int seq = a.row_seq ? a.row_seq[row] : row;
  const int jb = pos / kBlockTokens;
  int blk = -1;
  if (pos_ok && seq >= 0 && seq < a.nseq && jb < a.bt_stride) blk = a.bt[(size_t)seq * a.bt_stride + jb];
  if (blk < 0 || blk > a.num_blocks) {
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

// Cached tokens as fp32 values: eight neighbouring channels per thread.
template <int D>
__global__ void __launch_bounds__(kWriteThreads) kv_read_fp4_kernel(const KvReadFp4Args a) {
  constexpr int T = D / 8;
  const long long id = (long long)blockIdx.x * kWriteThreads + threadIdx.x;
  if (id >= (long long)a.n * 2 * a.nkv * T) return;
  const int i8 = 8 * (int)(id % T);
  const long long item = id / T;
  const int row = (int)(item / (2 * a.nkv)), hv = (int)(item % (2 * a.nkv));
  const bool is_v = hv >= a.nkv;
  const int h = is_v ? hv - a.nkv : hv;
  const int pos = a.positions[row], seq = a.row_seq ? a.row_seq[row] : row;
  const bool pos_ok = pos >= 0 && pos / kBlockTokens < a.bt_stride && seq >= 0 && seq < a.nseq;
  const int blk = pos_ok ? a.bt[(size_t)seq * a.bt_stride + pos / kBlockTokens] : -1;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (blk < 0 || blk > a.num_blocks) {
    if (i8 == 0 && hv == 0) set_err(a.err, pos_ok ? MBT_DEV_BLOCK_RANGE : MBT_DEV_POS_RANGE);
  } else {
    const unsigned char* unit = reinterpret_cast<const unsigned char*>(is_v ? a.vpool : a.kpool) +
                                ((size_t)blk * a.nkv + h) * fp4_unit_bytes(D);
    const int slot = pos % kBlockTokens;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(unit + slot * (D / 2) + i8 / 2);
    const float s = e4m3_to_f32(unit[kBlockTokens * (D / 2) + slot * (D / kFp4Group) + i8 / kFp4Group]);
    const float g = is_v ? a.v_scale : a.k_scale;
    uint32_t p[4];
    e2m1x8_to_h2(w, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {                       // code * scale is exact in fp32
      const float2 f = h2_to_float2(p[j]);
      v[2 * j] = f.x * s * g;
      v[2 * j + 1] = f.y * s * g;
    }
  }
  float* o = (is_v ? a.v_out : a.k_out) + ((size_t)row * a.nkv + h) * D + i8;
  *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace

cudaError_t launch_rope_kv_write_fp4(const RopeKvFp4Args& a, cudaStream_t s) {
  const long long total = (long long)a.n * (a.nq + 2 * a.nkv) * (a.d / 8);
  const long long grid = (total + kWriteThreads - 1) / kWriteThreads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.d == 64) rope_kv_write_fp4_kernel<64><<<(unsigned)grid, kWriteThreads, 0, s>>>(a);
  else rope_kv_write_fp4_kernel<128><<<(unsigned)grid, kWriteThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_fp4(const KvReadFp4Args& a, cudaStream_t s) {
  const long long total = (long long)a.n * 2 * a.nkv * (a.d / 8);
  const long long grid = (total + kWriteThreads - 1) / kWriteThreads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.d == 64) kv_read_fp4_kernel<64><<<(unsigned)grid, kWriteThreads, 0, s>>>(a);
  else kv_read_fp4_kernel<128><<<(unsigned)grid, kWriteThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mbt
