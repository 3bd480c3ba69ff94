// Rows in 8-bit floating point: quantisation, the SwiGLU that leaves its
// output and its 8-bit checkpoint, and the backward that starts from it.
//
// A row is cut into blocks of 128 columns (the last may be shorter).  A block
// has the scale 2^e, e the least integer >= -127 with max |x| <= 448 * 2^e
// (e = 0 for a block of zeros), held as the E8M0 byte e + 127; its values are
// the OCP E4M3 codes of x / 2^e, rounded to nearest even.  A power of two
// loses nothing against max|x| / 448: E4M3 is a floating format, so the
// division by 2^e is exact and only values below 2^-6 * 2^e (2^-14.8 of the
// block's maximum at most) meet the subnormal grid.  And it is the scale the
// matrix cores apply by themselves.  An infinite or NaN x becomes the NaN
// code; the other values of its block are scaled as if it were not there.
// Where the rows are computed (SwiGLU and its backward) the codes and scales are
// those of the exact values of the formula, not of an fp32 approximation.
#include "qgg_device.hpp"
#include "qgg_internal.hpp"

namespace qgg {

namespace {

// E8M0 byte of a block from the bits of its largest finite magnitude m 2^x (1
// <= m < 2): 448 = 1.75 * 2^8, so e = x - 8 for m <= 1.75, else x - 7 (the
// addition carries into the exponent exactly then); subnormals end at 0.
__device__ __forceinline__ int block_scale(uint32_t amax) {
  return amax ? max((int)((amax + 0x1FFFFFu) >> 23) - 8, 0) : 127;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// The scale as the conversion instructions take it: they use its exponent
// field, so code 0 stands for 2^-127 without being a subnormal.
__device__ __forceinline__ float scale_operand(int code) {
  return __uint_as_float((uint32_t)code << 23);
}

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// maximum over the 16 lanes of a DPP row
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}

typedef short s16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint2 convert8(const float v[8], int code) {
  const float s = scale_operand(code);
  s16x2_t lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[1], s, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2], v[3], s, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4], v[5], s, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6], v[7], s, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

// Codes of eight values of which some may not be finite: those become NaN.
__device__ __forceinline__ uint2 convert8_any(const float v[8], int code) {
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = mag_bits(v[i]) < kInfBits ? v[i] : 0.f;
  uint2 q = convert8(z, code);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (mag_bits(v[i]) >= kInfBits) (i < 4 ? q.x : q.y) |= 0x7Fu << (8 * (i & 3));
  return q;
}

// Block maximum of eight values a lane; the largest finite magnitude where the
// plain maximum is infinite or NaN (rare, so checked once a wavefront).
__device__ __forceinline__ uint32_t block_max(const float v[8], bool* odd) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
  m = row16_max(m);
  *odd = __any(m >= kInfBits);
  if (*odd) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]) < kInfBits ? mag_bits(v[i]) : 0u);
    m = row16_max(m);
  }
  return m;
}

// Eight values (a block is 16 lanes of eight) -> eight codes and the block's
// scale byte.  Every lane of the row must call it.
__device__ __forceinline__ uint2 quantize8(const float v[8], int* code) {
  bool odd;
  *code = block_scale(block_max(v, &odd));
  return odd ? convert8_any(v, *code) : convert8(v, *code);
}

__device__ __forceinline__ void widen8(u32x4_t w, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The same from BF16 pairs, without widening them: the maximum over packed
// 16-bit magnitudes, the conversion from BF16.
__device__ __forceinline__ uint2 quantize8_bf16(u32x4_t w, int* code) {
  u16x2_t m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu));
  const uint32_t top = row16_max((uint32_t)max(m[0], m[1]) << 16);
  if (__any(top >= kInfBits)) {
    float v[8];
    widen8(w, v);
    return quantize8(v, code);
  }
  *code = block_scale(top);
  const float s = scale_operand(*code);
  s16x2_t lo = {0, 0}, hi = {0, 0};
  const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_t, w0), s, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(bf16x2_t, w1), s, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_t, w2), s, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(bf16x2_t, w3), s, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

__device__ __forceinline__ float round_to_odd(double x) {
  float f = (float)x;
  if ((double)f != x && mag_bits(f) < kInfBits) {
    uint32_t b = __float_as_uint(f);
    if (fabs((double)f) > fabs(x)) --b;          // towards zero
    f = __uint_as_float(b | 1u);
  }
  return f;
}

// v[i] without putting the array into memory
typedef float f32x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ float pick(const float v[8], int i) {
  const f32x8_t x = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  float e = x[i];
  // pins what follows from it to its place: the double arithmetic of two rare
  // paths would otherwise be shared, and computed before either is entered
  asm volatile("" : "+v"(e));
  return e;
}

// Codes of eight values that are known to lie between lo[i] and hi[i], as those
// of the exact values.  Where the two ends have another code, exact(i) gives
// the value over again (in double, rounded to odd: the last bit of a rounded
// one is set, so that rounding it again decides as for the exact value); with
// fp32 arithmetic about one value in 50 000 needs it.  So a code does not hang
// on the order of the operations before it, and two programs, or a 64-bit
// reference, have the same.  kMargin bounds the relative width of an interval
// around a block's maximum: within it of a border of scales (or with values
// that are not finite) the whole block is taken exactly.  So is a block of
// values below kTiny, where a product on the way to one may have left the
// normal numbers and lost more than its interval allows; above kTiny that would
// take factors past 2^50 after such a product.
constexpr float kMargin = 0x1p-15f;
constexpr uint32_t kTiny = 67u << 23;            // 2^-60

// HI: |hi| >= |lo|.  `all`: a lane has a value that lo and hi do not hold.
template <bool HI, typename Exact>
__device__ __forceinline__ uint2 quantize8_exact(const float lo[8], const float hi[8], bool all,
                                                 Exact exact, int* code) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = max(top, mag_bits(hi[i]));
    if (!HI) top = max(top, mag_bits(lo[i]));
  }
  top = row16_max(top);
  *code = block_scale(top);
  const float low = __uint_as_float(top) * (1.0f - kMargin);
  if (__any(all || (top != 0 && top < kTiny) || top >= kInfBits ||
            block_scale(mag_bits(low)) != *code)) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = exact(i);
    return quantize8(v, code);
  }
  uint2 q = convert8(hi, *code);
  const uint2 ql = convert8(lo, *code);
  uint32_t dx = q.x ^ ql.x, dy = q.y ^ ql.y;
  while (__any((dx | dy) != 0)) {
    if ((dx | dy) != 0) {
      const int i = dx ? __builtin_ctz(dx) >> 3 : 4 + (__builtin_ctz(dy) >> 3);
      const uint32_t mask = 0xFFu << (8 * (i & 3));
      s16x2_t z = {0, 0};
      z = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(z, exact(i), 0.f, scale_operand(*code), false);
      const uint32_t byte = (__builtin_bit_cast(uint32_t, z) & 0xFFu) << (8 * (i & 3));
      if (i < 4) {
        q.x = (q.x & ~mask) | byte;
        dx &= ~mask;
      } else {
        q.y = (q.y & ~mask) | byte;
        dy &= ~mask;
      }
    }
  }
  return q;
}

__device__ __forceinline__ void decode8(uint2 w, int code, float v[8]) {
  const float s = scale_operand(code);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h ? w.y : w.x, s, false);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(h ? w.y : w.x, s, true);
    v[4 * h] = a[0];
    v[4 * h + 1] = a[1];
    v[4 * h + 2] = b[0];
    v[4 * h + 3] = b[1];
  }
}

__device__ __forceinline__ u32x4_t pack8(const float v[8]) {
  return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
}

// 16 lanes a block, eight columns a lane; lanes past the end of a short last
// block carry zeros.
__global__ __launch_bounds__(256) void k_fp8_quantize(const uint16_t* __restrict__ x, int64_t n,
                                                      int cols, int nb,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales) {
  const int l = threadIdx.x & 15;
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; b < n; b += (int64_t)gridDim.x * 16) {
    const int64_t r = b / nb;
    const int c = (int)(b - r * nb) * 128 + 8 * l;
    u32x4_t w = {0u, 0u, 0u, 0u};
    if (c < cols) w = *reinterpret_cast<const u32x4_t*>(x + r * cols + c);
    int code;
    const uint2 q = quantize8_bf16(w, &code);
    if (c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = q;
    if (l == 0) scales[b] = (uint8_t)code;
  }
}

__global__ __launch_bounds__(256) void k_fp8_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        int64_t n, int cols, int nb,
                                                        uint16_t* __restrict__ x) {
  const int per = cols / 8;                      // eight columns a thread
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < n; q += (int64_t)gridDim.x * 256) {
    const int64_t r = q / per;
    const int c = (int)(q - r * per) * 8;
    const int code = scales[r * nb + (c >> 7)];
    float v[8];
    decode8(*reinterpret_cast<const uint2*>(codes + r * cols + c), code, v);
    *reinterpret_cast<u32x4_t*>(x + r * cols + c) = pack8(v);
  }
}

// f = 1 / (1 + exp(-z)) and 1 - f, both to a few fp32 steps at every z: with
// t = exp(-|z|) they are 1 / (1 + t) and t / (1 + t).  t is the square of
// exp(-|z| / 2), whose exponential stays a normal number where t itself has
// become subnormal (the hardware's exponential flushes those).  In half steps
// (2^-24): the exponential's argument |z| / 2, itself 2, squared (|z| + 4) and
// 1; the sum 1, the reciprocal 2, the product 1: at most |z| + 9.
__device__ __forceinline__ void sigmoid2(float z, float* f, float* one_minus_f) {
  const float h = __expf(-0.5f * fabsf(z));
  const float t = h * h;
  const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
  *f = z >= 0.f ? big : small;
  *one_minus_f = z >= 0.f ? small : big;
}
constexpr float kHalfStep = 0x1p-24f;

// The same in fewer operations for z >= kFar (half steps: f |z| + 6, 1 - f |z|
// + 9), where exp(-z) and f are normal numbers.
constexpr float kFar = -87.0f;
__device__ __forceinline__ void sigmoid2_near(float z, float* f, float* one_minus_f) {
  const float e = __expf(-z);
  *f = __builtin_amdgcn_rcpf(1.0f + e);
  *one_minus_f = e * *f;
}

__device__ __forceinline__ bool any_far(const float z[8]) {
  bool far = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) far |= z[i] < kFar;
  return far;
}

__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

// One block of 128 columns of one row: gate and up in, a out (BF16 and / or
// E4M3), both halves of h out in E4M3.  65536 rows of 2 x 2048 with a8 and h8
// take 0.20 ms, 4.7 TB/s of the 5.0 that a copy of 2 GiB reaches; codes that
// need not be those of the exact values took 0.18.
__global__ __launch_bounds__(256) void k_swiglu_fp8(const uint16_t* __restrict__ h,
                                                    const int32_t* __restrict__ n_rows, int64_t n,
                                                    int inter, uint16_t* __restrict__ a,
                                                    uint8_t* __restrict__ a8,
                                                    uint8_t* __restrict__ a_scales,
                                                    uint8_t* __restrict__ h8,
                                                    uint8_t* __restrict__ h_scales) {
  const int l = threadIdx.x & 15;
  const int nb = inter >> 7;
  const int64_t live = n_rows ? min(n, (int64_t)*n_rows * nb) : n;
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; b < live;
       b += (int64_t)gridDim.x * 16) {
    const int64_t r = b / nb;
    const int blk = (int)(b - r * nb);
    const int c = blk * 128 + 8 * l;
    const int64_t at = r * 2 * inter + c;
    const u32x4_t gw = *reinterpret_cast<const u32x4_t*>(h + at);
    const u32x4_t uw = *reinterpret_cast<const u32x4_t*>(h + at + inter);
    int code;
    if (h8) {
      *reinterpret_cast<uint2*>(h8 + at) = quantize8_bf16(gw, &code);
      if (l == 0) h_scales[r * 2 * nb + blk] = (uint8_t)code;
      *reinterpret_cast<uint2*>(h8 + at + inter) = quantize8_bf16(uw, &code);
      if (l == 0) h_scales[r * 2 * nb + nb + blk] = (uint8_t)code;
    }
    if (!a && !a8) continue;
    float g[8], u[8];
    widen8(gw, g);
    widen8(uw, u);
    if (a) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f, f1;
        sigmoid2(g[i], &f, &f1);
        v[i] = g[i] * f * u[i];
      }
      *reinterpret_cast<u32x4_t*>(a + r * inter + c) = pack8(v);
    }
    if (a8) {
      float lo[8], hi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f, f1;
        sigmoid2_near(g[i], &f, &f1);
        const float v = g[i] * f * u[i];
        // half steps: f and two products
        const float w = __builtin_fmaf(fabsf(g[i]), kHalfStep, 9 * kHalfStep);
        lo[i] = __builtin_fmaf(-w, v, v);
        hi[i] = __builtin_fmaf(w, v, v);
      }
      auto exact = [&](int i) {
        const double z = pick(g, i);
        return round_to_odd(z * sigmoid64(z) * (double)pick(u, i));
      };
      *reinterpret_cast<uint2*>(a8 + r * inter + c) =
          quantize8_exact<true>(lo, hi, any_far(g), exact, &code);
      if (l == 0) a_scales[r * nb + blk] = (uint8_t)code;
    }
  }
}

// One workgroup per routed pair (32 a CU, each taking pairs in turn: 8 % less
// time than one launched for each).  gate and up come back from the checkpoint;
// d = g_pair * da; dh = [d up silu'(gate) | d silu(gate)] and
// dgates[pair] = sum_c da[c] silu(gate[c]) up[c].  silu'(z) = f (1 + z (1 - f)),
// f = 1 / (1 + exp(-z)).  A pair that the permutation dropped has no row; its
// dgates is 0.
// W: what is wanted (1: dh, 2: dh8, 4: dgates).  65536 pairs of 2 x 2048, dh8 and
// dgates: 0.21 ms for 0.81 GB, bound by vector instructions (the bounds of each
// value, their conversion at both ends) at 4 TB/s.
template <int W>
__global__ __launch_bounds__(256) void k_swiglu_fp8_bwd(
    const uint16_t* __restrict__ da, const uint8_t* __restrict__ h8,
    const uint8_t* __restrict__ h_scales, const float* __restrict__ gates,
    const int32_t* __restrict__ inv_perm, int64_t P, int inter, uint16_t* __restrict__ dh,
    uint8_t* __restrict__ dh8, uint8_t* __restrict__ dh_scales, float* __restrict__ dgates) {
  __shared__ float part[2][4];
  const int nb = inter >> 7;
  const int l = threadIdx.x & 15;
  int flip = 0;
  for (int64_t p = blockIdx.x; p < P; p += gridDim.x) {
    const int64_t r = inv_perm[p];
    if (r < 0) {
      if ((W & 4) && threadIdx.x == 0) dgates[p] = 0.f;
      continue;
    }
    const float gp = gates[p];
    float sum = 0.f;
    for (int blk = threadIdx.x >> 4; blk < nb; blk += 16) {
      const int c = blk * 128 + 8 * l;
      const int64_t at = r * 2 * inter + c;
      float g[8], u[8], d[8];
      const uint2 gq = *reinterpret_cast<const uint2*>(h8 + at);
      const uint2 uq = *reinterpret_cast<const uint2*>(h8 + at + inter);
      const int gs = h_scales[r * 2 * nb + blk], us = h_scales[r * 2 * nb + nb + blk];
      widen8(*reinterpret_cast<const u32x4_t*>(da + r * inter + c), d);
      decode8(gq, gs, g);
      decode8(uq, us, u);
      if constexpr (W != 2) {
        float dg[8], du[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, f1;
          if constexpr (W & 1) sigmoid2(g[i], &f, &f1);
          else sigmoid2_near(g[i], &f, &f1);
          const float s = g[i] * f;
          sum = __builtin_fmaf(d[i], s * u[i], sum);
          const float dd = gp * d[i];
          dg[i] = dd * u[i] * f * (1.0f + g[i] * f1);
          du[i] = dd * s;
        }
        if constexpr (W & 1) {
          *reinterpret_cast<u32x4_t*>(dh + at) = pack8(dg);
          *reinterpret_cast<u32x4_t*>(dh + at + inter) = pack8(du);
        }
      }
      if constexpr (W & 2) {
        float lo[8], hi[8];
        const bool far = any_far(g);
        int code;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, f1;
          sigmoid2_near(g[i], &f, &f1);
          // half steps: f |z| + 6; m = 1 + z (1 - f) with |z| + 10 of |z (1 -
          // f)| <= |m| + 1 and its own rounding; four products: of |m| + 1
          const float m = __builtin_fmaf(g[i], f1, 1.0f);
          const float w = __builtin_fmaf(fabsf(g[i]), 2 * kHalfStep, 22 * kHalfStep);
          const float slope = gp * d[i] * u[i] * f;
          const float em = __builtin_fmaf(w, fabsf(m), w);
          lo[i] = slope * (m - em);
          hi[i] = slope * (m + em);
        }
        auto exact_g = [&](int i) {
          const double z = pick(g, i);
          return round_to_odd((double)gp * pick(d, i) * pick(u, i) * sigmoid64(z) *
                              (1.0 + z * sigmoid64(-z)));
        };
        *reinterpret_cast<uint2*>(dh8 + at) =
            quantize8_exact<false>(lo, hi, far, exact_g, &code);
        if (l == 0) dh_scales[r * 2 * nb + blk] = (uint8_t)code;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float f, f1;
          sigmoid2_near(g[i], &f, &f1);
          const float w = __builtin_fmaf(fabsf(g[i]), 2 * kHalfStep, 22 * kHalfStep);
          const float v = gp * d[i] * (g[i] * f);
          lo[i] = __builtin_fmaf(-w, v, v);
          hi[i] = __builtin_fmaf(w, v, v);
        }
        auto exact_u = [&](int i) {
          const double z = pick(g, i);
          return round_to_odd((double)gp * pick(d, i) * z * sigmoid64(z));
        };
        *reinterpret_cast<uint2*>(dh8 + at + inter) =
            quantize8_exact<true>(lo, hi, far, exact_u, &code);
        if (l == 0) dh_scales[r * 2 * nb + nb + blk] = (uint8_t)code;
      }
    }
    if constexpr (W & 4) {
      sum = wave_sum_63(sum);
      // two sets of partial sums: the next pair's writes meet the last reads of
      // the one before only after another barrier
      if ((threadIdx.x & 63) == 63) part[flip][threadIdx.x >> 6] = sum;
      __syncthreads();
      if (threadIdx.x == 0)
        dgates[p] = (part[flip][0] + part[flip][1]) + (part[flip][2] + part[flip][3]);
      flip ^= 1;
    }
  }
}

// Workgroups of 256 for this many threads; the kernels stride over the rest
// (a launch holds fewer than 2^32 threads).
constexpr int64_t kMostGroups = 1 << 22;
constexpr int kRowGroups = 32;
unsigned groups(int64_t threads) {
  return (unsigned)std::min<int64_t>((threads + 255) / 256, kMostGroups);
}

}  // namespace

hipError_t launch_fp8_quantize(const uint16_t* x, int64_t rows, int cols, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  TimedLaunch timed_(kLOther, s);
  if (rows == 0) return hipSuccess;
  const int nb = (cols + 127) / 128;
  hipLaunchKernelGGL(k_fp8_quantize, dim3(groups(rows * nb * 16)), dim3(256), 0, s, x, rows * nb,
                     cols, nb, codes, scales);
  return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                 int cols, uint16_t* x, hipStream_t s) {
  TimedLaunch timed_(kLOther, s);
  if (rows == 0) return hipSuccess;
  const int64_t n = rows * (cols / 8);
  hipLaunchKernelGGL(k_fp8_dequantize, dim3(groups(n)), dim3(256), 0, s, codes, scales, n, cols,
                     (cols + 127) / 128, x);
  return hipGetLastError();
}

hipError_t launch_swiglu_fp8(const uint16_t* h, const int32_t* n_rows, int64_t P, int inter,
                             uint16_t* a, uint8_t* a8, uint8_t* a_scales, uint8_t* h8,
                             uint8_t* h_scales, hipStream_t s) {
  TimedLaunch timed_(kLOther, s);
  if (P == 0) return hipSuccess;
  const int64_t n = P * (inter / 128);
  hipLaunchKernelGGL(k_swiglu_fp8, dim3(groups(n * 16)), dim3(256), 0, s, h, n_rows, n, inter, a,
                     a8, a_scales, h8, h_scales);
  return hipGetLastError();
}

hipError_t launch_swiglu_fp8_bwd(const uint16_t* da, const uint8_t* h8, const uint8_t* h_scales,
                                 const float* gates, const int32_t* inv_perm, int64_t P, int inter,
                                 uint16_t* dh, uint8_t* dh8, uint8_t* dh_scales, float* dgates,
                                 hipStream_t s) {
  TimedLaunch timed_(kLOther, s);
  if (P == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<int64_t>(P, (int64_t)num_cus() * kRowGroups));
  auto go = [&](auto w) {
    hipLaunchKernelGGL(k_swiglu_fp8_bwd<decltype(w)::value>, grid, dim3(256), 0, s, da, h8,
                       h_scales, gates, inv_perm, P, inter, dh, dh8, dh_scales, dgates);
  };
  using std::integral_constant;
  switch ((dh ? 1 : 0) | (dh8 ? 2 : 0) | (dgates ? 4 : 0)) {
    case 1: go(integral_constant<int, 1>{}); break;
    case 2: go(integral_constant<int, 2>{}); break;
    case 3: go(integral_constant<int, 3>{}); break;
    case 4: go(integral_constant<int, 4>{}); break;
    case 5: go(integral_constant<int, 5>{}); break;
    case 6: go(integral_constant<int, 6>{}); break;
    default: go(integral_constant<int, 7>{}); break;
  }
  return hipGetLastError();
}

}  // namespace qgg
