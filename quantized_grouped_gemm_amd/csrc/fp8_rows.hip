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
#include "qgg_device.hpp"
#include "qgg_internal.hpp"

namespace qgg {

namespace {

// E8M0 byte of a block from the bits of its largest finite magnitude.
// 448 = 1.75 * 2^8, so with amax = m 2^x (1 <= m < 2): e = x - 8 for
// m <= 1.75, else x - 7.
__device__ __forceinline__ int block_scale(uint32_t amax_bits) {
  if (amax_bits == 0) return 127;
  uint32_t b = amax_bits;
  int x = 0;
  if (b < 0x00800000u) {                         // subnormal: normalise
    const int sh = __clz(b) - 8;
    b <<= sh;
    x = -126 - sh;
  } else {
    x = (int)(b >> 23) - 127;
  }
  const int e = (b & 0x007FFFFFu) <= 0x00600000u ? x - 8 : x - 7;
  return max(e + 127, 0);
}

// 2^-e for the scale byte e + 127 (e <= 120): always a normal number
__device__ __forceinline__ float inv_scale(int code) {
  return __uint_as_float((uint32_t)(254 - code) << 23);
}

// magnitude bits for the block maximum; 0 for what is not finite
__device__ __forceinline__ uint32_t mag_bits(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// maximum over the 16 lanes of a DPP row
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}

// Eight values (a block is 16 lanes of eight) -> eight codes and the block's
// scale byte.  Every lane of the row must call it.
__device__ __forceinline__ uint2 quantize8(const float v[8], int* code) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_bits(v[i]));
  *code = block_scale(row16_max(m));
  const float inv = inv_scale(*code);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __builtin_isfinite(v[i]) ? v[i] * inv : __uint_as_float(0x7FC00000u);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

__device__ __forceinline__ void widen8(u32x4_t w, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void decode8(uint2 w, float scale, float v[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, false);
  const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.x, true);
  const f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, false);
  const f32x2_t d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w.y, true);
  v[0] = a[0] * scale;
  v[1] = a[1] * scale;
  v[2] = b[0] * scale;
  v[3] = b[1] * scale;
  v[4] = c[0] * scale;
  v[5] = c[1] * scale;
  v[6] = d[0] * scale;
  v[7] = d[1] * scale;
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
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < cols) widen8(*reinterpret_cast<const u32x4_t*>(x + r * cols + c), v);
    int code;
    const uint2 q = quantize8(v, &code);
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
    float v[8];
    decode8(*reinterpret_cast<const uint2*>(codes + r * cols + c),
            e8m0_to_f32(scales[r * nb + (c >> 7)]), v);
    *reinterpret_cast<u32x4_t*>(x + r * cols + c) = pack8(v);
  }
}

// f = 1 / (1 + exp(-z)) and 1 - f, both to a few fp32 steps at every z: with
// t = exp(-|z|) they are 1 / (1 + t) and t / (1 + t).  t is the square of
// exp(-|z| / 2), whose exponential stays a normal number where t itself has
// become subnormal (the hardware's exponential flushes those).
__device__ __forceinline__ void sigmoid2(float z, float* f, float* one_minus_f) {
  const float h = __expf(-0.5f * fabsf(z));
  const float t = h * h;
  const float big = __builtin_amdgcn_rcpf(1.0f + t), small = t * big;
  *f = z >= 0.f ? big : small;
  *one_minus_f = z >= 0.f ? small : big;
}

// One block of 128 columns of one row: gate and up in, a out (BF16 and / or
// E4M3), both halves of h out in E4M3.  The output is formed in fp32 and
// rounded once, to whichever type it is stored in.
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
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4; b < live; b += (int64_t)gridDim.x * 16) {
    const int64_t r = b / nb;
    const int blk = (int)(b - r * nb);
    const int c = blk * 128 + 8 * l;
    const int64_t at = r * 2 * inter + c;
    float g[8], u[8], v[8];
    widen8(*reinterpret_cast<const u32x4_t*>(h + at), g);
    widen8(*reinterpret_cast<const u32x4_t*>(h + at + inter), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, f1;
      sigmoid2(g[i], &f, &f1);
      v[i] = g[i] * f * u[i];
    }
    if (a) *reinterpret_cast<u32x4_t*>(a + r * inter + c) = pack8(v);
    int code;
    if (a8) {
      *reinterpret_cast<uint2*>(a8 + r * inter + c) = quantize8(v, &code);
      if (l == 0) a_scales[r * nb + blk] = (uint8_t)code;
    }
    if (h8) {
      *reinterpret_cast<uint2*>(h8 + at) = quantize8(g, &code);
      if (l == 0) h_scales[r * 2 * nb + blk] = (uint8_t)code;
      *reinterpret_cast<uint2*>(h8 + at + inter) = quantize8(u, &code);
      if (l == 0) h_scales[r * 2 * nb + nb + blk] = (uint8_t)code;
    }
  }
}

// One workgroup per routed pair.  gate and up come back from the checkpoint;
// d = g_pair * da; dh = [d up silu'(gate) | d silu(gate)] and
// dgates[pair] = sum_c da[c] silu(gate[c]) up[c].  silu'(z) = f (1 + z (1 - f)),
// f = 1 / (1 + exp(-z)).  A pair that the permutation dropped has no row; its
// dgates is 0.
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
      if (dgates && threadIdx.x == 0) dgates[p] = 0.f;
      continue;
    }
    const float gp = gates[p];
    float sum = 0.f;
    for (int blk = threadIdx.x >> 4; blk < nb; blk += 16) {
      const int c = blk * 128 + 8 * l;
      const int64_t at = r * 2 * inter + c;
      float g[8], u[8], d[8], dg[8], du[8];
      decode8(*reinterpret_cast<const uint2*>(h8 + at), e8m0_to_f32(h_scales[r * 2 * nb + blk]), g);
      decode8(*reinterpret_cast<const uint2*>(h8 + at + inter),
              e8m0_to_f32(h_scales[r * 2 * nb + nb + blk]), u);
      widen8(*reinterpret_cast<const u32x4_t*>(da + r * inter + c), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f, f1;
        sigmoid2(g[i], &f, &f1);
        const float s = g[i] * f;
        sum += d[i] * (s * u[i]);
        const float dd = gp * d[i];
        dg[i] = dd * u[i] * (f * (1.0f + g[i] * f1));
        du[i] = dd * s;
      }
      if (dh) {
        *reinterpret_cast<u32x4_t*>(dh + at) = pack8(dg);
        *reinterpret_cast<u32x4_t*>(dh + at + inter) = pack8(du);
      }
      if (dh8) {
        int code;
        *reinterpret_cast<uint2*>(dh8 + at) = quantize8(dg, &code);
        if (l == 0) dh_scales[r * 2 * nb + blk] = (uint8_t)code;
        *reinterpret_cast<uint2*>(dh8 + at + inter) = quantize8(du, &code);
        if (l == 0) dh_scales[r * 2 * nb + nb + blk] = (uint8_t)code;
      }
    }
    if (!dgates) continue;
#pragma unroll
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, kWave);
    // two sets of partial sums: the next pair's writes meet the last reads of
    // the one before only after another barrier
    if ((threadIdx.x & 63) == 0) part[flip][threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
      dgates[p] = (part[flip][0] + part[flip][1]) + (part[flip][2] + part[flip][3]);
    flip ^= 1;
  }
}

// Workgroups of 256 for this many threads; the kernels stride over the rest
// (a launch holds fewer than 2^32 threads).
constexpr int64_t kMostGroups = 1 << 22;
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
  hipLaunchKernelGGL(k_swiglu_fp8_bwd, dim3((unsigned)std::min<int64_t>(P, kMostGroups)), dim3(256), 0, s,
                     da, h8, h_scales, gates, inv_perm, P, inter, dh, dh8, dh_scales, dgates);
  return hipGetLastError();
}

}  // namespace qgg
