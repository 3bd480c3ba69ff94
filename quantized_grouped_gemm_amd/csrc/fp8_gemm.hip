// Grouped product of routed rows with 8-bit expert weights:
//   y[i][:] = a_row(i) . W_e^T   (reduce over K)   or   a_row(i) . W_e   (reduce over N)
// with E4M3 codes on both sides, an E8M0 scale per 128 reduced columns of a
// row of a, and a scale (E8M0 or fp32) per 128 x 128 block of W_e.  For one
// output, with r the reduction index in blocks of 128,
//   y = sum_R sa[i][R] sw[R, c / 128] sum_{r in R} a8[i][r] w8[r, c].
// v_mfma_scale_f32_16x16x128_f8f6f4 forms one block's inner sum for 16 x 16
// outputs and applies a power of two to each operand by itself, so E8M0 scales
// cost nothing; with fp32 weight scales the block's sum lands in a fresh
// accumulator and one fused multiply-add per output carries the scale.
//
// Operands: W is the MFMA's A matrix (16 output columns), the activation rows
// its B matrix (16 rows), so a lane ends with four consecutive output columns
// of one row.  The order of the 128 reduced values inside an MFMA is free as
// long as both operands share it: lane (i, q) holds bytes 16 q .. 16 q + 15 of
// the first and of the second 64.
#include "qgg_device.hpp"
#include "qgg_internal.hpp"

namespace qgg {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));

constexpr int kBN = 256;                         // output columns per workgroup, 64 a wavefront

__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// Eight rows x 16 columns of bytes by a transposing LDS read: within each
// 16-lane group, lane p points at eight bytes (row p / 2, half p & 1) and
// lane i receives column i of the eight rows.
__device__ __forceinline__ i32x2_t lds_tr8(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)p);
}

// The tile of up to MT rows that is number `t` of the experts' tiles, experts
// ascending: thread tid looks at experts 4 tid .. 4 tid + 3 (first[] = tiles
// before them) and the one that holds it leaves {expert, row0, rows} in LDS.
struct TileFinder {
  int first[4], cnt[4];
  int total;
  __device__ void init(const int32_t* counts, int E, int MT, int* lds) {
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * threadIdx.x + j;
      cnt[j] = e < E ? counts[e] : 0;
      first[j] = sum;
      sum += (cnt[j] + MT - 1) / MT;
    }
    const int before = block_excl_scan(sum, lds, &total);
#pragma unroll
    for (int j = 0; j < 4; ++j) first[j] += before;
  }
  __device__ void find(int t, const int32_t* offsets, int MT, int* out) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = t - first[j];
      if (k >= 0 && k * MT < cnt[j]) {
        out[0] = 4 * threadIdx.x + j;
        out[1] = offsets[4 * threadIdx.x + j] + k * MT;
        out[2] = min(MT, cnt[j] - k * MT);
      }
    }
  }
};

// One item: rows [row0, row0 + nrows) of an expert x 256 columns, NMB live
// 16-row blocks.
template <bool TRANS, bool WF32, int MB, int NMB>
__device__ __forceinline__ void fp8_item(const Fp8GemmArgs& g, int expert, int row0, int nrows,
                                         int nt, uint8_t* as, uint8_t* ws, uint8_t* sc) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int i16 = lane & 15, q = lane >> 4;
  const int red = TRANS ? g.N : g.K;             // reduced width
  const int cols = TRANS ? g.K : g.N;            // output width
  const int steps = (red + 127) >> 7;
  const int KB = g.K >> 7;                       // scale columns of W

  const __amdgpu_buffer_rsrc_t arsrc = raw_buffer(g.a, (uint32_t)(g.a_rows * red));
  uint32_t aoff[MB / 2];
  int acol[MB / 2];
#pragma unroll
  for (int i = 0; i < MB / 2; ++i) {
    const int p = 256 * i + tid;
    const int r = p >> 3;
    const int rr = row0 + (r < nrows ? r : 0);
    const int64_t src = g.tokens ? g.perm[rr] / g.topk : rr;
    acol[i] = ((p & 7) ^ swz(r)) * 16;
    aoff[i] = (uint32_t)(src * red + acol[i]);
  }
  // scale bytes of the tile's rows: sc[step][i16][mb]
  for (int v = tid; v < 16 * NMB * steps; v += 256) {
    const int r = v / steps, st = v - r * steps;
    const int rr = row0 + (r < nrows ? r : 0);
    const int64_t src = g.tokens ? g.perm[rr] / g.topk : rr;
    sc[(st * 16 + (r & 15)) * MB + (r >> 4)] = g.a_scales[src * steps + st];
  }

  const int base = nt * kBN + wave * 64;
  const bool active = base < cols;
  const int cbase = active ? base : cols - 64;
  const uint32_t wbytes = (uint32_t)g.N * (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t wrsrc = raw_buffer(g.w + (int64_t)expert * wbytes, wbytes);
  const int64_t nscales = (int64_t)((g.N + 127) >> 7) * KB;
  const uint8_t* s8 = static_cast<const uint8_t*>(g.w_scales) + (WF32 ? 4 : 1) * expert * nscales;

  f32x4_t acc[NMB][4];
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int st = 0; st < steps; ++st) {
#pragma unroll
    for (int i = 0; i < MB / 2; ++i) {
      const uint32_t off = st * 128 + acol[i] < red ? aoff[i] + st * 128 : 0xFFFFFFF0u;
      copy16_to_lds(arsrc, off, 0, as + (256 * i + 64 * wave) * 16);
    }
    i32x8_t w[4];
    if constexpr (TRANS) {
      uint8_t* mine = ws + wave * 8192;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int slot = 64 * j + lane, r = slot >> 2;
        const int chunk = (slot & 3) ^ ((r >> 1) & 3);
        const uint32_t n = st * 128 + r;
        const uint32_t off = n < (uint32_t)g.N ? n * (uint32_t)g.K + cbase + 16 * chunk : 0xFFFFFFF0u;
        copy16_to_lds(wrsrc, off, 0, mine + j * 1024);
      }
    } else {
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const uint32_t n = cbase + 16 * (i16 >> 2) + 4 * nb + (i16 & 3);
        const uint32_t off = n * (uint32_t)g.K + st * 128 + 16 * q;
        const u32x4_t lo = __builtin_amdgcn_raw_buffer_load_b128(wrsrc, off, 0, 0);
        const u32x4_t hi = __builtin_amdgcn_raw_buffer_load_b128(wrsrc, off + 64, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[nb][j] = (int)lo[j];
          w[nb][4 + j] = (int)hi[j];
        }
      }
    }
    const int64_t si = TRANS ? (int64_t)st * KB + (cbase >> 7) : (int64_t)(cbase >> 7) * KB + st;
    const float wf = WF32 ? reinterpret_cast<const float*>(s8)[si] : 1.0f;
    const int wsc = WF32 ? 127 : s8[si];
    __builtin_amdgcn_s_waitcnt(vm_lgkm0_imm(0));
    __syncthreads();
    if constexpr (TRANS) {
      const uint8_t* mine = ws + wave * 8192;
      const int p = i16;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          // reduced values 16 q + 64 (t / 2) + 8 (t & 1) .. + 7, columns 16 nb ..
          const int r = 16 * q + 64 * (t >> 1) + 8 * (t & 1) + (p >> 1);
          const int slot = r * 4 + (nb ^ ((r >> 1) & 3));
          const i32x2_t v = lds_tr8(mine + slot * 16 + (p & 1) * 8);
          w[nb][2 * t] = v[0];
          w[nb][2 * t + 1] = v[1];
        }
    }
#pragma unroll
    for (int mb = 0; mb < NMB; ++mb) {
      const int r = 16 * mb + i16;
      const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(as + r * 128 + ((q ^ swz(r)) << 4));
      const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(as + r * 128 + (((q + 4) ^ swz(r)) << 4));
      i32x8_t x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = (int)lo[j];
        x[4 + j] = (int)hi[j];
      }
      const int xs = sc[(st * 16 + i16) * MB + mb];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        if constexpr (WF32) {
          const f32x4_t part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              w[nb], x, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, xs);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[mb][nb][j] = __builtin_fmaf(part[j], wf, acc[mb][nb][j]);
        } else {
          acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[nb], x, acc[mb][nb], 0,
                                                                         0, 0, wsc, 0, xs);
        }
      }
    }
    __syncthreads();
  }
  if (!active) return;
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    const int r = 16 * mb + i16;
    if (r >= nrows) continue;
    uint16_t* out = g.y + (int64_t)(row0 + r) * cols + cbase;
    if constexpr (TRANS) {
      // block nb holds columns 16 nb + 4 q .. + 3
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
        *reinterpret_cast<uint2*>(out + 16 * nb + 4 * q) =
            make_uint2(pack_bf16x2(acc[mb][nb][0], acc[mb][nb][1]),
                       pack_bf16x2(acc[mb][nb][2], acc[mb][nb][3]));
    } else {
      // block nb holds columns 16 q + 4 nb .. + 3
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_t*>(out + 16 * q + 8 * h) =
            u32x4_t{pack_bf16x2(acc[mb][2 * h][0], acc[mb][2 * h][1]),
                    pack_bf16x2(acc[mb][2 * h][2], acc[mb][2 * h][3]),
                    pack_bf16x2(acc[mb][2 * h + 1][0], acc[mb][2 * h + 1][1]),
                    pack_bf16x2(acc[mb][2 * h + 1][2], acc[mb][2 * h + 1][3])};
    }
  }
}

template <bool TRANS, bool WF32, int MB>
__global__ __launch_bounds__(256) void k_fp8_gemm(Fp8GemmArgs g, int ntn) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int scratch[16];
  __shared__ int tile[3];
  uint8_t* as = lds;                             // [16 MB][128]
  uint8_t* ws = as + 16 * MB * 128;              // TRANS: [4 waves][128][64]
  uint8_t* sc = ws + (TRANS ? 32768 : 0);        // row scales [steps][16][MB]
  TileFinder tf;
  tf.init(g.counts, g.E, 16 * MB, scratch);
  const int items = tf.total * ntn;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int t = it / ntn;
    __syncthreads();
    tf.find(t, g.offsets, 16 * MB, tile);
    __syncthreads();
    const int expert = __builtin_amdgcn_readfirstlane(tile[0]);
    const int row0 = __builtin_amdgcn_readfirstlane(tile[1]);
    const int nrows = __builtin_amdgcn_readfirstlane(tile[2]);
    const int nt = it - t * ntn;
    const int live = (nrows + 15) >> 4;
    if constexpr (MB == 8) {
      if (live > 6) fp8_item<TRANS, WF32, MB, 8>(g, expert, row0, nrows, nt, as, ws, sc);
      else if (live > 4) fp8_item<TRANS, WF32, MB, 6>(g, expert, row0, nrows, nt, as, ws, sc);
      else if (live > 2) fp8_item<TRANS, WF32, MB, 4>(g, expert, row0, nrows, nt, as, ws, sc);
      else fp8_item<TRANS, WF32, MB, 2>(g, expert, row0, nrows, nt, as, ws, sc);
    } else if constexpr (MB == 4) {
      if (live > 2) fp8_item<TRANS, WF32, MB, 4>(g, expert, row0, nrows, nt, as, ws, sc);
      else if (live > 1) fp8_item<TRANS, WF32, MB, 2>(g, expert, row0, nrows, nt, as, ws, sc);
      else fp8_item<TRANS, WF32, MB, 1>(g, expert, row0, nrows, nt, as, ws, sc);
    } else {
      if (live > 1) fp8_item<TRANS, WF32, MB, 2>(g, expert, row0, nrows, nt, as, ws, sc);
      else fp8_item<TRANS, WF32, MB, 1>(g, expert, row0, nrows, nt, as, ws, sc);
    }
  }
}

// 16-row blocks per tile: an expert has at most one row per token, so small
// batches fit every expert in one tile; larger ones go by the mean rows.
int tile_blocks(const Fp8GemmArgs& g) {
  const int64_t mean = (g.P + g.E - 1) / g.E;
  const int64_t rows = std::min<int64_t>(g.T, 64) == g.T ? g.T : mean;
  return rows <= 32 ? 2 : (rows <= 64 ? 4 : 8);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  TimedLaunch timed_(g.trans ? kLGemmT : kLGemm, s);
  const int mb = tile_blocks(g);
  const int ntn = ((g.trans ? g.K : g.N) + kBN - 1) / kBN;
  const int steps = ((g.trans ? g.N : g.K) + 127) / 128;
  const size_t lds = (size_t)16 * mb * 128 + (g.trans ? 32768 : 0) + (size_t)steps * 16 * mb;
  const int64_t tiles = std::min<int64_t>(g.P, g.P / (16 * mb) + g.E);
  const int64_t grid = std::min<int64_t>(tiles * ntn, (int64_t)num_cus() * 2);
  auto go = [&](auto trans, auto wf32, auto mbc) {
    hipLaunchKernelGGL((k_fp8_gemm<decltype(trans)::value, decltype(wf32)::value, decltype(mbc)::value>),
                       dim3((unsigned)grid), dim3(256), lds, s, g, ntn);
  };
  auto by_mb = [&](auto trans, auto wf32) {
    using std::integral_constant;
    if (mb == 8) go(trans, wf32, integral_constant<int, 8>{});
    else if (mb == 4) go(trans, wf32, integral_constant<int, 4>{});
    else go(trans, wf32, integral_constant<int, 2>{});
  };
  if (g.trans) {
    if (g.w_f32) by_mb(std::true_type{}, std::true_type{});
    else by_mb(std::true_type{}, std::false_type{});
  } else {
    if (g.w_f32) by_mb(std::false_type{}, std::true_type{});
    else by_mb(std::false_type{}, std::false_type{});
  }
  return hipGetLastError();
}

}  // namespace qgg
