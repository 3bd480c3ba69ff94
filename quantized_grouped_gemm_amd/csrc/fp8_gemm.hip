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


// Tile row r of an LDS stage is 128 bytes; its 16-byte chunk c sits at slot c ^
// (r & 7), so that eight consecutive rows' reads of one chunk hit distinct banks.

// Eight rows x 16 columns of bytes by a transposing LDS read: within each
// 16-lane group, lane p points at eight bytes (row p / 2, half p & 1) and
// lane i receives column i of the eight rows.
__device__ __forceinline__ i32x2_t lds_tr8(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)p);
}

// first[e] = tiles of up to MT rows of the experts before e, first[E] = all of
// them (256 threads, four experts each; E <= 1024).
__device__ __forceinline__ void count_tiles(const int32_t* counts, int E, int MT, int* first,
                                            int* scratch) {
  int n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * threadIdx.x + j;
    n[j] = sum;
    sum += ((e < E ? counts[e] : 0) + MT - 1) / MT;
  }
  int total;
  const int before = block_excl_scan(sum, scratch, &total);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (4 * (int)threadIdx.x + j < E) first[4 * threadIdx.x + j] = before + n[j];
  if (threadIdx.x == 0) first[E] = total;
  __syncthreads();
}

// Tile number t: the thread that looks at its expert leaves {expert, row0,
// rows} in out.
__device__ __forceinline__ void find_tile(int t, const int* first, const int32_t* counts,
                                          const int32_t* offsets, int E, int MT, int* out) {
  for (int e = threadIdx.x; e < E; e += 256) {
    const int k = t - first[e];
    if (k >= 0 && t < first[e + 1]) {
      out[0] = e;
      out[1] = offsets[e] + k * MT;
      out[2] = min(MT, counts[e] - k * MT);
    }
  }
}

// Stages in the LDS ring of activation tiles, and weight steps in flight per
// wavefront in registers (one step is 64 columns x 128 = 8 KiB).
constexpr int kNBuf = 4;
template <int MB>
constexpr int w_ring() { return 2; }

// One reduction step of a wavefront's 16 NB columns of W.
template <int NB>
struct WStep {
  i32x8_t w[NB];
};

struct Item {
  int expert, row0, nrows, nt;
};

// Copies of the activation tile: slot p = 256 i + tid of a stage is slot p & 7
// of tile row p / 8.  Rows past the tile's end repeat its first; columns past
// the reduced width read zeros (offsets outside the buffer do).
template <int NCA>
struct RowCopy {
  const uint8_t* a;
  uint32_t bytes;
  uint32_t off[NCA];
  int col;
  __device__ __forceinline__ void init(const Fp8GemmArgs& g, const Item& it, int red) {
    a = g.a;
    bytes = (uint32_t)(g.a_rows * red);
    col = ((threadIdx.x & 7) ^ ((threadIdx.x >> 3) & 7)) * 16;
#pragma unroll
    for (int i = 0; i < NCA; ++i) {
      const int r = 32 * i + (threadIdx.x >> 3);
      const int rr = it.row0 + (r < it.nrows ? r : 0);
      const uint32_t src = g.tokens ? g.perm[rr] / g.topk : rr;
      off[i] = src * (uint32_t)red + (uint32_t)col;
    }
  }
  // step `st` of a width that is a multiple of 128: past the end the buffer is
  // taken to be empty
  __device__ __forceinline__ void copy_whole(int st, int steps, int wave, uint8_t* buf) const {
    const __amdgpu_buffer_rsrc_t rsrc = raw_buffer(a, st < steps ? bytes : 0u);
#pragma unroll
    for (int i = 0; i < NCA; ++i)
      copy16_to_lds(rsrc, off[i], (uint32_t)st * 128u, buf + (256 * i + 64 * wave) * 16);
  }
  // step `st` of any width
  __device__ __forceinline__ void copy_part(int st, int red, int wave, uint8_t* buf) const {
    const __amdgpu_buffer_rsrc_t rsrc = raw_buffer(a, bytes);
    const bool in = st * 128 + col < red;
#pragma unroll
    for (int i = 0; i < NCA; ++i)
      copy16_to_lds(rsrc, in ? off[i] + st * 128 : 0xFFFFFFF0u, 0,
                    buf + (256 * i + 64 * wave) * 16);
  }
};

// Scale bytes of the tile's rows for the steps [st0, st0 + n): sc[step -
// st0][row & 15][row >> 4], so that a lane reads the MB scales of its rows (one
// per 16-row block) at once.  Steps at and past `steps` get 1.0.
constexpr int kPiece = 64;

template <int MB, int NMB>
__device__ __forceinline__ void stage_scales(const Fp8GemmArgs& g, const Item& it, int st0, int n,
                                             int steps, uint8_t* sc) {
  const bool words = (steps & 3) == 0 && (reinterpret_cast<uintptr_t>(g.a_scales) & 3) == 0;
  for (int v = threadIdx.x; v < 32 * NMB; v += 256) {
    const int r = v >> 1;                        // two threads a row
    const int rr = it.row0 + (r < it.nrows ? r : 0);
    const int64_t src = g.tokens ? g.perm[rr] / g.topk : rr;
    const uint8_t* row = g.a_scales + src * steps + st0;
    uint8_t* out = sc + (r & 15) * MB + (r >> 4);
    if (words) {                                 // st0 and n are multiples of 4 then
#pragma unroll 4
      for (int w = v & 1; w < n / 4; w += 2) {
        const uint32_t x = reinterpret_cast<const uint32_t*>(row)[w];
#pragma unroll
        for (int j = 0; j < 4; ++j) out[(4 * w + j) * 16 * MB] = (uint8_t)(x >> (8 * j));
      }
    } else {
      for (int i = v & 1; i < n; i += 2) out[i * 16 * MB] = st0 + i < steps ? row[i] : 127;
    }
  }
}

// The wavefront's own weight scales of the same steps: wt[wave][step - st0],
// read at `scales` + step * stride (past `steps` the last one again).
template <bool WF32>
__device__ __forceinline__ void stage_w_scales(const void* scales, int64_t at, int stride, int st0,
                                               int n, int steps, uint32_t* wt) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = lane; i < n; i += 64) {
    const int64_t si = at + (int64_t)min(st0 + i, steps - 1) * stride;
    wt[wave * kPiece + i] = WF32 ? static_cast<const uint32_t*>(scales)[si]
                                 : static_cast<const uint8_t*>(scales)[si];
  }
}

// MB scale bytes of a lane as MFMA scale operands: block mb is byte mb & 3 of
// word mb / 4.
template <int MB>
__device__ __forceinline__ void read_scales(const uint8_t* sc, int st, int i16, int x[2]) {
  const uint8_t* at = sc + (st * 16 + i16) * MB;
  if constexpr (MB == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    x[0] = (int)v.x;
    x[1] = (int)v.y;
  } else if constexpr (MB == 4) {
    x[0] = *reinterpret_cast<const int*>(at);
  } else {
    x[0] = *reinterpret_cast<const uint16_t*>(at);
  }
}

// Rows of block mb; `at` = lane's offset of chunk q in row i16
__device__ __forceinline__ i32x8_t read_rows(const uint8_t* as, int mb, int at) {
  const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(as + mb * 2048 + at);
  const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(as + mb * 2048 + (at ^ 64));
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ int rows_at(int i16, int q) { return i16 * 128 + ((q ^ (i16 & 7)) << 4); }

// acc += scales * (W block . rows of block mb)
template <bool WF32, int SEL>
__device__ __forceinline__ void mfma_block(const i32x8_t& w, const i32x8_t& x, uint32_t ws, int xs,
                                           f32x4_t& acc) {
  if constexpr (WF32) {
    const f32x4_t part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        w, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, SEL, xs);
    const float f = __uint_as_float(ws);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = __builtin_fmaf(part[j], f, acc[j]);
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, (int)ws, SEL, xs);
  }
}

// One reduction step: the operand rows of the next 16-row block are read from
// LDS while the matrix core works on this one's (the group barriers pin two
// reads, four MFMAs, two reads, ...).
template <bool WF32, int NMB, int NB>
__device__ __forceinline__ void mfma_step(const uint8_t* as, const WStep<NB>& w, uint32_t ws, const int xs[2],
                                          int at, f32x4_t (&acc)[NMB][NB]) {
  using std::integral_constant;
  i32x8_t x = read_rows(as, 0, at);
  auto row_block = [&](auto mbc) {
    constexpr int mb = decltype(mbc)::value;
    if constexpr (mb < NMB) {
      i32x8_t nx = x;
      if constexpr (mb + 1 < NMB) nx = read_rows(as, mb + 1, at);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        mfma_block<WF32, (mb & 3)>(w.w[nb], x, ws, xs[mb >> 2], acc[mb][nb]);
      x = nx;
    }
  };
  row_block(integral_constant<int, 0>{});
  row_block(integral_constant<int, 1>{});
  row_block(integral_constant<int, 2>{});
  row_block(integral_constant<int, 3>{});
  row_block(integral_constant<int, 4>{});
  row_block(integral_constant<int, 5>{});
  row_block(integral_constant<int, 6>{});
  row_block(integral_constant<int, 7>{});
}

template <bool WF32, int NMB, int NB>
__device__ __forceinline__ void mfma_schedule() {
  __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    if (mb + 1 < NMB) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (WF32) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      if (mb + 1 == NMB) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    }
  }
}

// One item of y = a W^T: rows [row0, row0 + nrows) of an expert x 64 NB
// columns, NMB live 16-row blocks.  Weights go from memory straight into the MFMA's A
// registers, w_ring steps ahead; the rows go through a ring of LDS stages,
// kNBuf - 1 ahead; the barrier that ends a step waits for the next step's
// copies only.  The loop is branch-free, four steps a round: past the last step
// the weights repeat it and the rows are zeros with scale 1, which adds nothing.
template <bool WF32, int MB, int NMB, int NB>
__device__ __forceinline__ void nt_item(const Fp8GemmArgs& g, const Item& it, const LdsRing4& As,
                                        uint8_t* sc, uint32_t* wt) {
  constexpr int kRing = w_ring<MB>();
  constexpr int kNCA = NMB / 2 > 0 ? NMB / 2 : 1;
  constexpr int kStageLoads = kNCA + 2 * NB;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int i16 = lane & 15, q = lane >> 4;
  const int steps = g.K >> 7;
  const int at = rows_at(i16, q);
  RowCopy<kNCA> rc;
  rc.init(g, it, g.K);

  // this wavefront's columns, in NB / 4 groups of 64 that share a scale; a
  // group past the edge repeats the last columns and stores nothing
  constexpr int kG = NB / 4;
  const int base = it.nt * 64 * NB + wave * 16 * NB;
  int cg[kG];
#pragma unroll
  for (int j = 0; j < kG; ++j) cg[j] = min(base + 64 * j, g.N - 64);
  const uint32_t wbytes = (uint32_t)g.N * (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t wrsrc = raw_buffer(g.w + (int64_t)it.expert * wbytes, wbytes);
  const int64_t sat = ((int64_t)it.expert * ((g.N + 127) >> 7) + (cg[0] >> 7)) * steps;
  uint32_t wv[kG];
#pragma unroll
  for (int j = 0; j < kG; ++j)
    wv[j] = (uint32_t)(cg[j] + 16 * (i16 >> 2) + (i16 & 3)) * (uint32_t)g.K + 16 * q;
  auto load_w = [&](int st, WStep<NB>& w) {
    const int s = st < steps ? st : steps - 1;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const uint32_t so = (uint32_t)s * 128u + (uint32_t)(nb & 3) * 4u * (uint32_t)g.K;
      const u32x4_t lo = __builtin_amdgcn_raw_buffer_load_b128(wrsrc, wv[nb >> 2], so, 0);
      const u32x4_t hi = __builtin_amdgcn_raw_buffer_load_b128(wrsrc, wv[nb >> 2], so + 64, 0);
      w.w[nb] = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                        (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
  };

  f32x4_t acc[NMB][NB];
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  using std::integral_constant;
  for (int st0 = 0; st0 < steps; st0 += kPiece) {
    const int n = (min(kPiece, steps - st0) + 3) & ~3;
    WStep<NB> ring[kRing];
    rc.copy_whole(st0, steps, wave, As.b[0]);
    rc.copy_whole(st0 + 1, steps, wave, As.b[1]);
    rc.copy_whole(st0 + 2, steps, wave, As.b[0] + 16 * MB * 128);
    compiler_fence();
#pragma unroll
    for (int r = 0; r < kRing; ++r) load_w(st0 + r, ring[r]);
    stage_scales<MB, NMB>(g, it, st0, n, steps, sc);
    stage_w_scales<WF32>(g.w_scales, sat, 1, st0, n, steps, wt);
    stage_barrier<0>();
    // step i reads stage (i / 2) & 1 of object i & 1 while step i + 3 goes to
    // the other object
    auto kstage = [&](int i, WStep<NB>& w, const uint8_t* rows, uint8_t* next) {
      rc.copy_whole(st0 + i + kNBuf - 1, steps, wave, next);
      int xs[2];
      read_scales<MB>(sc, i, i16, xs);
      mfma_step<WF32, NMB, NB>(rows, w, wt[wave * kPiece + i], xs, at, acc);
      load_w(st0 + i + kRing, w);
      mfma_schedule<WF32, NMB, NB>();
      // the copies of step i + 1 were issued two steps ago
      stage_barrier<2 * kStageLoads>();
    };
    constexpr int kStage = 16 * MB * 128;
#pragma nounroll
    for (int i = 0; i < n; i += 2) {
      const int odd = (i >> 1) & 1;
      kstage(i, ring[0], As.b[0] + odd * kStage, As.b[1] + (odd ^ 1) * kStage);
      kstage(i + 1, ring[1], As.b[1] + odd * kStage, As.b[0] + odd * kStage);
    }
    // the copies past the last step land, and every wavefront is done with the
    // ring and the scales, before they are written again
    __builtin_amdgcn_s_waitcnt(vm_lgkm0_imm(0));
    __syncthreads();
  }
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    const int r = 16 * mb + i16;
    if (r >= it.nrows) continue;
    // block 4 j + nb holds columns 16 q + 4 nb .. + 3 of group j
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      if (base + 64 * j >= g.N) continue;
      uint16_t* out = g.y + (int64_t)(it.row0 + r) * g.N + cg[j] + 16 * q;
      const f32x4_t* v = acc[mb] + 4 * j;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_t*>(out + 8 * h) = u32x4_t{
            pack_bf16x2(v[2 * h][0], v[2 * h][1]), pack_bf16x2(v[2 * h][2], v[2 * h][3]),
            pack_bf16x2(v[2 * h + 1][0], v[2 * h + 1][1]),
            pack_bf16x2(v[2 * h + 1][2], v[2 * h + 1][3])};
    }
  }
}

// One item of y = a W: the weight step (128 rows of W x 64 columns a wavefront)
// goes through LDS and comes back through transposing reads.
template <bool WF32, int MB, int NMB>
__device__ __forceinline__ void t_item(const Fp8GemmArgs& g, const Item& it, uint8_t* as,
                                       uint8_t* ws, uint8_t* sc, uint32_t* wt) {
  constexpr int kNCA = NMB / 2 > 0 ? NMB / 2 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int i16 = lane & 15, q = lane >> 4;
  const int steps = (g.N + 127) >> 7;
  const int KB = g.K >> 7;
  const int at = rows_at(i16, q);
  RowCopy<kNCA> rc;
  rc.init(g, it, g.N);

  const int base = it.nt * 256 + wave * 64;
  const bool active = base < g.K;
  const int cbase = active ? base : g.K - 64;
  const uint32_t wbytes = (uint32_t)g.N * (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t wrsrc = raw_buffer(g.w + (int64_t)it.expert * wbytes, wbytes);
  const int64_t sat = (int64_t)it.expert * steps * KB + (cbase >> 7);
  uint8_t* mine = ws + wave * 8192;

  f32x4_t acc[NMB][4];
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  for (int st = 0; st < steps; ++st) {
    if (st % kPiece == 0) {
      const int n = (min(kPiece, steps - st) + 3) & ~3;
      stage_scales<MB, NMB>(g, it, st, n, steps, sc);
      stage_w_scales<WF32>(g.w_scales, sat, KB, st, n, steps, wt);
    }
    rc.copy_part(st, g.N, wave, as);
    // slot 4 r + s of a wavefront's 8 KiB holds chunk s ^ (r / 2 & 3) of row r
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = 64 * j + lane, r = slot >> 2;
      const int chunk = (slot & 3) ^ ((r >> 1) & 3);
      const uint32_t n = st * 128 + r;
      const uint32_t off = n < (uint32_t)g.N ? n * (uint32_t)g.K + cbase + 16 * chunk : 0xFFFFFFF0u;
      copy16_to_lds(wrsrc, off, 0, mine + j * 1024);
    }
    WStep<4> w;
    __builtin_amdgcn_s_waitcnt(vm_lgkm0_imm(0));
    __syncthreads();
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // reduced values 16 q + 64 (t / 2) + 8 (t & 1) .. + 7, columns 16 nb ..
        const int r = 16 * q + 64 * (t >> 1) + 8 * (t & 1) + (i16 >> 1);
        const int slot = r * 4 + (nb ^ ((r >> 1) & 3));
        const i32x2_t v = lds_tr8(mine + slot * 16 + (i16 & 1) * 8);
        w.w[nb][2 * t] = v[0];
        w.w[nb][2 * t + 1] = v[1];
      }
    int xs[2];
    read_scales<MB>(sc, st % kPiece, i16, xs);
    mfma_step<WF32, NMB, 4>(as, w, wt[wave * kPiece + st % kPiece], xs, at, acc);
    __syncthreads();
  }
  if (!active) return;
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    const int r = 16 * mb + i16;
    if (r >= it.nrows) continue;
    // block nb holds columns 16 nb + 4 q .. + 3
    uint16_t* out = g.y + (int64_t)(it.row0 + r) * g.K + cbase + 4 * q;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
      *reinterpret_cast<uint2*>(out + 16 * nb) =
          make_uint2(pack_bf16x2(acc[mb][nb][0], acc[mb][nb][1]),
                     pack_bf16x2(acc[mb][nb][2], acc[mb][nb][3]));
  }
}

// Workgroups take items (tile, 64 NB columns) in order, eight interleaved
// stretches of them, one per XCD (workgroup b runs on XCD b mod 8): the columns
// of a tile and the tiles of an expert then share one L2.
template <bool TRANS, bool WF32, int MB, int NB>
__global__ __launch_bounds__(256, NB == 8 ? 1 : 2) void k_fp8_gemm(Fp8GemmArgs g, int ntn) {
  // separate objects: the compiler tells a copy into one from a read of another
  __shared__ __attribute__((aligned(16))) uint8_t b0[16 * MB * 256];
  __shared__ __attribute__((aligned(16))) uint8_t b1[TRANS ? 32768 : 16 * MB * 256];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kPiece * 16 * MB];
  const LdsRing4 As{{b0, b1, nullptr, nullptr}};
  __shared__ int scratch[16];
  __shared__ int tile[3];
  __shared__ uint32_t wt[4 * kPiece];
  __shared__ int tiles_before[1025];
  count_tiles(g.counts, g.E, 16 * MB, tiles_before, scratch);
  const int items = tiles_before[g.E] * ntn;
  const int per = (items + 7) >> 3;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, items);
  for (int i = first + (blockIdx.x >> 3); i < last; i += gridDim.x >> 3) {
    const int t = i / ntn;
    __syncthreads();
    find_tile(t, tiles_before, g.counts, g.offsets, g.E, 16 * MB, tile);
    __syncthreads();
    Item it;
    it.expert = __builtin_amdgcn_readfirstlane(tile[0]);
    it.row0 = __builtin_amdgcn_readfirstlane(tile[1]);
    it.nrows = __builtin_amdgcn_readfirstlane(tile[2]);
    it.nt = i - t * ntn;
    const int live = (it.nrows + 15) >> 4;
    auto run = [&](auto n) {
      constexpr int NMB = decltype(n)::value;
      if constexpr (TRANS) t_item<WF32, MB, NMB>(g, it, b0, b1, sc, wt);
      else nt_item<WF32, MB, NMB, NB>(g, it, As, sc, wt);
    };
    using std::integral_constant;
    if constexpr (MB == 8) {
      if (live > 6) run(integral_constant<int, 8>{});
      else if (live > 4) run(integral_constant<int, 6>{});
      else if (live > 2) run(integral_constant<int, 4>{});
      else run(integral_constant<int, 2>{});
    } else if constexpr (MB == 4) {
      if (live > 2) run(integral_constant<int, 4>{});
      else if (live > 1) run(integral_constant<int, 2>{});
      else run(integral_constant<int, 1>{});
    } else {
      if (live > 1) run(integral_constant<int, 2>{});
      else run(integral_constant<int, 1>{});
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

template <bool TRANS, bool WF32, int MB, int NB>
static void launch(const Fp8GemmArgs& g, int64_t tiles, hipStream_t s) {
  const int ntn = ((TRANS ? g.K : g.N) + 64 * NB - 1) / (64 * NB);
  // a multiple of 8: one stretch of items per XCD
  const int64_t resident = (int64_t)num_cus() / 8 * 8 * (NB == 8 ? 1 : 2);
  const int64_t grid = std::min<int64_t>((tiles * ntn + 7) / 8 * 8, resident);
  hipLaunchKernelGGL((k_fp8_gemm<TRANS, WF32, MB, NB>), dim3((unsigned)grid), dim3(256), 0, s, g,
                     ntn);
}

template <bool TRANS, bool WF32>
static void launch_sized(const Fp8GemmArgs& g, hipStream_t s) {
  const int mb = tile_blocks(g);
  const char* xx = getenv("QGG_X");
  const int64_t tiles = std::min<int64_t>(g.P, g.P / (16 * mb) + g.E);
  if (mb == 2) launch<TRANS, WF32, 2, 4>(g, tiles, s);
  else if (mb == 4) launch<TRANS, WF32, 4, 4>(g, tiles, s);
  else if (TRANS || WF32 || xx || tiles * (g.N / 512) < num_cus()) launch<TRANS, WF32, 8, 4>(g, tiles, s);
  else launch<false, false, 8, 8>(g, tiles, s);
}

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  TimedLaunch timed_(g.trans ? kLGemmT : kLGemm, s);
  if (g.trans && g.w_f32) launch_sized<true, true>(g, s);
  else if (g.trans) launch_sized<true, false>(g, s);
  else if (g.w_f32) launch_sized<false, true>(g, s);
  else launch_sized<false, false>(g, s);
  return hipGetLastError();
}

}  // namespace qgg
