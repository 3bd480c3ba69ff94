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
// long as both operands share it: lane (i, q) holds the 32 bytes from 64 (q &
// 1) + 32 (q / 2) of its row.
#include "qgg_device.hpp"
#include "qgg_internal.hpp"

namespace qgg {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));


// LDS has 64 banks of four bytes, so 16 lanes reading 16 bytes each are served
// at once if they touch each 16-byte slot of 256 bytes once.  Chunk c of a row
// sits at slot c ^ swz(row); the swizzles make the 16 lanes of an operand read
// (and the 32 of a transposing one) touch them all:
// activation rows r = 16 mb + 0 .. 15, 128 bytes each
__device__ __forceinline__ int swz_a(int r) { return (r ^ ((r >> 3) & 1)) & 7; }
// columns 64 g + 16 (i / 4) + 4 nb + i % 4 of W, i = 0 .. 15, 128 bytes each
__device__ __forceinline__ int swz_w(int r) { return ((r >> 1) & 1) | ((r >> 3) & 6); }
// rows of W r0 + 0 .. 7 and r0 + 64 .. 71, 256 bytes each
__device__ __forceinline__ int swz_t(int r) { return (r & 7) | ((r >> 3) & 8); }

// Eight rows x 16 columns of bytes by a transposing LDS read: within each
// 16-lane group, lane p points at eight bytes (row p / 2, half p & 1) and
// lane i receives column i of the eight rows.
__device__ __forceinline__ i32x2_t lds_tr8(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)p);
}

// first[e] = tiles of up to MT rows of the experts before e, first[E] = all of
// them (four experts a thread; E <= 1024, at least 256 threads).
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

// Item i: experts ascending, in an expert column group by column group, and
// the tiles of a column group side by side, so that the workgroups which read
// the same weights do so at the same time and share them in their L2.  The
// thread that looks at its expert leaves {expert, row0, rows, column group}.
__device__ __forceinline__ void find_item(int i, int ntn, const int* first, const int32_t* counts,
                                          const int32_t* offsets, int E, int* out) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const int f = first[e], n = first[e + 1] - f;
    const int p = i - f * ntn;
    if (p >= 0 && p < n * ntn) {
      const int nt = p / n, k = p - nt * n;
      const int c = counts[e];
      const int64_t blocks = (c + 15) >> 4;      // split into equal numbers of blocks
      const int b0 = (int)(k * blocks / n), b1 = (int)((k + 1) * blocks / n);
      out[0] = e;
      out[1] = offsets[e] + 16 * b0;
      out[2] = min(16 * b1, c) - 16 * b0;
      out[3] = nt;
    }
  }
}

// Stages in the LDS ring of activation tiles.
constexpr int kNBuf = 4;

// One reduction step of a wavefront's 64 columns of W, as MFMA operands.
struct WStep {
  i32x8_t w[4];
};

// The same as it is loaded.  Memory is read fastest where the four lanes of a
// quad take 64 consecutive bytes, while an MFMA operand wants a lane to hold
// one row: with one row a lane, every 16-byte piece is a cache access of its
// own (64 a load, which took 84 % of the kernel's cycles).  So
// lane 16 q + 4 a + p of load j of a pair of 16-row blocks (X, Y) takes chunk
// p of half q & 1 of row 4 a + j of block q < 2 ? X : Y; a 4 x 4 transposition
// in each quad gives the lane row 4 a + p's four chunks, and an exchange of
// the wavefront's halves splits them between X's operand and Y's.
struct WRaw {
  u32x4_t r[2][4];                               // [pair][j]
};

template <int CTRL>
__device__ __forceinline__ uint32_t quad_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Operands of one pair of blocks (x: the first, y: the second).
struct WPair {
  i32x8_t x, y;
};

__device__ __forceinline__ WPair to_operands(const u32x4_t (&raw)[4], int lane) {
  const bool odd1 = lane & 1, odd2 = lane & 2;
  WPair out;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {                // exchange bit 1 of j and of the lane
      const uint32_t x = raw[j][d], y = raw[j + 2][d];
      const uint32_t mx = quad_move<0x4E>(x), my = quad_move<0x4E>(y);
      v[j] = odd2 ? my : x;
      v[j + 2] = odd2 ? y : mx;
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {             // bit 0
      const uint32_t x = v[j], y = v[j + 1];
      const uint32_t mx = quad_move<0xB1>(x), my = quad_move<0xB1>(y);
      v[j] = odd1 ? my : x;
      v[j + 1] = odd1 ? y : mx;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const auto sw = __builtin_amdgcn_permlane32_swap(v[t], v[t + 2], false, false);
      out.x[4 * t + d] = (int)sw[0];
      out.y[4 * t + d] = (int)sw[1];
    }
  }
  return out;
}

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
    col = ((threadIdx.x & 7) ^ swz_a(threadIdx.x >> 3)) * 16;
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
    const uint32_t at = st < steps ? (uint32_t)st * 128u : 0u;
#pragma unroll
    for (int i = 0; i < NCA; ++i)
      copy16_to_lds(rsrc, off[i], at, buf + (256 * i + 64 * wave) * 16);
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

// MB scale bytes of a lane as MFMA scale operand: block mb is byte mb.
template <int MB>
__device__ __forceinline__ int read_scales(const uint8_t* sc, int st, int i16) {
  const uint8_t* at = sc + (st * 16 + i16) * MB;
  return MB == 4 ? *reinterpret_cast<const int*>(at) : *reinterpret_cast<const uint16_t*>(at);
}

// Rows of block mb; `at` = offset of the first of the lane's two chunks
__device__ __forceinline__ i32x8_t read_rows(const uint8_t* as, int mb, int at) {
  const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(as + mb * 2048 + at);
  const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(as + mb * 2048 + (at ^ 16));
  return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                 (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ int rows_at(int i16, int q) {
  return i16 * 128 + (((4 * (q & 1) + 2 * (q >> 1)) ^ swz_a(i16)) << 4);
}

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
template <bool WF32, int NMB>
__device__ __forceinline__ void mfma_step(const uint8_t* as, const WStep& w, uint32_t ws,
                                          int xs, int at, f32x4_t (&acc)[NMB][4]) {
  using std::integral_constant;
  i32x8_t x = read_rows(as, 0, at);
  auto row_block = [&](auto mbc) {
    constexpr int mb = decltype(mbc)::value;
    if constexpr (mb < NMB) {
      i32x8_t nx = x;
      if constexpr (mb + 1 < NMB) nx = read_rows(as, mb + 1, at);
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
        mfma_block<WF32, mb>(w.w[nb], x, ws, xs, acc[mb][nb]);
      x = nx;
    }
  };
  row_block(integral_constant<int, 0>{});
  row_block(integral_constant<int, 1>{});
  row_block(integral_constant<int, 2>{});
  row_block(integral_constant<int, 3>{});
}

template <bool WF32, int NMB>
__device__ __forceinline__ void mfma_schedule() {
  __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    if (mb + 1 < NMB) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (WF32) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
      if (mb + 1 == NMB) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
    }
  }
}

// One item of y = a W^T: rows [row0, row0 + nrows) of an expert x 256
// columns, NMB live 16-row blocks.  Weights go from memory straight into
// registers, kRing steps ahead (a step of a wavefront is 64 columns x 128 = 8
// KiB), past the caches, since one item uses them; the rows go through a ring of
// LDS stages, kNBuf - 1 ahead; the barrier that ends a step waits for the next
// step's copies only.  The loop is branch-free, in rounds of kRing steps: past
// the last step the weights repeat it and the rows are zeros with scale 1, which
// adds nothing.  Bound by the weights' bytes: 64 tokens over 384 uneven experts
// of [4096][7168] take 217 us, 300 tokens over 64 experts 299 us, 6.3 TB/s of
// the 6.3 that a plain stream of the same bytes reaches.
template <bool WF32, int MB, int NMB>
__device__ __forceinline__ void nt_item(const Fp8GemmArgs& g, const Item& it, const LdsRing4& As,
                                        uint8_t* sc, uint32_t* wt) {
  constexpr int kNCA = NMB / 2 > 0 ? NMB / 2 : 1;
  constexpr int kStageLoads = kNCA + 8;
  constexpr int kRing = MB == 2 ? 4 : 2;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int i16 = lane & 15, q = lane >> 4;
  const int steps = g.K >> 7;
  const int at = rows_at(i16, q);
  RowCopy<kNCA> rc;
  rc.init(g, it, g.K);

  const int base = it.nt * 256 + wave * 64;
  const bool active = base < g.N;
  const int cbase = active ? base : g.N - 64;    // a wave past the edge repeats the last columns
  const uint32_t wbytes = (uint32_t)g.N * (uint32_t)g.K;
  const __amdgpu_buffer_rsrc_t wrsrc = raw_buffer(g.w + (int64_t)it.expert * wbytes, wbytes);
  const int64_t sat = ((int64_t)it.expert * ((g.N + 127) >> 7) + (cbase >> 7)) * steps;
  const int a4 = (lane >> 2) & 3, p4 = lane & 3;
  const uint32_t wv =
      (uint32_t)(cbase + 16 * a4 + 4 * (q >> 1)) * (uint32_t)g.K + 64 * (q & 1) + 16 * p4;
  auto load_w = [&](int st, WRaw& w) {
    const int s = st < steps ? st : steps - 1;
#pragma unroll
    for (int pr = 0; pr < 2; ++pr)
#pragma unroll
      for (int j = 0; j < 4; ++j)                // row 16 a + 4 nb + j
        w.r[pr][j] = __builtin_amdgcn_raw_buffer_load_b128(
            wrsrc, wv, (uint32_t)s * 128u + (uint32_t)(8 * pr + j) * (uint32_t)g.K,
            kStreamed);
  };

  f32x4_t acc[NMB][4];
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  using std::integral_constant;
  for (int st0 = 0; st0 < steps; st0 += kPiece) {
    const int n = (min(kPiece, steps - st0) + 3) & ~3;
    WRaw ring[kRing];
    rc.copy_whole(st0, steps, wave, As.b[0]);
    rc.copy_whole(st0 + 1, steps, wave, As.b[1]);
    rc.copy_whole(st0 + 2, steps, wave, As.b[2]);
    compiler_fence();
#pragma unroll
    for (int r = 0; r < kRing; ++r) load_w(st0 + r, ring[r]);
    stage_scales<MB, NMB>(g, it, st0, n, steps, sc);
    stage_w_scales<WF32>(g.w_scales, sat, 1, st0, n, steps, wt);
    stage_barrier<0>();
    auto kstage = [&](int i, WRaw& raw, const uint8_t* rows, uint8_t* next) {
      rc.copy_whole(st0 + i + kNBuf - 1, steps, wave, next);
      compiler_fence();                          // the wait below counts on this order
      const int xs = read_scales<MB>(sc, i, i16);
      const uint32_t ws = wt[wave * kPiece + i];
      WStep w;
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        const WPair p = to_operands(raw.r[pr], lane);
        w.w[2 * pr] = p.x;
        w.w[2 * pr + 1] = p.y;
      }
      mfma_step<WF32, NMB>(rows, w, ws, xs, at, acc);
      load_w(st0 + i + kRing, raw);
      mfma_schedule<WF32, NMB>();
      // the copies of step i + 1 were issued two steps ago, before weights
      stage_barrier<2 * kStageLoads + 8>();
    };
#pragma nounroll
    for (int i = 0; i < n; i += kNBuf)
#pragma unroll
      for (int j = 0; j < kNBuf; ++j)
        kstage(i + j, ring[j % kRing], As.b[j], As.b[(j + kNBuf - 1) % kNBuf]);
    // the copies past the last step land, and every wavefront is done with the
    // ring and the scales, before they are written again
    __builtin_amdgcn_s_waitcnt(vm_lgkm0_imm(0));
    __syncthreads();
  }
  if (!active) return;
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    const int r = 16 * mb + i16;
    if (r >= it.nrows) continue;
    // block nb holds columns 16 q + 4 nb .. + 3
    uint16_t* out = g.y + (int64_t)(it.row0 + r) * g.N + cbase + 16 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<u32x4_t*>(out + 8 * h) =
          u32x4_t{pack_bf16x2(acc[mb][2 * h][0], acc[mb][2 * h][1]),
                  pack_bf16x2(acc[mb][2 * h][2], acc[mb][2 * h][3]),
                  pack_bf16x2(acc[mb][2 * h + 1][0], acc[mb][2 * h + 1][1]),
                  pack_bf16x2(acc[mb][2 * h + 1][2], acc[mb][2 * h + 1][3])};
  }
}

// One item of y = a W: the weight step (128 rows of W x 64 columns a wavefront)
// goes through LDS and comes back through transposing reads.  The copies take
// whole lines: in pieces of 64 bytes, past the caches, a line is fetched twice.
// Two workgroups a CU hide each other's waits; 64 tokens over 384 uneven experts
// of [4096][7168] take 248 us, a seventh more than the other direction.
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
  // four rows of 256 bytes at a time; slot s of row r holds chunk s ^ swz_t(r)
  const int wrow = (wave >> 1) * 64 + (wave & 1) * 4 + (lane >> 4);
  const int chunk = (lane & 15) ^ swz_t(wrow);
  const uint32_t woff = (uint32_t)wrow * (uint32_t)g.K +
                        (uint32_t)(min(it.nt * 256 + 64 * (chunk >> 2), g.K - 64) + 16 * (chunk & 3));
  const int tr_row = 64 * (q & 1) + 32 * (q >> 1) + (i16 >> 1);
  const int tr_at = tr_row * 256 + (((4 * wave) ^ swz_t(tr_row)) << 4) + (i16 & 1) * 8;

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
    // W rows past N lie past the buffer's end
#pragma unroll
    for (int j = 0; j < 8; ++j)
      copy16_to_lds<kStreamed>(wrsrc, woff + (uint32_t)(st * 128 + 8 * j) * (uint32_t)g.K, 0,
                               ws + ((wave >> 1) * 64 + (wave & 1) * 4 + 8 * j) * 256);
    WStep w;
    __builtin_amdgcn_s_waitcnt(vm_lgkm0_imm(0));
    __syncthreads();
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // reduced values tr_row's eight + 8 t, columns 16 nb ..
        const i32x2_t v = lds_tr8(ws + (tr_at ^ (nb << 4)) + t * 2048);
        w.w[nb][2 * t] = v[0];
        w.w[nb][2 * t + 1] = v[1];
      }
    const int xs = read_scales<MB>(sc, st % kPiece, i16);
    mfma_step<WF32, NMB>(as, w, wt[wave * kPiece + st % kPiece], xs, at, acc);
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

// Workgroups take items (tile, 256 columns) in order, from eight stretches of
// them, one per XCD (workgroup b runs on XCD b mod 8): the columns of a tile and
// the tiles of an expert then share one L2.
template <bool TRANS, bool WF32, int MB>
__global__ __launch_bounds__(256, 2) void k_fp8_gemm(Fp8GemmArgs g, int ntn) {
  // separate objects: the compiler tells a copy into one from a read of another
  constexpr int kRows = 16 * MB * 128;
  __shared__ __attribute__((aligned(16))) uint8_t b0[kRows];
  __shared__ __attribute__((aligned(16))) uint8_t b1[TRANS ? 32768 : kRows];
  __shared__ __attribute__((aligned(16))) uint8_t b2[TRANS ? 16 : kRows];
  __shared__ __attribute__((aligned(16))) uint8_t b3[TRANS ? 16 : kRows];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kPiece * 16 * MB];
  const LdsRing4 As{{b0, b1, b2, b3}};
  __shared__ int scratch[16];
  __shared__ int item[4];
  __shared__ uint32_t wt[4 * kPiece];
  __shared__ int tiles_before[1025];
  count_tiles(g.counts, g.E, 16 * MB, tiles_before, scratch);
  const int items = tiles_before[g.E] * ntn;
  const int per = (items + 7) >> 3;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, items);
  for (int i = first + (blockIdx.x >> 3); i < last; i += gridDim.x >> 3) {
    __syncthreads();
    find_item(i, ntn, tiles_before, g.counts, g.offsets, g.E, item);
    __syncthreads();
    Item it;
    it.expert = __builtin_amdgcn_readfirstlane(item[0]);
    it.row0 = __builtin_amdgcn_readfirstlane(item[1]);
    it.nrows = __builtin_amdgcn_readfirstlane(item[2]);
    it.nt = __builtin_amdgcn_readfirstlane(item[3]);
    const int live = (it.nrows + 15) >> 4;
    auto run = [&](auto n) {
      constexpr int NMB = decltype(n)::value;
      if constexpr (TRANS) t_item<WF32, MB, NMB>(g, it, b0, b1, sc, wt);
      else nt_item<WF32, MB, NMB>(g, it, As, sc, wt);
    };
    using std::integral_constant;
    if constexpr (MB == 4) {
      if (live > 2) run(integral_constant<int, 4>{});
      else if (live > 1) run(integral_constant<int, 2>{});
      else run(integral_constant<int, 1>{});
    } else {
      if (live > 1) run(integral_constant<int, 2>{});
      else run(integral_constant<int, 1>{});
    }
  }
}

// ---- large tiles
// 288 rows x 256 columns on eight wavefronts, two (halves of the rows) by four
// (64 columns each): the most that the accumulators (144 registers a lane) and
// two LDS stages of rows and weights (68 KiB each) leave room for.  A step's 36
// matrix instructions on each of 8 wavefronts take 2304 cycles a CU, its LDS
// reads (a row block by four wavefronts, a weight by two) and copies 2208 at 128
// bytes a cycle, so neither waits long for the other; the rest of the time goes
// into bringing 68 KiB a step to each CU.  8192 tokens, top-8 of 256 experts of
// [4096][7168]: y = a W^T 1.88 ms (2.05 Pop/s), y = a W 2.11 ms (1.82 Pop/s);
// without the copies 1.09 and 1.28 ms, with a quarter of the matrix instructions
// 1.79 and 2.1 ms.  On the way here tiles of 256 rows, which half of these
// experts exceed, took 2.38 ms against 2.18; a step that read its weights from
// LDS at its start 2.18 and 2.57 against 2.08 and 2.26.  Weights go past the
// caches: 7 % less time where an expert is one tile (its rows stay in L2), 0 to
// 2 % more where several tiles share them.
constexpr int kBigBlocks = 18;
struct BigStage {
  uint8_t* a;                                    // [256][128]
  uint8_t* w;                                    // y = a W^T: [256 columns][128]
};                                               // y = a W: [128][256 columns]

template <bool TRANS, bool WF32, int NMB>
__device__ __forceinline__ void big_item(const Fp8GemmArgs& g, const Item& it, const BigStage& s0,
                                         const BigStage& s1, uint8_t* sc, uint32_t* wt) {
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int i16 = lane & 15, q = lane >> 4;
  const int half = wave >> 2, nq = wave & 3;
  const int blocks = (it.nrows + 15) >> 4, h0 = (blocks + 1) >> 1;   // blocks of the first half
  const int red = TRANS ? g.N : g.K, cols = TRANS ? g.K : g.N;
  const int steps = (red + 127) >> 7;

  // row copies: slot tid & 7 of rows 64 i + tid / 8
  const uint32_t abytes = (uint32_t)(g.a_rows * red);
  const int acol = ((tid & 7) ^ swz_a(tid >> 3)) * 16;
  uint32_t aoff[NMB > 8 ? 5 : 4];
#pragma unroll
  for (int i = 0; i < (NMB > 8 ? 5 : 4); ++i) {
    const int r = 64 * i + (tid >> 3);
    const int rr = it.row0 + (r < it.nrows ? r : 0);
    const uint32_t src = g.tokens ? g.perm[rr] / g.topk : rr;
    aoff[i] = src * (uint32_t)red + (uint32_t)acol;
  }
  // weight copies
  const uint32_t wbytes = (uint32_t)g.N * (uint32_t)g.K;
  const uint8_t* wbase = g.w + (int64_t)it.expert * wbytes;
  uint32_t woff;
  if constexpr (TRANS) {
    // four rows of 256 bytes at a time; slot s of row r holds chunk s ^ swz_t(r)
    const int r = (wave >> 2) * 64 + (wave & 3) * 4 + (lane >> 4);
    const int chunk = (lane & 15) ^ swz_t(r);
    const int c = min(it.nt * 256 + 64 * (chunk >> 2), cols - 64);
    woff = (uint32_t)r * (uint32_t)g.K + (uint32_t)(c + 16 * (chunk & 3));
  } else {
    woff = (uint32_t)(tid >> 3) * (uint32_t)g.K + (uint32_t)(((tid & 7) ^ swz_w(tid >> 3)) * 16);
  }
  // (copies that are not wanted, of rows past the tile or steps past the piece,
  // read an empty buffer: no branches, and every step issues the same number)
  auto copy_a = [&](int st, bool live, const BigStage& s) {
    const bool in = TRANS ? st * 128 + acol < red : true;
    const uint32_t at = live ? (uint32_t)st * 128u : 0u;
    auto copy = [&](int i, bool wanted) {
      copy16_to_lds(raw_buffer(g.a, wanted ? abytes : 0u), in ? aoff[i] : 0xFFFFFFF0u - at, at,
                    s.a + (512 * i + 64 * wave) * 16);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) copy(i, live && 4 * i < blocks);
    if (NMB > 8 && wave < 4) copy(4, live);      // rows 256 .. 287
  };
  auto copy_w = [&](int st, bool live, const BigStage& s) {
    const __amdgpu_buffer_rsrc_t rsrc = raw_buffer(wbase, live ? wbytes : 0u);
    const uint32_t s0 = live ? st : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TRANS) {
        // W rows past N lie past the buffer's end
        copy16_to_lds<kStreamed>(rsrc, woff + (s0 * 128u + 16u * i) * (uint32_t)g.K, 0,
                      s.w + ((wave >> 2) * 64 + (wave & 3) * 4 + 16 * i) * 256);
      } else {
        const uint32_t c = min(it.nt * 256 + 64 * i, cols - 64);
        copy16_to_lds<kStreamed>(rsrc, woff, c * (uint32_t)g.K + s0 * 128u,
                      s.w + (512 * i + 64 * wave) * 16);
      }
    }
  };

  const int base = it.nt * 256 + nq * 64;
  const bool active = base < cols;
  const int cbase = active ? base : cols - 64;
  const int KB = g.K >> 7;
  const int64_t sat = TRANS ? (int64_t)it.expert * steps * KB + (cbase >> 7)
                            : ((int64_t)it.expert * ((g.N + 127) >> 7) + (cbase >> 7)) * steps;
  const int at = rows_at(i16, q);
  const int ah = at + half * h0 * 2048;
  const int tr_row = 64 * (q & 1) + 32 * (q >> 1) + (i16 >> 1);
  const int tr_at = tr_row * 256 + (((4 * nq) ^ swz_t(tr_row)) << 4) + (i16 & 1) * 8;

  f32x4_t acc[NMB][4];
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb)
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto read_w = [&](const BigStage& s, int nb, WStep& w) {
    if constexpr (TRANS) {
      // reduced values 64 (q & 1) + 32 (q / 2) + 8 t .. + 7, columns 16 nb ..:
      // row r = tr_row + 8 t, chunk 4 nq + nb, whose slot differs by swz_t(r)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const i32x2_t v = lds_tr8(s.w + ((tr_at ^ (nb << 4)) + t * 2048));
        w.w[nb][2 * t] = v[0];
        w.w[nb][2 * t + 1] = v[1];
      }
    } else {
      // MFMA row i of block nb is column 16 (i / 4) + 4 nb + (i & 3)
      const int r = nq * 64 + 16 * (i16 >> 2) + 4 * nb + (i16 & 3);
      const int o = r * 128 + (((4 * (q & 1) + 2 * (q >> 1)) ^ swz_w(r)) << 4);
      const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(s.w + o);
      const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(s.w + (o ^ 16));
      w.w[nb] = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                        (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    }
  };
  // Step i of n: its weights are in registers and its rows in s; rows of step
  // i + 1 go to t.  The last two row blocks run column block by column block,
  // and the registers of each one's weights are loaded for the next step behind
  // its last use: the matrix core works on while LDS delivers them.  So the
  // weights of step i + 2 (which come from memory) can start with step i, the
  // rows of step i + 1 (which the L2 mostly holds) too.
  WStep w;
  auto step = [&](int st0, int i, int n, const BigStage& s, const BigStage& t) {
    copy_a(st0 + i + 1, i + 1 < n, t);
    compiler_fence();                            // the waits below count on this order
    copy_w(st0 + i + 2, i + 2 < n, s);
    compiler_fence();
    int xs[3];
    const uint2 v = *reinterpret_cast<const uint2*>(sc + ((i * 2 + half) * 16 + i16) * 8);
    xs[0] = (int)v.x;
    xs[1] = (int)v.y;
    xs[2] = NMB > 8 ? sc[kPiece * 256 + (i * 2 + half) * 16 + i16] : 0;
    const uint32_t ws = wt[nq * kPiece + i];
    i32x8_t x = read_rows(s.a, 0, ah);
    auto row_block = [&](auto mbc) {
      constexpr int mb = decltype(mbc)::value;
      if constexpr (mb + 2 < NMB) {
        const i32x8_t nx = read_rows(s.a, mb + 1, ah);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          mfma_block<WF32, (mb & 3)>(w.w[nb], x, ws, xs[mb >> 2], acc[mb][nb]);
        x = nx;
      }
    };
    using std::integral_constant;
    row_block(integral_constant<int, 0>{});
    row_block(integral_constant<int, 1>{});
    row_block(integral_constant<int, 2>{});
    row_block(integral_constant<int, 3>{});
    row_block(integral_constant<int, 4>{});
    row_block(integral_constant<int, 5>{});
    row_block(integral_constant<int, 6>{});
    const i32x8_t y = read_rows(s.a, NMB - 1, ah);
    stage_barrier<8>();                          // weights of step i + 1 have landed
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      mfma_block<WF32, ((NMB - 2) & 3)>(w.w[nb], x, ws, xs[(NMB - 2) >> 2], acc[NMB - 2][nb]);
      mfma_block<WF32, ((NMB - 1) & 3)>(w.w[nb], y, ws, xs[(NMB - 1) >> 2], acc[NMB - 1][nb]);
      read_w(t, nb, w);
    }
    stage_barrier<4>();                          // and its rows
  };

  const bool words = (steps & 3) == 0 && (reinterpret_cast<uintptr_t>(g.a_scales) & 3) == 0;
  for (int st0 = 0; st0 < steps; st0 += kPiece) {
    const int n = min(kPiece, steps - st0);
    copy_a(st0, true, s0);
    copy_w(st0, true, s0);
    copy_w(st0 + 1, n > 1, s1);
    // scales: sc[step][half][row & 15][block of the half], those of a ninth block
    // behind them, wt[column group][step]
    for (int v = tid; v < 32 * blocks; v += 512) {
      const int r = v >> 1, b = r >> 4, hb = b >= h0;
      const int rr = it.row0 + (r < it.nrows ? r : 0);
      const int64_t src = g.tokens ? g.perm[rr] / g.topk : rr;
      const uint8_t* row = g.a_scales + src * steps + st0;
      const int k = b - hb * h0, at = hb * 16 + (r & 15);
      uint8_t* out = sc + (k < 8 ? at * 8 + k : kPiece * 256 + at);
      const int stride = k < 8 ? 256 : 32;
      if (words) {                               // n is a multiple of 4 then
#pragma unroll 8
        for (int w = v & 1; w < n / 4; w += 2) {
          const uint32_t x = reinterpret_cast<const uint32_t*>(row)[w];
#pragma unroll
          for (int j = 0; j < 4; ++j) out[(4 * w + j) * stride] = (uint8_t)(x >> (8 * j));
        }
      } else {
#pragma unroll 8
        for (int j = v & 1; j < n; j += 2) out[j * stride] = row[j];
      }
    }
    if (half == 0)
      for (int j = lane; j < n; j += 64) {
        const int64_t si = sat + (int64_t)(st0 + j) * (TRANS ? KB : 1);
        wt[nq * kPiece + j] = WF32 ? static_cast<const uint32_t*>(g.w_scales)[si]
                                   : static_cast<const uint8_t*>(g.w_scales)[si];
      }
    stage_barrier<0>();
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) read_w(s0, nb, w);
    stage_barrier<63>();
#pragma nounroll
    for (int i = 0; i < n; i += 2) {
      step(st0, i, n, s0, s1);
      if (i + 1 >= n) break;
      step(st0, i + 1, n, s1, s0);
    }
    stage_barrier<0>();
  }
  if (!active) return;
#pragma unroll
  for (int mb = 0; mb < NMB; ++mb) {
    const int r = 16 * (half * h0 + mb) + i16;
    if (r >= it.nrows || (half == 0 && mb >= h0)) continue;
    uint16_t* out = g.y + (int64_t)(it.row0 + r) * cols + cbase;
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

template <bool TRANS, bool WF32>
__global__ __launch_bounds__(512, 1) void k_fp8_gemm_big(Fp8GemmArgs g, int ntn) {
  __shared__ __attribute__((aligned(16))) uint8_t a0[36864];
  __shared__ __attribute__((aligned(16))) uint8_t a1[36864];
  __shared__ __attribute__((aligned(16))) uint8_t w0[32768];
  __shared__ __attribute__((aligned(16))) uint8_t w1[32768];
  __shared__ __attribute__((aligned(16))) uint8_t sc[kPiece * 288];
  __shared__ uint32_t wt[4 * kPiece];
  __shared__ int tiles_before[1025];
  __shared__ int scratch[16];
  __shared__ int item[4];
  const BigStage s0{a0, w0}, s1{a1, w1};
  count_tiles(g.counts, g.E, 16 * kBigBlocks, tiles_before, scratch);
  const int items = tiles_before[g.E] * ntn;
  const int per = (items + 7) >> 3;
  const int first = (blockIdx.x & 7) * per, last = min(first + per, items);
  for (int i = first + (blockIdx.x >> 3); i < last; i += gridDim.x >> 3) {
    __syncthreads();
    find_item(i, ntn, tiles_before, g.counts, g.offsets, g.E, item);
    __syncthreads();
    Item it;
    it.expert = __builtin_amdgcn_readfirstlane(item[0]);
    it.row0 = __builtin_amdgcn_readfirstlane(item[1]);
    it.nrows = __builtin_amdgcn_readfirstlane(item[2]);
    it.nt = __builtin_amdgcn_readfirstlane(item[3]);
    const int h0 = (((it.nrows + 15) >> 4) + 1) >> 1;
    auto run = [&](auto n) {
      big_item<TRANS, WF32, decltype(n)::value>(g, it, s0, s1, sc, wt);
    };
    using std::integral_constant;
    if (h0 > 8) run(integral_constant<int, 9>{});
    else if (h0 > 6) run(integral_constant<int, 8>{});
    else if (h0 > 5) run(integral_constant<int, 6>{});
    else if (h0 > 4) run(integral_constant<int, 5>{});
    else if (h0 > 2) run(integral_constant<int, 4>{});
    else run(integral_constant<int, 2>{});
  }
}

// 16-row blocks per tile (an expert has at most one row per token, so up to 64
// tokens every expert fits one tile of four).  Measured with weights [64][4096]
// [7168], top-8, y = a W^T and y = a W, in us:
//   mean rows             24         48         72        100
//   four blocks     310 / 348  325 / 372  587 / 600  592 / 578
//   eighteen        334 / 388  347 / 390  370 / 411  379 / 430
// Two blocks leave registers for four steps of weights in flight instead of two.
// That pays where the items do not fill the card (one token: 55 us against 66),
// not beside another workgroup on the same CU (4 tokens 136 against 132, 16 tokens
// 266 against 253).
int tile_blocks(const Fp8GemmArgs& g, int ntn) {
  if (!g.trans && g.T <= 32 && std::min<int64_t>(g.P, g.E) * ntn <= num_cus()) return 2;
  return g.T <= 64 || (g.P + g.E - 1) / g.E <= 64 ? 4 : kBigBlocks;
}

}  // namespace

template <bool TRANS, bool WF32>
static void launch_sized(const Fp8GemmArgs& g, hipStream_t s) {
  const int ntn = ((TRANS ? g.K : g.N) + 255) / 256;
  const int mb = tile_blocks(g, ntn);
  const int64_t tiles = std::min<int64_t>(g.P, g.P / (16 * mb) + g.E);
  // a multiple of 8: one stretch of items per XCD
  const int64_t items = (tiles * ntn + 7) / 8 * 8, cus = num_cus() / 8 * 8;
  const dim3 grid((unsigned)std::min<int64_t>(items, mb == kBigBlocks ? cus : 2 * cus));
  if (mb == kBigBlocks)
    hipLaunchKernelGGL((k_fp8_gemm_big<TRANS, WF32>), grid, dim3(512), 0, s, g, ntn);
  else if (mb == 4)
    hipLaunchKernelGGL((k_fp8_gemm<TRANS, WF32, 4>), grid, dim3(256), 0, s, g, ntn);
  else if constexpr (!TRANS)
    hipLaunchKernelGGL((k_fp8_gemm<TRANS, WF32, 2>), grid, dim3(256), 0, s, g, ntn);
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
