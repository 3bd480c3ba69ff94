// Scored routing: softmax or sigmoid scores, a balance bias that enters the
// choice only, groups of experts, top-k, renormalised gates; and its backward.
//
// For one token with logits l[0..E):
//   s_e = exp(l_e - max l) / sum exp(l - max l)   or   1 / (1 + exp(-l_e))
//   c_e = s_e + bias_e                            (the choice value)
//   group score = sum of the group's group_top largest c; the topk_group
//   largest groups stay (equal scores: lower group first)
//   the k largest c of the kept groups, equal values in ascending id
//   w_j = s[id_j], divided by their sum when renorm, times scale.
// The choice is that of scores and choice values in double: it compares nearby
// numbers, and in 24 bits near values become ties or swap (about two tokens in
// a batch of 8192 with 256 experts).  Few comparisons need that, though, so a
// token is first decided in fp32, by the logits themselves where no bias enters
// (both scores grow with them) and else by fp32 choice values; where two
// neighbours of the order, the last kept and the first dropped, or two groups
// lie closer than the error of what was compared, the token is decided again
// in double.
#include "qgg_device.hpp"
#include "qgg_internal.hpp"

namespace qgg {

namespace {

template <typename L>
__device__ __forceinline__ float load_logit(const L* p) {
  if constexpr (sizeof(L) == 4) return *p;
  else return bf16_to_f32(*p);
}

// double -> uint64 with the same order; every value, -inf included, maps above 0
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto step = [&](auto ctrl, auto rows) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                     decltype(rows)::value, 0xF, false));
  };
  using std::integral_constant;
  step(integral_constant<int, 0xB1>{}, integral_constant<int, 0xF>{});   // quad_perm 1,0,3,2
  step(integral_constant<int, 0x4E>{}, integral_constant<int, 0xF>{});   // quad_perm 2,3,0,1
  step(integral_constant<int, 0x141>{}, integral_constant<int, 0xF>{});  // row_half_mirror
  step(integral_constant<int, 0x140>{}, integral_constant<int, 0xF>{});  // row_mirror
  step(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast:15
  step(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast:31
  return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// maximum of values that are not NaN
__device__ __forceinline__ float wave_max_f32(float v) {
  return key_value(wave_max_u32(order_key(v)));
}

__device__ __forceinline__ float wave_sum_f32(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wave_sum_63(v)), 63));
}

__device__ __forceinline__ double read_lane_f64(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ float read_lane_f32(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Layout of the groups over a wavefront: 2^sh lanes each, the largest power of
// two that gives every group its lanes.
__device__ __forceinline__ int group_shift(int n_group) {
  int sh = 0;
  while ((n_group << (sh + 1)) <= 64) ++sh;
  return sh;
}

// k rounds of a wavefront arg-max over the lanes' keys (0: no candidate); among
// equal keys the lowest id.  Lane j < k ends with the j-th id.
template <int NV>
__device__ __forceinline__ int take64(uint64_t (&key)[NV], int k, int lane) {
  uint64_t best = 0;
  int best_i = 0, my_id = 0;
  auto lane_best = [&]() {
    best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) {
        best = key[i];
        best_i = i;
      }
  };
  lane_best();
  for (int j = 0; j < k; ++j) {
    const uint64_t top = wave_max_u64(best);
    uint64_t holders = __ballot(best == top);
    int win = __ffsll((unsigned long long)holders) - 1;
    int id = 64 * __builtin_amdgcn_readlane(best_i, win) + win;
    for (holders &= holders - 1; holders; holders &= holders - 1) {
      const int h = __ffsll((unsigned long long)holders) - 1;
      const int hid = 64 * __builtin_amdgcn_readlane(best_i, h) + h;
      if (hid < id) {
        id = hid;
        win = h;
      }
    }
    if (lane == j) my_id = id;
    if (lane == win) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == best_i) key[i] = 0;
      lane_best();
    }
  }
  return my_id;
}

// The same on 32-bit keys whose low four bits are 15 - i (entry i of a lane is
// expert 64 i + lane): the key itself then says which entry it is, and equal
// values go to the lower id by the order of keys and lanes alone.  Each lane
// sorts its keys once, so that a round looks at one key a lane and the lane that
// gives one moves up the rest.  Lane j <= k ends with the j-th key in *order
// (the k-th one not taken; 0: none left).
constexpr uint32_t kEntry = 15;

template <int NV>
__device__ __forceinline__ void sort_down(uint32_t (&v)[NV]) {
#pragma unroll
  for (int size = 2; size <= NV; size *= 2)      // bitonic
#pragma unroll
    for (int step = size / 2; step; step /= 2)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i ^ step;
        if (j > i) {
          const uint32_t hi = max(v[i], v[j]), lo = min(v[i], v[j]);
          const bool down = (i & size) == 0;
          v[i] = down ? hi : lo;
          v[j] = down ? lo : hi;
        }
      }
}

template <int NV>
__device__ __forceinline__ int take32(uint32_t (&key)[NV], int k, int lane, uint32_t* order) {
  sort_down<NV>(key);
  uint32_t keys = 0;
  int ids = 0;
  for (int j = 0;; ++j) {
    const uint32_t top = wave_max_u32(key[0]);
    keys = lane == j ? top : keys;
    if (j == k) break;
    const int win = __ffsll((unsigned long long)__ballot(key[0] == top)) - 1;
    ids = lane == j ? 64 * (int)(kEntry - (top & kEntry)) + win : ids;
    const bool mine = lane == win;
#pragma unroll
    for (int i = 0; i + 1 < NV; ++i) key[i] = mine ? key[i + 1] : key[i];
    key[NV - 1] = mine ? 0u : key[NV - 1];
  }
  *order = keys;
  return ids;
}

// The value of a lane of the other half of a block of 2 off lanes, all of whose
// halves are uniform.
__device__ __forceinline__ int partner_bits(int v, int off) {
  switch (off) {
    case 1: return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);    // quad_perm 1,0,3,2
    case 2: return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);    // quad_perm 2,3,0,1
    case 4: return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);   // row_half_mirror
    case 8: return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);   // row_mirror
    default: return __shfl_xor(v, off, kWave);
  }
}
__device__ __forceinline__ float partner(float v, int off) {
  return __int_as_float(partner_bits(__float_as_int(v), off));
}
__device__ __forceinline__ double partner(double v, int off) {
  const long long u = __double_as_longlong(v);
  const uint32_t lo = partner_bits((int)(u & 0xFFFFFFFF), off);
  const uint32_t hi = partner_bits((int)(u >> 32), off);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Two best of each group from the wavefront's row of choice values: the lane's
// group holds them in all of its lanes afterwards.
template <typename F>
__device__ __forceinline__ void group_best(const F* row, int size, int n_group, int sh, int lane,
                                           F& b1, F& b2) {
  const int per = 1 << sh, g = lane >> sh;
  b1 = b2 = -INFINITY;
  if (g < n_group)
    for (int i = lane & (per - 1); i < size; i += per) {
      const F v = row[g * size + i];
      b2 = max(b2, min(b1, v));
      b1 = max(b1, v);
    }
  for (int off = 1; off < per; off <<= 1) {
    const F o1 = partner(b1, off), o2 = partner(b2, off);
    b2 = max(min(b1, o1), max(b2, o2));
    b1 = max(b1, o1);
  }
}

__device__ __forceinline__ float lane_value(float v, int lane) { return read_lane_f32(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) { return read_lane_f64(v, lane); }

// Kept groups as bits g << sh: the topk_group largest scores, the lower group
// first among equals.
template <typename F>
__device__ __forceinline__ uint64_t keep_groups(F score, const RouteOpts& o, int sh, int lane) {
  const int g = lane >> sh;
  int rank = 0;
  for (int j = 0; j < o.n_group; ++j) {
    const F other = lane_value(score, j << sh);
    rank += other > score || (other == score && j < g);
  }
  return __ballot(rank < o.topk_group && (lane & ((1 << sh) - 1)) == 0 && g < o.n_group);
}

// The choice in double.
template <int NV>
__device__ __forceinline__ int choose64(const float (&l)[NV], const float* bias, int E, int k,
                                         const RouteOpts& o, int lane, double* row) {
  double c[NV];
  if (o.softmax) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
    m = wave_max_f32(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)m);
      sum += c[i];
    }
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = sum > 0.0 ? c[i] / sum : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  uint64_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    const float b = bias && e < E ? bias[e] : 0.f;
    c[i] = l[i] == -INFINITY || !__builtin_isfinite(b) ? -INFINITY : c[i] + (double)b;
    key[i] = e < E ? order_key64(c[i]) : 0;
  }
  if (o.topk_group < o.n_group) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i < E) row[lane + 64 * i] = c[i];
    wave_lds_sync();
    const int size = E / o.n_group, sh = group_shift(o.n_group);
    double b1, b2;
    group_best(row, size, o.n_group, sh, lane, b1, b2);
    const uint64_t kept = keep_groups(o.group_top == 2 ? b1 + b2 : b1, o, sh, lane);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (o.group_of(e) << sh)) & 1)) key[i] = 0;
    }
  }
  return take64<NV>(key, k, lane);
}

// The choice in fp32; *sure is false where a comparison that decided lies
// within its error.  Errors, in absolute terms: a sigmoid is off by (|l| + 6)
// half steps of e / (1 + e)^2 or of itself, under 8 in all (2^-21); a softmax
// by |l - max| + 24 half steps of p, under 25 (2^-19); the bias adds half a
// step of the sum, the cut of a key's low bits 2^-20 of what it holds.  EXACT:
// the logits are BF16, which the cut leaves whole, so that equal keys are equal
// logits.
template <int NV, bool EXACT, typename LoadL>
__device__ __forceinline__ int choose32(const float (&l)[NV], const float* bias, int E, int k,
                                         const RouteOpts& o, int lane, float* row, LoadL load_l, bool* sure) {
  const bool grouped = o.topk_group < o.n_group;
  const bool by_score = bias || (grouped && o.group_top == 2);
  const float err = o.softmax ? 0x1p-19f : 0x1p-21f;
  float x[NV], c[NV];                            // what orders experts; what orders groups
  float m = -INFINITY;
  if (o.softmax && by_score) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
    m = wave_max_f32(m);
  }
  if (by_score) {
    if (o.softmax) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        c[i] = l[i] == -INFINITY ? 0.f : __expf(l[i] - m);
        sum += c[i];
      }
      sum = wave_sum_f32(sum);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] *= inv;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      const float b = bias && e < E ? bias[e] : 0.f;
      c[i] = l[i] == -INFINITY || !__builtin_isfinite(b) ? -INFINITY : c[i] + b;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = bias ? c[i] : l[i];
    if (!by_score) c[i] = l[i];
  }
  bool ok = true;
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)                   // -0 -> +0; above 0 even for -inf
    key[i] = lane + 64 * i < E ? (order_key(x[i] + 0.0f) & ~kEntry) | (kEntry - i) : 0;
  if (grouped) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i < E) row[lane + 64 * i] = c[i];
    wave_lds_sync();
    const int size = E / o.n_group, sh = group_shift(o.n_group);
    float b1, b2;
    group_best(row, size, o.n_group, sh, lane, b1, b2);
    const float score = o.group_top == 2 ? b1 + b2 : b1;
    const uint64_t kept = keep_groups(score, o, sh, lane);
    float lo = INFINITY, hi = -INFINITY;         // lowest kept, highest dropped
    for (int j = 0; j < o.n_group; ++j) {
      const float v = read_lane_f32(score, j << sh);
      if ((kept >> (j << sh)) & 1) lo = fminf(lo, v);
      else hi = fmaxf(hi, v);
    }
    if (by_score) ok = lo == hi ? lo == -INFINITY
                                : lo - hi > 4.0f * err + 0x1p-21f * fmaxf(fabsf(lo), fabsf(hi));
    else ok = lo == hi || lo - hi > 1e-9f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> (o.group_of(e) << sh)) & 1)) key[i] = 0;
    }
  }
  uint32_t order;
  const int id = take32<NV>(key, k, lane, &order);
  // lane j in 1 .. k compares the j-th value with the one before it
  const float v = key_value(order & ~kEntry);
  const float prev = __shfl_up(v, 1, kWave);
  const bool next = lane >= 1 && lane <= k && order != 0;
  bool close;
  if (bias) {
    close = !(prev - v > 2.0f * err + 0x1p-18f * fmaxf(fabsf(prev), fabsf(v)));
    // softmax gates are formed from the kept logits alone; where the whole
    // row's sum would round their scores to zero, the other path says so
    if (o.softmax && lane < k && !(load_l(id) - m > -600.0f)) ok = false;
  } else {
    // logits order as their scores do in double, unless they are so near, or
    // so large or small, that scores round to one number
    const float top = o.softmax ? (by_score ? m : read_lane_f32(v, 0)) : 0.f;
    close = EXACT ? prev != v && !(prev - v > 1e-9f)
                  : !(prev - v > 1e-9f + 0x1p-18f * fmaxf(fabsf(prev), fabsf(v)));
    close |= !(v - top > -600.0f) || (!o.softmax && prev > 20.0f);
  }
  ok &= !(next && close);
  ok = __all(ok);
  *sure = ok;
  return id;
}

// One wavefront per token; lane l holds experts l, l + 64, ... (NV of them).
// Bound by latency: k dependent rounds of a reduction over the lanes.  64 tokens,
// 384 experts, softmax: 6.5 us against 9.2 with 64-bit keys through LDS permutes;
// 8192 tokens, 256 experts in 8 groups, sigmoid: 18 us, where 8.9 MB are the
// bytes of 2 us.
template <int NV, typename L>
__global__ __launch_bounds__(256) void k_route_scored(const L* __restrict__ logits,
                                                      const float* __restrict__ bias, int T, int E,
                                                      int k, RouteOpts o,
                                                      int32_t* __restrict__ ids,
                                                      float* __restrict__ gates,
                                                      int32_t* __restrict__ err) {
  extern __shared__ double row_lds[];            // [4][E] choice values (grouped choice only)
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= T) return;
  const L* row = logits + (int64_t)t * E;
  double* mine = row_lds + (int64_t)wave * E;
  float l[NV];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = -INFINITY;
    if (e < E) {
      const float x = load_logit(row + e);
      if (__builtin_isfinite(x)) l[i] = x;
      else bad = true;
      if (err && bias && !__builtin_isfinite(bias[e])) bad = true;
    }
  }
  if (err && __any(bad) && lane == 0) atomicOr(err, 1);

  auto load_l = [&](int e) {
    const float x = load_logit(row + e);
    return __builtin_isfinite(x) ? x : -INFINITY;
  };
  bool sure;
  int id = choose32<NV, sizeof(L) == 2>(l, bias, E, k, o, lane, reinterpret_cast<float*>(mine),
                                        load_l, &sure);
  if (!sure) {
    wave_lds_sync();
    id = choose64<NV>(l, bias, E, k, o, lane, mine);
  }
  const float kl = lane < k ? load_l(id) : -INFINITY;
  double m = 0.0, total = 1.0;                   // softmax: maximum and sum of the row
  if (o.softmax) {
    if (o.renorm && sure) {                      // any common factor cancels
      m = (double)wave_max_f32(kl);
    } else {
      float top = l[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
      m = (double)wave_max_f32(top);
      total = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i) total += l[i] == -INFINITY ? 0.0 : exp((double)l[i] - m);
      total = wave_sum_f64(total);
    }
  }
  double w = 0.0;
  if (kl != -INFINITY)
    w = o.softmax ? exp((double)kl - m) / total : 1.0 / (1.0 + exp(-(double)kl));
  if (o.renorm) {
    double sum = 0.0;
    for (int j = 0; j < k; ++j) sum += read_lane_f64(w, j);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < k) {
    ids[(int64_t)t * k + lane] = id;
    gates[(int64_t)t * k + lane] = (float)(w * (double)o.scale);
  }
}

// Backward of the gates with the choice held fixed: dlogits from dgates.
// Lane j < k owns the token's j-th kept expert.  With w = gate / scale:
//   sigmoid, renorm   dl_i = scale (dg_i - <dg, w>) w_i (1 - s_i)
//   sigmoid           dl_i = scale dg_i s_i (1 - s_i)
//   softmax, renorm   dl_i = scale (dg_i - <dg, w>) w_i
//   softmax           dl_e = scale p_e (dg_e - <dg, p>) for every expert e
// An id that occurs twice gets the sum; ids outside [0, E) and experts whose
// logit is not finite contribute nothing.  The row is put together in LDS and
// stored once.  Kept scores are formed in double (at most 32 a token), the
// dense softmax in fp32.
template <int NV, typename L>
__global__ __launch_bounds__(256) void k_route_scored_bwd(const L* __restrict__ logits,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ dgates, int T,
                                                          int E, int k, RouteOpts o,
                                                          L* __restrict__ dlogits) {
  extern __shared__ float grad_lds[];            // [4][E]
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= T) return;
  const L* row = logits + (int64_t)t * E;
  float* acc = grad_lds + (int64_t)wave * E;
  int id = -1;
  float dg = 0.f, lj = -INFINITY;
  if (lane < k) {
    id = ids[(int64_t)t * k + lane];
    if (id < 0 || id >= E) id = -1;
    else {
      lj = load_logit(row + id);
      if (!__builtin_isfinite(lj)) lj = -INFINITY;
      else dg = dgates[(int64_t)t * k + lane];
    }
  }
  const bool live = lj != -INFINITY;
  const bool dense = o.softmax && !o.renorm;
  double v = 0.0;                                // this lane's share of dl[id] / scale
  float p[NV];
  float inner = 0.f;                             // <dg, p> of the dense form
  if (!dense) {
    double w, slope = 1.0;
    if (o.softmax) {
      const float m = wave_max_f32(lj);
      w = live ? exp((double)lj - (double)m) : 0.0;
    } else {
      const double z = live ? exp(-fabs((double)lj)) : 0.0;      // both forms without overflow
      const double big = 1.0 / (1.0 + z), small = z / (1.0 + z);
      w = !live ? 0.0 : (lj >= 0.f ? big : small);
      slope = lj >= 0.f ? small : big;
    }
    if (o.renorm) {
      const double sum = wave_sum_f64(w);
      w = sum > 0.0 ? w / sum : 0.0;
      v = ((double)dg - wave_sum_f64((double)dg * w)) * w * slope;
    } else {
      v = (double)dg * w * slope;
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      p[i] = e < E ? load_logit(row + e) : -INFINITY;
      if (!__builtin_isfinite(p[i])) p[i] = -INFINITY;
      m = fmaxf(m, p[i]);
    }
    m = wave_max_f32(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = p[i] == -INFINITY ? 0.f : expf(p[i] - m);
      sum += p[i];
    }
    sum = wave_sum_f32(sum);
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] *= inv;
    v = live ? (double)dg * (double)(expf(lj - m) * inv) : 0.0;
    inner = wave_sum_f32((float)v);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    if (e < E) acc[e] = dense ? -p[i] * inner : 0.f;
  }
  // shares of one id in ascending lane order; the first lane of an id adds them
  double total = 0.0;
  bool first = id >= 0;
  for (int j = 0; j < k; ++j) {
    const int other = __builtin_amdgcn_readlane(id, j);
    const double add = read_lane_f64(v, j);
    if (other == id) {
      total += add;
      if (j < lane) first = false;
    }
  }
  wave_lds_sync();
  if (first && lane < k) acc[id] += (float)total;
  wave_lds_sync();
  L* out = dlogits + (int64_t)t * E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    if (e < E) {
      const float g = o.scale * acc[e];
      if constexpr (sizeof(L) == 4) out[e] = g;
      else out[e] = (uint16_t)f32_to_bf16_rne(g);
    }
  }
}

}  // namespace

// f(NV) for the least NV in {1, 2, 4, 8, 16} with 64 NV >= E
template <typename F>
static void for_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 64) f(integral_constant<int, 1>{});
  else if (E <= 128) f(integral_constant<int, 2>{});
  else if (E <= 256) f(integral_constant<int, 4>{});
  else if (E <= 512) f(integral_constant<int, 8>{});
  else f(integral_constant<int, 16>{});
}

hipError_t launch_route_scored(const void* logits, bool bf16, const float* bias, int T, int E,
                               int k, const RouteOpts& o, int32_t* ids, float* gates, int32_t* err,
                               hipStream_t s) {
  TimedLaunch timed_(kLRoute, s);
  if (T == 0) return hipSuccess;
  const dim3 grid((T + 3) / 4);
  const size_t lds = o.topk_group < o.n_group ? (size_t)4 * E * sizeof(double) : 0;
  for_experts(E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (bf16)
      hipLaunchKernelGGL((k_route_scored<NV, uint16_t>), grid, dim3(256), lds, s,
                         static_cast<const uint16_t*>(logits), bias, T, E, k, o, ids, gates, err);
    else
      hipLaunchKernelGGL((k_route_scored<NV, float>), grid, dim3(256), lds, s,
                         static_cast<const float*>(logits), bias, T, E, k, o, ids, gates, err);
  });
  return hipGetLastError();
}

hipError_t launch_route_scored_bwd(const void* logits, bool bf16, const int32_t* ids,
                                   const float* dgates, int T, int E, int k, const RouteOpts& o,
                                   void* dlogits, hipStream_t s) {
  TimedLaunch timed_(kLRouterBwd, s);
  if (T == 0) return hipSuccess;
  const dim3 grid((T + 3) / 4);
  const size_t lds = (size_t)4 * E * sizeof(float);
  for_experts(E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (bf16)
      hipLaunchKernelGGL((k_route_scored_bwd<NV, uint16_t>), grid, dim3(256), lds, s,
                         static_cast<const uint16_t*>(logits), ids, dgates, T, E, k, o,
                         static_cast<uint16_t*>(dlogits));
    else
      hipLaunchKernelGGL((k_route_scored_bwd<NV, float>), grid, dim3(256), lds, s,
                         static_cast<const float*>(logits), ids, dgates, T, E, k, o,
                         static_cast<float*>(dlogits));
  });
  return hipGetLastError();
}

}  // namespace qgg
