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
// Scores and choice values are formed in double: a choice is a comparison of
// nearby numbers, and rounding s to 24 bits would turn near values into ties
// or swap them (about two tokens in a batch of 8192 with 256 experts).
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

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

__device__ __forceinline__ double read_lane_f64(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// One wavefront per token; lane l holds experts l, l + 64, ... (NV of them).
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
  float l[NV];
  double s[NV], c[NV];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    l[i] = -INFINITY;
    if (e < E) {
      const float x = load_logit(row + e);
      if (__builtin_isfinite(x)) l[i] = x;
      else bad = true;
    }
  }
  if (o.softmax) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
    m = wave_max_f32(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)m);
      sum += s[i];
    }
    sum = wave_sum_f64(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = l[i] == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    c[i] = l[i] == -INFINITY ? -INFINITY : s[i];
    if (bias && e < E) {
      const float b = bias[e];
      if (!__builtin_isfinite(b)) {
        bad = true;
        c[i] = -INFINITY;
      } else {
        c[i] += (double)b;
      }
    }
  }
  if (__any(bad) && lane == 0 && err) atomicOr(err, 1);

  uint64_t key[NV];                              // 0: not a candidate
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = lane + 64 * i < E ? order_key64(c[i]) : 0;

  if (o.topk_group < o.n_group) {
    double* mine = row_lds + (int64_t)wave * E;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 64 * i < E) mine[lane + 64 * i] = c[i];
    wave_lds_sync();
    const int size = E / o.n_group;
    // 2^sh lanes a group: the largest power of two that gives every group its lanes
    int sh = 0;
    while ((o.n_group << (sh + 1)) <= 64) ++sh;
    const int per = 1 << sh;
    const int g = lane >> sh, sub = lane & (per - 1);
    double b1 = -INFINITY, b2 = -INFINITY;       // the group's two best
    if (g < o.n_group)
      for (int i = sub; i < size; i += per) {
        const double v = mine[g * size + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    for (int off = 1; off < per; off <<= 1) {
      const double o1 = __shfl_xor(b1, off, kWave), o2 = __shfl_xor(b2, off, kWave);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    const double score = o.group_top == 2 ? b1 + b2 : b1;
    int rank = 0;
    for (int j = 0; j < o.n_group; ++j) {
      const double other = read_lane_f64(score, j << sh);
      rank += other > score || (other == score && j < g);
    }
    const uint64_t kept = __ballot(rank < o.topk_group && sub == 0 && g < o.n_group);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((kept >> ((e / size) << sh)) & 1)) key[i] = 0;
    }
  }

  // k rounds of a wavefront arg-max; among equal values the lowest id
  uint64_t best = 0;
  int best_i = 0;
  double best_s = 0.0;
  auto lane_best = [&]() {
    best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) {
        best = key[i];
        best_i = i;
        best_s = s[i];
      }
  };
  lane_best();
  int my_id = 0;
  double my_w = 0.0, sum = 0.0;
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
    const double w = read_lane_f64(best_s, win);
    sum += w;
    if (lane == j) {
      my_id = id;
      my_w = w;
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i == best_i) key[i] = 0;
      lane_best();
    }
  }
  if (lane < k) {
    double w = my_w;
    if (o.renorm) w = sum > 0.0 ? w / sum : 0.0;
    ids[(int64_t)t * k + lane] = my_id;
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
